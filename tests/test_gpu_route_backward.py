"""The routing's gradient on the GPU against its formulas in 64 bits
(tests/learn_ref.py), against torch's autograd of the routing, and on its
edges: masks, duplicate and bad experts, accumulation, no tokens, graphs."""
import pytest
import torch

import learn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import block_scaled_fp4_route_amd as m
    return m


class Case:
    def __init__(self, m, T, E, k, H, masked=0.0, seed=0):
        g = torch.Generator().manual_seed(7000 * T + 10 * E + k + H + seed)
        self.m, self.T, self.E, self.k, self.H = m, T, E, k, H
        rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.x, self.Wr, self.dw, self.din = rnd(T, H), rnd(E, H) * 0.02, rnd(T, k) * 0.1, rnd(T, E) * 1e-3
        top = torch.topk(rnd(T, E), k, dim=1)
        self.idx, self.w = top.indices.to(torch.int32), torch.softmax(top.values, 1)
        self.mask = (torch.rand(T, generator=g) >= masked) if masked else None

    def run(self, dw=True, din=True, dx=True, dWr=True, acc=0, before=None, inplace=False, ws=None):
        m, T, E, H, dev = self.m, self.T, self.E, self.H, "cuda"
        self.d = m.desc(H, 64, E, self.k, "nvfp4")
        up = lambda t: t.to(dev).contiguous()  # noqa: E731
        self.dev = [up(t) for t in (self.x, self.Wr, self.idx, self.w, self.dw, self.din)]
        x, Wr, idx, w, dwd, dind = self.dev
        md = None if self.mask is None else self.mask.to(torch.uint8).to(dev)
        before = before or {}
        out = {"dlogits": dind if inplace else torch.full((T, E), 7.0, device=dev),
               "dx": up(before["dx"]) if "dx" in before else torch.full((T, H), 7.0, device=dev),
               "dWr": up(before["dWr"]) if "dWr" in before else torch.full((E, H), 7.0, device=dev)}
        n = m.moe_route_backward_workspace_bytes(self.d, T)
        ws = torch.full((n,), 0xA5, dtype=torch.uint8, device=dev) if ws is None else ws
        self.args = (self.d, x, T, Wr, idx, w, dwd if dw else None, md, dind if din else None, out["dlogits"],
                     out["dx"] if dx else None, out["dWr"] if dWr else None, acc, ws)
        m.moe_route_backward(*self.args)
        torch.cuda.synchronize()
        return {"dlogits": out["dlogits"], "dx": out["dx"] if dx else None, "dWr": out["dWr"] if dWr else None}

    def want(self, dw=True, din=True):
        return ref.route_backward(self.x, self.Wr, self.idx, self.w, self.dw if dw else None, self.mask,
                                  self.din if din else None, self.T, self.E, self.k)

    def check(self, out, dw=True, din=True):
        want = self.want(dw, din)
        for name, v in out.items():
            if v is not None:
                ref.close(v, *want[name], name)


@pytest.mark.parametrize("T,E,k,H", [(1, 1, 1, 256), (1, 512, 10, 2560), (2, 5, 5, 256), (17, 384, 6, 4096), (33, 33, 3, 512),
                                     (64, 64, 8, 768), (127, 129, 2, 256), (129, 130, 32, 1280), (311, 384, 6, 512),
                                     (600, 512, 10, 256), (70, 1023, 7, 256), (40, 1024, 32, 8192), (5000, 9, 2, 256),
                                     (1100, 513, 10, 2560), (33, 260, 6, 4096), (4100, 130, 4, 1280), (40000, 20, 3, 256),
                                     (70, 1023, 7, 8192), (100000, 33, 3, 256), (4100, 300, 4, 2560), (600, 1024, 9, 1024)])
def test_shapes(m, T, E, k, H):
    c = Case(m, T, E, k, H)
    c.check(c.run())


@pytest.mark.parametrize("dw,din,dx,dWr", [(True, False, True, True), (False, True, True, True), (True, True, False, True),
                                           (True, True, True, False), (True, True, False, False)])
@pytest.mark.parametrize("T,E,H", [(90, 60, 512), (1100, 512, 1024)])
def test_parts_left_out(m, dw, din, dx, dWr, T, E, H):
    c = Case(m, T, E, 4, H, 0.2)
    c.check(c.run(dw, din, dx, dWr), dw, din)


def test_norm_of_the_error(m):
    """Beside the elementwise worst case: roundings of both signs add up like
    a random walk, sqrt(3 K) EPS / sqrt(3) of the products' norm for the sums
    and 2^-22 sqrt(3) for the operands' parts; four times that is allowed."""
    c = Case(m, 2451, 512, 10, 2560)
    out, want = c.run(), c.want()
    for name, K, a, b in (("dx", 512, want["dlogits"][0], c.Wr.double()), ("dWr", 2451, want["dlogits"][0].t(), c.x.double())):
        size = torch.sqrt((a ** 2) @ (b ** 2))  # root of the sum of squared products
        off = (out[name].cpu().double() - want[name][0]).norm() / size.norm()
        assert off <= 4 * (K ** 0.5 * ref.EPS + 3 ** 0.5 * 2.0 ** -22), (name, off)


@pytest.mark.parametrize("T,H", [(200, 512), (2300, 2560)])
def test_masked_rows_hold_anything(m, T, H):
    a, b = Case(m, T, 96, 5, H, 0.4), Case(m, T, 96, 5, H, 0.4)
    off = (~b.mask).nonzero()[:, 0]
    b.x[off] = float("nan")
    b.dw[off] = float("inf")
    b.din[off[::2]] = float("nan")
    b.din[off[1::2]] = -float("inf")
    b.idx[off] = -7
    x, y = a.run(), b.run()
    for name in x:
        assert torch.equal(x[name], y[name]), name
    a.check(x)
    assert not x["dx"][off.cuda()].any()


@pytest.mark.parametrize("T,E,H", [(30, 24, 256), (1100, 130, 4096)])
def test_all_masked(m, T, E, H):
    c = Case(m, T, E, 3, H)
    c.mask = torch.zeros(T, dtype=torch.bool)
    out = c.run()
    assert all(not v.any() for v in out.values())


def test_an_expert_named_twice(m):
    c = Case(m, 50, 40, 4, 256)
    c.idx[:, 2] = c.idx[:, 0]
    c.idx[::2, 3] = c.idx[::2, 0]
    c.check(c.run())


@pytest.mark.parametrize("bad", [-1, 40, 1 << 30])
def test_bad_expert(m, bad):
    c = Case(m, 50, 40, 4, 256)
    c.idx[20, 2] = bad
    out = c.run()
    assert torch.isnan(out["dlogits"][20]).all() and torch.isnan(out["dx"][20]).all() and torch.isnan(out["dWr"]).all()
    rest = [t for t in range(50) if t != 20]
    c.idx[20, 2] = 0
    want = c.want()
    for name in ("dlogits", "dx"):
        ref.close(out[name][rest], want[name][0][rest], want[name][1][rest], name)
    # without dw the experts are not looked at
    c.idx[20, 2] = bad
    c.check(c.run(dw=False), dw=False)


@pytest.mark.parametrize("T,H", [(30, 256), (700, 1024), (9000, 256), (9000, 2560)])
def test_accumulate(m, T, H):
    c = Case(m, T, 40, 4, H)
    g = torch.Generator().manual_seed(1)
    old = {"dx": torch.randn((T, H), generator=g), "dWr": torch.randn((40, H), generator=g)}
    want = c.want()
    for acc in (1, 2, 3):
        out = c.run(acc=acc, before=old)
        for bit, name in ((1, "dx"), (2, "dWr")):
            v, e = want[name]
            if acc & bit:
                v, e = v + old[name].double(), e + ref.EPS * (v.abs() + old[name].double().abs()) * 2
            ref.close(out[name], v, e, name)


@pytest.mark.parametrize("T,E,H", [(90, 60, 512), (1100, 513, 1024)])
def test_in_place_on_dlogits(m, T, E, H):
    c = Case(m, T, E, 4, H, 0.2)
    a, b = c.run(), c.run(inplace=True)
    for name in a:
        assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("T,E,H", [(90, 60, 512), (1100, 512, 1024)])
def test_logits_gradients_at_any_float(m, T, E, H):
    """dlogits_in and dlogits_out need no more than a float's alignment."""
    c = Case(m, T, E, 4, H, 0.2)
    want = c.run()
    wide = torch.full((2, T * E + 8), 7.0, device="cuda")
    wide[0, 1:1 + T * E] = c.dev[5].view(-1)
    args = list(c.args)
    for at in (1, 2):
        wide[1] = 7.0
        args[8], args[9] = wide[0, 1:], wide[1, at:]
        m.moe_route_backward(*args)
        assert torch.equal(wide[1, at:at + T * E].view(T, E), want["dlogits"])
        assert (wide[1, :at] == 7).all() and (wide[1, at + T * E:] == 7).all()
        assert torch.equal(args[10], want["dx"]) and torch.equal(args[11], want["dWr"])


def test_no_tokens(m):
    c = Case(m, 0, 40, 4, 256)
    out = c.run()
    assert not out["dWr"].any()
    old = torch.randn(40, 256)
    assert torch.equal(c.run(acc=2, before={"dWr": old})["dWr"].cpu(), old)


def test_against_autograd(m):
    """The gradient of sum(dw * w(logits)) + sum(din * logits) by torch's autograd in 64 bits."""
    c = Case(m, 60, 48, 5, 256)
    x, Wr = c.x.double().requires_grad_(), c.Wr.double().requires_grad_()
    logits = x @ Wr.t()
    logits.retain_grad()
    idx = torch.topk(logits, 5, dim=1).indices
    w = torch.softmax(logits.gather(1, idx), 1)
    ((w * c.dw.double()).sum() + (logits * c.din.double()).sum()).backward()
    c.idx, c.w = idx.to(torch.int32), w.detach().float()
    out, want = c.run(), c.want()
    for name, g in (("dlogits", logits.grad), ("dx", x.grad), ("dWr", Wr.grad)):
        # w is rounded to fp32 before the call: one EPS of it more in ds, through both products
        more = (4 * ref.EPS * g.abs() + 4 * ref.EPS * g.abs().max())
        ref.close(out[name], g, want[name][1] + more, name)


@pytest.mark.parametrize("T,H", [(150, 512), (700, 1024), (1500, 4096)])
@pytest.mark.parametrize("far", [30, 110])
def test_large_and_small_values(m, T, H, far):
    """Tokens, experts and columns of very unlike sizes keep their relative
    accuracy, each along the axis that a product does not sum over."""
    c = Case(m, T, 96, 5, H)
    g = torch.Generator().manual_seed(5)
    size = lambda *s: 2.0 ** torch.randint(-far, far // 2, s, generator=g)  # noqa: E731
    c.din *= size(T, 1)
    c.Wr *= 2.0 ** torch.randint(-10, 20, (1, H), generator=g)
    c.check(c.run(dw=False, dWr=False), dw=False)
    c = Case(m, T, 96, 5, H)
    c.din *= size(1, 96)
    c.x *= 2.0 ** torch.randint(-10, 20, (1, H), generator=g)
    c.check(c.run(dw=False, dx=False), dw=False)


@pytest.mark.parametrize("T,H", [(700, 1024), (1500, 4096)])
def test_zero_rows_and_columns(m, T, H):
    c = Case(m, T, 96, 5, H)
    c.din[3:200], c.din[:, 7], c.Wr[:, 100:300], c.Wr[9], c.x[:, 5] = 0.0, 0.0, 0.0, 0.0, 0.0
    c.check(c.run(dw=False), dw=False)


@pytest.mark.parametrize("T,H", [(40, 256), (700, 1024), (4100, 4096)])
def test_infinite_and_nan_values(m, T, H):
    c = Case(m, T, 33, 3, H)
    c.din[5, 3] = float("inf")
    c.din[9, 8] = float("nan")
    c.Wr[3, 17] = 0.0
    out, want = c.run(dw=False), c.want(dw=False)
    ok = [t for t in range(T) if t not in (5, 9)]
    ref.close(out["dx"][ok], want["dx"][0][ok], want["dx"][1][ok], "dx")
    assert not torch.isfinite(out["dx"][5]).any() and torch.isnan(out["dx"][9]).all()
    ok = [e for e in range(33) if e not in (3, 8)]
    ref.close(out["dWr"][ok], want["dWr"][0][ok], want["dWr"][1][ok], "dWr")
    assert not torch.isfinite(out["dWr"][3]).any() and torch.isnan(out["dWr"][8]).all()


@pytest.mark.parametrize("T,E,H", [(700, 130, 512), (1100, 513, 1024)])
def test_repeats_streams_and_graphs(m, T, E, H):
    a, b = Case(m, T, E, 6, H, 0.1), Case(m, 300, 256, 8, 256)
    want = []
    graphs = []
    ws = torch.zeros(max(m.moe_route_backward_workspace_bytes(m.desc(c.H, 64, c.E, c.k, "nvfp4"), c.T) for c in (a, b)),
                     dtype=torch.uint8, device="cuda")
    for c in (a, b):
        first = c.run()
        again = c.run(ws=ws)
        for name in first:
            assert torch.equal(first[name], again[name]), name
        c.out = again
        want.append(first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_route_backward(*c.args)
        graphs.append(g)
    for turn in range(3):
        for c in (a, b):
            for v in c.out.values():
                v.fill_(9)
        for g in (graphs if turn % 2 else graphs[::-1]):
            g.replay()
        torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        for c, w in zip((a, b), want):
            for k, v in c.out.items():
                assert torch.equal(v, w[k]), (turn, k)
        m.moe_route_backward(*a.args)
    s = torch.cuda.Stream()
    for v in a.out.values():
        v.fill_(9)
    torch.cuda.synchronize()
    m.moe_route_backward(*a.args, stream=s)
    s.synchronize()
    for k, v in a.out.items():
        assert torch.equal(v, want[0][k])


def test_long_batch_offsets_past_32_bits(m):
    """2^20 tokens of 2560: more than 2^31 elements of x and dx."""
    T, E, k, H = 1 << 20, 8, 2, 2560
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.empty((T, H), device=dev)
    for part in x.split(1 << 17):
        part.normal_(generator=g)
    Wr, din = torch.randn((E, H), device=dev, generator=g), torch.randn((T, E), device=dev, generator=g)
    d = m.desc(H, 64, E, k, "nvfp4")
    dx, dWr = torch.empty((T, H), device=dev), torch.empty((E, H), device=dev)
    ws = torch.empty(m.moe_route_backward_workspace_bytes(d, T), dtype=torch.uint8, device=dev)
    m.moe_route_backward(d, x, T, Wr, None, None, None, None, din, None, dx, dWr, 0, ws)
    torch.cuda.synchronize()
    t = torch.cat([torch.arange(8), torch.randint(0, T, (200,), generator=torch.Generator().manual_seed(1)), torch.arange(T - 8, T)])
    G = din.cpu().double()
    ref.close(dx[t.to(dev)], *ref.mm(G[t], ref.cpu64(Wr), pairs=True), "dx")
    # some columns of dWr over all tokens
    c = torch.tensor([0, 1, 777, 1280, 2559])
    ref.close(dWr[:, c.to(dev)], *ref.mm(G.t().contiguous(), x[:, c.to(dev)].cpu().double(), pairs=True), "dWr")


@pytest.mark.parametrize("T,E,H", [(91, 64, 512), (1101, 512, 1024), (1023, 520, 1280), (8191, 32, 2560)])
@pytest.mark.parametrize("dw", [True, False])
def test_in_place_on_whole_vectors(m, T, E, H, dw):
    """dlogits_out is dlogits_in where rows are loaded and written 16 bytes at a time, in batches of odd length."""
    c = Case(m, T, E, 4, H, 0.2)
    a, b = c.run(dw=dw), c.run(dw=dw, inplace=True)
    for name in a:
        assert torch.equal(a[name], b[name]), name
    c.check(b, dw=dw)


@pytest.mark.parametrize("T,E,H", [(3000, 1, 8192), (2047, 3, 8192), (5000, 9, 256), (1500, 2, 2560)])
def test_parts_of_long_sums_are_bounded(m, T, E, H):
    """Below 2^29 multiplications dWr is summed over parts of at most 1024
    tokens. Beside 2^26 a 1, or a few ones added together, is half a step at
    most and lost, so of T - 1 ones no more than those of the first token's own
    part may be missing (and one step where the parts are added)."""
    c = Case(m, T, E, 1, H)
    c.din.fill_(1.0)
    c.x.fill_(1.0)
    c.x[0] = 2.0 ** 26
    out = c.run(dw=False, dx=False)["dWr"].double().cpu()
    assert (out <= 2.0 ** 26 + T + 8).all() and (out >= 2.0 ** 26 + T - 1 - 1024 - 8).all(), (out.min() - 2.0 ** 26).item()


@pytest.mark.parametrize("T,E,H", [(8191, 8, 4096), (8191, 33, 2560), (2100, 64, 4096), (16500, 64, 768)])
def test_few_experts_multiply_in_fp32(m, T, E, H):
    """Up to 64 experts, batches of any length have fp32 products: operands
    2^30 apart within a row, whose products are alike, keep fp32's accuracy."""
    c = Case(m, T, E, min(E, 4), H, 0.1)
    for s in range(2):
        c.din = torch.randn(T, E, generator=torch.Generator().manual_seed(T + s))
        if s == 0:  # along the experts
            c.din[:, 1:] *= 2.0 ** -30
            c.Wr[0] *= 2.0 ** -30
        else:       # along the tokens
            c.din[2:] *= 2.0 ** -30
            c.x[:2] *= 2.0 ** -30
        out = c.run(dw=False)
        G = c.din.double() * c.mask[:, None]
        if s == 0:
            ref.close(out["dx"], *ref.mm(G, c.Wr.double()), "dx")
        else:
            ref.close(out["dWr"], *ref.mm(G.t().contiguous(), c.x.double()), "dWr")


@pytest.mark.parametrize("T,E,H", [(3000, 72, 2560), (9000, 65, 1024)])
@pytest.mark.parametrize("acc", [1, 2, 3])
def test_accumulate_in_pairs(m, T, E, H, acc):
    c = Case(m, T, E, 4, H)
    g = torch.Generator().manual_seed(1)
    old = {"dx": torch.randn((T, H), generator=g), "dWr": torch.randn((E, H), generator=g)}
    want, out = c.want(), c.run(acc=acc, before=old)
    for bit, name in ((1, "dx"), (2, "dWr")):
        v, e = want[name]
        if acc & bit:
            v, e = v + old[name].double(), e + ref.EPS * (v.abs() + old[name].double().abs()) * 2
        ref.close(out[name], v, e, name)


def test_infinite_and_nan_values_in_pairs(m):
    c = Case(m, 4100, 72, 3, 2560)
    c.din[5, 3], c.din[9, 8], c.Wr[3, 17] = float("inf"), float("nan"), 0.0
    out, want = c.run(dw=False), c.want(dw=False)
    ok = [t for t in range(4100) if t not in (5, 9)]
    ref.close(out["dx"][ok], want["dx"][0][ok], want["dx"][1][ok], "dx")
    assert not torch.isfinite(out["dx"][5]).any() and torch.isnan(out["dx"][9]).all()
    ok = [e for e in range(72) if e not in (3, 8)]
    ref.close(out["dWr"][ok], want["dWr"][0][ok], want["dWr"][1][ok], "dWr")
    assert not torch.isfinite(out["dWr"][3]).any() and torch.isnan(out["dWr"][8]).all()


def test_long_batch_of_pairs_past_32_bits(m):
    """2^20 tokens of 2304 with 72 experts: more than 2^31 elements of x, dx and the pairs."""
    T, E, H, dev = 1 << 20, 72, 2304, "cuda"
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.empty((T, H), device=dev)
    for part in x.split(1 << 17):
        part.normal_(generator=g)
    Wr, din = torch.randn((E, H), device=dev, generator=g), torch.randn((T, E), device=dev, generator=g)
    d = m.desc(H, 64, E, 2, "nvfp4")
    dx, dWr = torch.empty((T, H), device=dev), torch.empty((E, H), device=dev)
    ws = torch.empty(m.moe_route_backward_workspace_bytes(d, T), dtype=torch.uint8, device=dev)
    m.moe_route_backward(d, x, T, Wr, None, None, None, None, din, None, dx, dWr, 0, ws)
    torch.cuda.synchronize()
    t = torch.cat([torch.arange(8), torch.randint(0, T, (200,), generator=torch.Generator().manual_seed(1)), torch.arange(T - 8, T)])
    G = din.cpu().double()
    ref.close(dx[t.to(dev)], *ref.mm(G[t], ref.cpu64(Wr), pairs=True), "dx")
    c = torch.tensor([0, 1, 777, 1280, H - 1])
    ref.close(dWr[:, c.to(dev)], *ref.mm(G.t().contiguous(), x[:, c.to(dev)].cpu().double(), pairs=True), "dWr")


@pytest.mark.parametrize("T,E,H", [(1100, 512, 1024), (4100, 130, 1280), (2451, 384, 4096)])
def test_fp32_products_on_request(m, T, E, H):
    """Operands 2^30 apart within a row, whose products are alike: pairs keep
    2^-39 of the row's largest, fp32 products all of it."""
    for along in range(2):
        c = Case(m, T, E, 4, H, 0.1)
        c.din = torch.randn(T, E, generator=torch.Generator().manual_seed(T + along))
        if along == 0:
            c.din[:, 1:] *= 2.0 ** -30
            c.Wr[0] *= 2.0 ** -30
        else:
            c.din[2:] *= 2.0 ** -30
            c.x[:2] *= 2.0 ** -30
        G = c.din.double() * c.mask[:, None]
        want = ref.mm(G, c.Wr.double()) if along == 0 else ref.mm(G.t().contiguous(), c.x.double())
        name = "dWr" if along else "dx"
        ref.close(c.run(dw=False, acc=m.MOE_FP32_PRODUCTS)[name], *want, name)
        if along == 0:  # (over the tokens each part of the sum has its own power of two)
            d = (c.run(dw=False)[name].cpu().double() - want[0]).abs()
            assert (d > want[1]).any()  # the sizes do tell the forms apart


def test_fp32_products_with_all_else(m):
    c = Case(m, 1101, 512, 6, 1024, 0.2)
    g = torch.Generator().manual_seed(1)
    old = {"dx": torch.randn((1101, 1024), generator=g), "dWr": torch.randn((512, 1024), generator=g)}
    G, eG = c.want()["dlogits"]
    x = c.x.double() * c.mask[:, None]
    want = {"dx": ref.mm(G, c.Wr.double(), ea=eG), "dWr": ref.mm(G.t().contiguous(), x, ea=eG.t().contiguous())}
    for acc in range(4):
        out = c.run(acc=acc + m.MOE_FP32_PRODUCTS, before=old, inplace=acc == 1)
        for bit, name in ((1, "dx"), (2, "dWr")):
            v, e = want[name]
            if acc & bit:
                v, e = v + old[name].double(), e + ref.EPS * (v.abs() + old[name].double().abs()) * 2
            ref.close(out[name], v, e, name)
        ref.close(out["dlogits"], G, eG, "dlogits")
    few = Case(m, 90, 60, 4, 512)
    a, b = few.run(), few.run(acc=m.MOE_FP32_PRODUCTS)
    assert all(torch.equal(a[k], b[k]) for k in a)
