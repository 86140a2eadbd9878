"""Low-rank adapters on the GPU, forward and backward, against their formulas
in 64 bits (tests/learn_ref.py) and against differences, over types, ranks,
orders of tokens and strides; bad ids and ranks; untrained adapters;
accumulation; no tokens; streams and graphs."""
import pytest
import torch

import learn_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import block_scaled_fp4_route_amd as m
    return m


def ptrs(ts):
    return torch.tensor([0 if t is None else t.data_ptr() for t in ts], dtype=torch.int64, device="cuda")


def strided(t, pad):
    """The same rows with `pad` elements of junk behind each."""
    if t is None or not pad:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + pad), 3.0, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide


class Case:
    def __init__(self, m, dt, T, K, N, ranks, order="mixed", R=None, seed=0):
        g = torch.Generator().manual_seed(31 * T + K + N + len(ranks) + seed)
        self.m, self.T, self.K, self.N, self.n, self.dt = m, T, K, N, len(ranks), DT[dt]
        self.R = R or max(max(ranks), 1)
        wt = torch.float16 if dt == "f16" else torch.bfloat16
        rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.A = [(rnd(r, K) * K ** -0.5).to(wt).cuda() for r in ranks]
        self.B = [(rnd(r, N) * 0.1).to(wt).cuda() for r in ranks]
        self.ranks = torch.tensor(ranks, dtype=torch.int32).cuda()
        self.scales = torch.tensor([0.5 + 0.25 * a for a in range(self.n)]).cuda()
        if order == "mixed":
            ids = torch.randint(-1, self.n, (T,), generator=g)
        elif order == "runs":
            ids = torch.sort(torch.randint(-1, self.n, (T,), generator=g)).values.flip(0)
        else:  # one adapter for all
            ids = torch.zeros(T, dtype=torch.int64)
        self.ids = ids.to(torch.int32).cuda()
        self.x, self.dy = rnd(T, K).to(self.dt).cuda(), rnd(T, N).to(self.dt).cuda()
        self.base, self.dxb = rnd(T, N).to(self.dt).cuda(), rnd(T, K).to(self.dt).cuda()
        self.l = m.lora_desc(K, N, self.n, self.R, self.dt)
        self.tabs = None

    def table(self):
        if self.tabs is None:
            self.tabs = (ptrs(self.A), ptrs(self.B))
        return (self.ids, *self.tabs, self.ranks, self.scales)

    def ws(self, back):
        return torch.full((self.m.moe_lora_workspace_bytes(self.l, self.T, back),), 0xA5, dtype=torch.uint8, device="cuda")

    def apply(self, base="own", inplace=False, pads=(0, 0, 0), stream=None, ws=None):
        T, K, N = self.T, self.K, self.N
        x, b = strided(self.x, pads[0]), None if base is None else strided(self.base.clone(), pads[1])
        y = b if inplace else torch.full((T, N + pads[2]), 7.0, dtype=self.dt, device="cuda")
        self.args = (self.l, x, K + pads[0], T, *self.table(), b, N + pads[1], y, y.shape[1] if T else N,
                     self.ws(False) if ws is None else ws)
        torch.cuda.synchronize()
        self.m.moe_lora_apply(*self.args, stream=stream)
        torch.cuda.synchronize()
        if y.shape[1] > N:
            junk = 3.0 if inplace else 7.0
            assert (y[:, N:] == junk).all()  # nothing behind the rows is written
        return y[:, :N]

    def want(self, base="own"):
        return ref.lora(self.x, self.ids, self.A, self.B, self.scales, None if base is None else self.base, self.dt, self.n)

    def backward(self, dx=True, base=True, grads=True, acc=0, old=None, skip=(), pads=(0, 0, 0), inplace=False, ws=None):
        T, K, N = self.T, self.K, self.N
        x, dy = strided(self.x, pads[0]), strided(self.dy, pads[1])
        b = strided(self.dxb.clone(), pads[2]) if base else None
        o = b if inplace else torch.full((T, K + pads[2]), 7.0, dtype=self.dt, device="cuda")
        self.dA = [torch.full(a.shape, 7.0, device="cuda") if old is None else old[0][i].clone() for i, a in enumerate(self.A)]
        self.dB = [torch.full(a.shape, 7.0, device="cuda") if old is None else old[1][i].clone() for i, a in enumerate(self.B)]
        self.gp = (ptrs([None if ("A", i) in skip else t for i, t in enumerate(self.dA)]),
                   ptrs([None if ("B", i) in skip else t for i, t in enumerate(self.dB)]))
        self.args = (self.l, x, K + pads[0], dy, N + pads[1], T, *self.table(), b, K + pads[2], o if dx else None, K + pads[2],
                     *(self.gp if grads else (None, None)), acc, self.ws(True) if ws is None else ws)
        torch.cuda.synchronize()
        self.m.moe_lora_backward(*self.args)
        torch.cuda.synchronize()
        return o[:, :K] if dx else None

    def check_backward(self, dx, base=True):
        if dx is not None:
            v = ref.lora(self.dy, self.ids, self.B, self.A, self.scales, self.dxb if base else None, self.dt, self.n)
            ref.close(dx, *v, "dx")
        for a, (wa, wb) in enumerate(ref.lora_grads(self.x, self.dy, self.ids, self.A, self.B, self.scales, self.n)):
            ref.close(self.dA[a], *wa, ("dA", a))
            ref.close(self.dB[a], *wb, ("dB", a))


SHAPES = [(1, 8, 8, [1], "one"), (1, 2560, 8192, [16, 8], "one"), (2, 16, 2560, [3, 1, 0], "mixed"),
          (17, 264, 40, [5, 16, 7], "mixed"), (64, 2560, 640, [16] * 8, "mixed"), (65, 2560, 640, [16] * 8, "mixed"),
          (65, 8, 8, [128], "one"), (130, 520, 1032, [33, 64, 1, 17], "mixed"), (300, 640, 2560, [8, 3], "runs"),
          (257, 1000, 264, [128, 100], "mixed"), (700, 256, 512, [20, 31, 48], "runs"), (1500, 136, 24, [2] * 40, "mixed"),
          (512, 72, 520, [16, 9], "mixed"), (513, 72, 520, [16, 9], "mixed"), (64, 72, 520, [128, 1, 40], "mixed"), (8, 4096, 2560, [16], "one"),
          (40, 8192, 256, [32, 8, 31], "mixed")]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,N,ranks,order", SHAPES)
def test_apply(m, dt, T, K, N, ranks, order):
    c = Case(m, dt, T, K, N, ranks, order)
    ref.close(c.apply(), *c.want(), "y")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,N,ranks,order", SHAPES)
def test_backward(m, dt, T, K, N, ranks, order):
    c = Case(m, dt, T, K, N, ranks, order)
    c.check_backward(c.backward())


@pytest.mark.parametrize("T", [5, 200, 600])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_bases_places_and_strides(m, dt, T):
    c = Case(m, dt, T, 264, 520, [16, 5, 9])
    y = c.apply()
    assert torch.equal(y, c.apply(inplace=True))
    assert torch.equal(y, c.apply(pads=(8, 16, 24)))
    assert torch.equal(y, c.apply(pads=(24, 8, 8), inplace=True))
    ref.close(c.apply(base=None), *c.want(base=None), "y")
    rows = c.ids < 0
    assert torch.equal(y[rows], c.base[rows]) and rows.any()
    dx = c.backward()
    first = [t.clone() for t in c.dA + c.dB]
    for kw in ({"inplace": True}, {"pads": (8, 16, 24)}, {"pads": (16, 8, 8), "inplace": True}):
        assert torch.equal(dx, c.backward(**kw))
        assert all(torch.equal(a, b) for a, b in zip(first, c.dA + c.dB))
    c.check_backward(c.backward(base=False), base=False)
    assert c.backward(dx=False) is None
    assert all(torch.equal(a, b) for a, b in zip(first, c.dA + c.dB))
    assert torch.equal(dx, c.backward(grads=False))


@pytest.mark.parametrize("T", [40, 400])
def test_max_rank_above_the_ranks(m, T):
    """The tables' largest rank only sizes the workspace; results agree with the tight one to the bound."""
    for R in (16, 30, 40, 128):
        c = Case(m, "bf16", T, 264, 520, [16, 5, 9], R=R)
        ref.close(c.apply(), *c.want(), "y")
        c.check_backward(c.backward())


@pytest.mark.parametrize("T", [6, 90, 600])
def test_no_adapter_at_all(m, T):
    c = Case(m, "bf16", T, 264, 520, [16, 5])
    c.ids.fill_(-3)
    c.x.fill_(float("nan"))  # rows without an adapter are not read
    assert torch.equal(c.apply(), c.base) and torch.equal(c.apply(inplace=True), c.base)
    assert not c.apply(base=None).any()
    dx = c.backward()
    assert torch.equal(dx, c.dxb) and all(not t.any() for t in c.dA + c.dB)


@pytest.mark.parametrize("T", [8, 150, 700])
def test_bad_ids(m, T):
    c = Case(m, "f32", T, 64, 72, [4, 4])
    c.ids[3], c.ids[T - 1] = 2, 1 << 30
    ref.close(c.apply(), *c.want(), "y")
    assert torch.isnan(c.apply()[3]).all()
    c.check_backward(c.backward())


@pytest.mark.parametrize("T", [8, 150, 700])
@pytest.mark.parametrize("bad", [-1, 17, 1 << 30])
def test_bad_rank(m, T, bad):
    c = Case(m, "f32", T, 64, 72, [16, 4, 16])
    c.ids[:4] = 1
    y, v = c.apply(), c.want()
    dx = c.backward()
    good = [t.clone() for t in c.dA + c.dB]
    c.ranks[1] = bad
    y2, rows = c.apply(), c.ids == 1
    assert torch.isnan(y2[rows]).all() and torch.equal(y2[~rows], y[~rows])
    dx2 = c.backward()
    assert torch.isnan(dx2[rows]).all() and torch.equal(dx2[~rows], dx[~rows])
    for i, (a, b) in enumerate(zip(good, c.dA + c.dB)):
        assert (b == 7.0).all() if i % 3 == 1 else torch.equal(a, b)
    ref.close(y, *v, "y")


@pytest.mark.parametrize("T,R", [(8, 16), (8, 128), (150, 16), (700, 16)])
@pytest.mark.parametrize("side", [0, 1])
def test_null_factors(m, T, R, side):
    """As a rank that is not usable; not looked at beside a rank of 0 or without tokens."""
    c = Case(m, "bf16", T, 264, 1032, [16, 4, 0, 7], R=R)
    c.ids[c.ids == 3] = 2
    c.ids[:4] = torch.tensor([1, 0, 2, 1], device="cuda")
    y, dx = c.apply(), c.backward()
    good = [t.clone() for t in c.dA + c.dB]
    rows = c.ids == 1
    c.tabs = tuple(ptrs([None if i in (2, 3) or (i == 1 and s == side) else f for i, f in enumerate(t)])
                   for s, t in enumerate((c.A, c.B)))
    y2, dx2 = c.apply(), c.backward()
    assert torch.isnan(y2[rows]).all() and torch.equal(y2[~rows], y[~rows])
    assert torch.isnan(dx2[rows]).all() and torch.equal(dx2[~rows], dx[~rows])
    for i, (a, b) in enumerate(zip(good, c.dA + c.dB)):
        assert (b == 7.0).all() if i % 4 == 1 else torch.equal(a, b)


@pytest.mark.parametrize("T", [20, 900])
def test_accumulate_and_untrained(m, T):
    c = Case(m, "bf16", T, 264, 136, [8, 3, 5, 2])
    c.ids[c.ids == 3] = 0  # adapter 3 has no token
    c.check_backward(c.backward())
    assert not c.dA[3].any() and not c.dB[3].any()
    g = torch.Generator().manual_seed(2)
    old = ([torch.randn(a.shape, generator=g).cuda() for a in c.A], [torch.randn(b.shape, generator=g).cuda() for b in c.B])
    c.backward(acc=1, old=old, skip={("A", 1), ("B", 2)})
    want = ref.lora_grads(c.x, c.dy, c.ids, c.A, c.B, c.scales, c.n)
    for a in range(4):
        for name, got, o, (v, e) in (("A", c.dA[a], old[0][a], want[a][0]), ("B", c.dB[a], old[1][a], want[a][1])):
            if (name, a) in {("A", 1), ("B", 2)}:
                assert torch.equal(got, o)
            else:
                ref.close(got, v + o.cpu().double(), e + 2 * ref.EPS * (v.abs() + o.cpu().double().abs()), (name, a))
    assert torch.equal(c.dA[3], old[0][3])


def test_one_side_only(m):
    c = Case(m, "f16", 100, 64, 72, [4, 8])
    c.backward()
    dA, dB = [t.clone() for t in c.dA], [t.clone() for t in c.dB]
    args = list(c.args)
    for t in c.dA + c.dB:
        t.fill_(7.0)
    m.moe_lora_backward(*args[:15], c.gp[0], None, 0, args[-1])
    assert all(torch.equal(a, b) for a, b in zip(dA, c.dA)) and all((t == 7).all() for t in c.dB)
    m.moe_lora_backward(*args[:15], None, c.gp[1], 0, args[-1])
    assert all(torch.equal(a, b) for a, b in zip(dB, c.dB))


def test_no_tokens(m):
    c = Case(m, "bf16", 0, 64, 72, [4, 8])
    c.apply()
    c.backward()
    assert all(not t.any() for t in c.dA + c.dB)
    old = ([torch.ones_like(t) for t in c.dA], [torch.ones_like(t) for t in c.dB])
    c.backward(acc=1, old=old)
    assert all((t == 1).all() for t in c.dA + c.dB)


def test_infinite_activations(m):
    """An infinity reaches its own row as fp32 arithmetic has it, and no other row."""
    for dt in DT:
        for T in (9, 100, 600):
            c = Case(m, dt, T, 64, 72, [4], "one")
            y = c.apply()
            c.x[2, 5], c.x[4, 9] = float("inf"), float("nan")
            z = c.apply()
            rest = [t for t in range(T) if t not in (2, 4)]
            assert torch.equal(y[rest], z[rest])
            assert not torch.isfinite(z[2]).any() and torch.isnan(z[4]).all()


def test_fp32_activations_keep_all_bits(m):
    """x = 1 + 2^-23 against a factor row that cancels the ones: what is left
    is the last bit, which a rounded activation would lose."""
    for T in (3, 70, 600):
        c = Case(m, "f32", T, 16, 8, [1], "one")
        c.x[:] = 1.0 + 2.0 ** -23
        c.x[:, 8:] = 1.0
        c.A[0][0, :8], c.A[0][0, 8:] = 1.0, -1.0
        c.B[0][:] = 1.0
        c.scales[:] = 1.0
        y = c.apply(base=None)
        assert (y == 8 * 2.0 ** -23).all()


def test_strides_past_32_bits(m):
    """Rows 2^31 and more elements apart."""
    c = Case(m, "bf16", 3, 64, 72, [4], "one")
    y, dx = c.apply(), None
    ld = (1 << 30) + 64
    wide = torch.empty(2 * ld + 128, dtype=torch.bfloat16, device="cuda")
    xw = wide.as_strided((3, 64), (ld, 1))
    xw.copy_(c.x)
    out = torch.empty(2 * ld + 128, dtype=torch.bfloat16, device="cuda")
    m.moe_lora_apply(c.l, wide, ld, 3, *c.table(), c.base, 72, out, ld, c.ws(False))
    assert torch.equal(out.as_strided((3, 72), (ld, 1)), y)
    dx = c.backward()
    m.moe_lora_backward(c.l, wide, ld, c.dy, 72, 3, *c.table(), c.dxb, 64, out, ld, None, None, 0, c.ws(True))
    assert torch.equal(out.as_strided((3, 64), (ld, 1)), dx)
    # and through the grouped kernels
    T = 70
    c = Case(m, "bf16", T, 64, 72, [128], "one")
    y = c.apply()
    ld = (1 << 31) // 64 + 64
    wide = torch.empty((T - 1) * ld + 128, dtype=torch.bfloat16, device="cuda")
    wide.as_strided((T, 64), (ld, 1)).copy_(c.x)
    out = torch.empty((T - 1) * ld + 128, dtype=torch.bfloat16, device="cuda")
    m.moe_lora_apply(c.l, wide, ld, T, *c.table(), c.base, 72, out, ld, c.ws(False))
    assert torch.equal(out.as_strided((T, 72), (ld, 1)), y)
    dx = c.backward()
    old = [t.clone() for t in c.dA + c.dB]
    m.moe_lora_backward(c.l, wide, ld, c.dy, 72, T, *c.table(), c.dxb, 64, out, ld, *c.gp, 0, c.ws(True))
    assert torch.equal(out.as_strided((T, 64), (ld, 1)), dx)
    assert all(torch.equal(a, b) for a, b in zip(old, c.dA + c.dB))
    wide.as_strided((T, 72), (ld, 1)).copy_(c.dy)
    m.moe_lora_backward(c.l, c.x, 64, wide, ld, T, *c.table(), c.dxb, 64, out, ld, *c.gp, 0, c.ws(True))
    assert torch.equal(out.as_strided((T, 64), (ld, 1)), dx)
    assert all(torch.equal(a, b) for a, b in zip(old, c.dA + c.dB))


def test_a_workspace_for_the_longest_batch(m):
    ws = None
    for T in (3000, 700, 65, 64, 3):
        c = Case(m, "bf16", T, 264, 520, [16, 64, 3], R=64)
        y, dx = c.apply(), c.backward()
        grads = c.dA + c.dB
        ws = c.ws(True) if ws is None else ws
        assert torch.equal(y, c.apply(ws=ws)) and torch.equal(dx, c.backward(ws=ws))
        assert all(torch.equal(a, b) for a, b in zip(grads, c.dA + c.dB))


def test_gradients_against_differences(m):
    """y is linear in each factor, so the difference of the framework's own
    fp32 forward over a step h of one element is exact up to its rounding:
    off by at most sum|dy| times y's bound over h, beside the gradient's own bound."""
    c = Case(m, "f32", 70, 24, 16, [3, 2])
    c.backward(dx=False)
    dA, dB = [t.clone() for t in c.dA], [t.clone() for t in c.dB]
    h = 0.5
    bounds = ref.lora_grads(c.x, c.dy, c.ids, c.A, c.B, c.scales, c.n)
    for side, (facs, grads) in enumerate(((c.A, dA), (c.B, dB))):
        for a in range(2):
            for (i, j) in ((0, 0), (1, 7), (facs[a].shape[0] - 1, 15)):
                old = facs[a][i, j].item()
                ys, steps, off = [], [], 0.0
                for sign in (1, -1):
                    facs[a][i, j] = old + sign * h  # rounded to bf16; the step taken is what counts
                    steps.append(facs[a][i, j].item())
                    ys.append((c.apply().double() * c.dy.double()).sum().item())
                    off += (c.want()[1] * c.dy.cpu().double().abs()).sum().item()
                facs[a][i, j] = old
                diff = (ys[0] - ys[1]) / (steps[0] - steps[1])
                assert abs(diff - grads[a][i, j].item()) \
                    <= off / abs(steps[0] - steps[1]) + bounds[a][side][1][i, j].item()


def test_repeats_streams_and_graphs(m):
    cases = [Case(m, "bf16", 300, 264, 520, [16, 5, 9]), Case(m, "f16", 40, 520, 264, [8, 30]), Case(m, "f32", 90, 64, 72, [128])]
    need = max(m.moe_lora_workspace_bytes(c.l, c.T, True) for c in cases)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    runs = []
    for c in cases:
        want = c.apply(), c.backward(), [t.clone() for t in c.dA + c.dB]
        y = c.apply(ws=ws)
        fwd = c.args
        dx = c.backward(ws=ws)
        bwd = c.args
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_lora_apply(*fwd)
            m.moe_lora_backward(*bwd)
        runs.append((c, y, dx, list(c.dA + c.dB), want, g, fwd, bwd))
    for turn in range(3):
        for c, y, dx, gr, want, g, fwd, bwd in runs:
            for t in (y, dx, *gr):
                t.fill_(9)
        for r in (runs if turn % 2 else runs[::-1]):
            r[5].replay()
        torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        for c, y, dx, gr, want, g, fwd, bwd in runs:
            assert torch.equal(y, want[0]) and torch.equal(dx, want[1]) and all(torch.equal(a, b) for a, b in zip(gr, want[2]))
        m.moe_lora_apply(*runs[0][6])
    # two at once, each with its own workspace, on streams of their own
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = runs[0], runs[1]
    for r in (a, b):
        r[1].fill_(9)
    wa, wb = a[0].ws(False), b[0].ws(False)
    torch.cuda.synchronize()
    m.moe_lora_apply(*a[6][:-1], wa, stream=sa)
    m.moe_lora_apply(*b[6][:-1], wb, stream=sb)
    torch.cuda.synchronize()
    assert torch.equal(a[1], a[4][0]) and torch.equal(b[1], b[4][0])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,R,K,N", [(9, 1, 64, 72), (9, 1, 2560, 8192), (70, 128, 64, 72), (600, 17, 264, 520), (600, 64, 1032, 72),
                                     (9000, 33, 64, 72)])
def test_infinities_keep_their_class(m, dt, T, R, K, N):
    """Infinite activations and factors beside values of few bits: an infinite
    product stays infinite, with its sign, and only 0 times an infinity or
    opposite infinities make a NaN, whatever the batch and the rank that
    choose the kernels. The formula in 64 bits says which."""
    c = Case(m, dt, T, K, N, [1, 1, 1], "mixed", R=R)
    inf, nan = float("inf"), float("nan")
    few = torch.tensor([1.0, -0.5, 1.0 + 2.0 ** -7, -3.0, 0.0, 2.0 ** -3, 1.0 + 2.0 ** -10, 0.40625])  # and one of 11 bits
    for t in (c.x, c.dy, *c.A, *c.B):
        t.copy_(few[torch.arange(t.numel()) * 5 % 8].view(t.shape))
    c.scales[:] = torch.tensor([1.0, -2.0, 0.0])
    c.ids[:8] = torch.tensor([0, 0, 1, 1, 2, -1, 0, 1], device="cuda")
    c.x[0, 0], c.x[1, 3], c.x[2, K - 1], c.x[4, 8], c.x[6, 9] = inf, -inf, inf, inf, nan
    c.dy[3, 5], c.dy[7, N - 1], c.dy[6, 2] = inf, -inf, nan
    c.A[1][0, 7], c.B[0][0, 3], c.B[0][0, 8], c.B[1][0, N - 2], c.B[1][0, 10] = inf, inf, -inf, -inf, nan
    y, want = c.apply(), c.want()
    assert torch.isinf(want[0]).any() and torch.isnan(want[0]).any() and torch.isfinite(want[0]).any()
    ref.close(y, *want, "y")
    c.check_backward(c.backward())
    # and where nothing but the activations is infinite
    c = Case(m, dt, T, K, N, [1, 1], "mixed", R=R)
    for t in (c.x, c.dy, *c.A, *c.B):
        t.copy_(few[torch.arange(t.numel()) * 5 % 8].view(t.shape))
    c.ids[:4] = torch.tensor([0, 1, 0, 1], device="cuda")
    c.x[0, 1], c.x[1, 2], c.dy[2, 3], c.dy[3, 1] = inf, -inf, inf, -inf
    ref.close(c.apply(), *c.want(), "y")
    c.check_backward(c.backward())


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,N,ranks,order", [
    (8193, 64, 72, [5, 16, 1], "mixed"), (16500, 64, 72, [17, 3], "mixed"),  # ids in more than one span of 8192
    (13500, 264, 520, [16, 9, 33], "runs"),  # pieces of three tiles, several an adapter, the last ones ragged
    (9000, 1032, 2056, [64, 7], "mixed"),    # pieces of four tiles
    (1 << 20, 8, 16, [3, 1], "mixed")])      # the longest batch: pieces of 64 tiles
def test_long_batches(m, dt, T, K, N, ranks, order):
    c = Case(m, dt, T, K, N, ranks, order)
    ref.close(c.apply(), *c.want(), "y")
    c.check_backward(c.backward())


@pytest.mark.parametrize("T,dt", [(1, "bf16"), (300, "f16"), (3000, "f32"), (3000, "bf16")])
def test_as_many_adapters_as_the_tables_hold(m, T, dt):
    c = Case(m, dt, T, 64, 72, [a % 4 for a in range(1024)], "mixed")
    ref.close(c.apply(), *c.want(), "y")
    c.check_backward(c.backward())


@pytest.mark.parametrize("T,K,N,r", [(40, 2560, 640, 16), (600, 64, 2560, 16), (600, 2560, 64, 64), (2500, 264, 520, 128), (4000, 520, 264, 17)])
def test_norm_of_the_error(m, T, K, N, r):
    """Beside the elementwise worst case: over random values the roundings of a
    sum of L products add up like a random walk. The i-th partial sum is about
    sqrt(i / L) of the root S of the sum of squared products, and one rounding
    has a variance of EPS^2 / 3 of its square, so the error is about
    sqrt(L / 6) EPS S. A product of parts has up to eight terms, sqrt(8) at
    most; four times the walk is allowed. Leaving out the third part of an
    operand, 2^-16.4 of it by the root mean square, is more at every size here."""
    c = Case(m, "f32", T, K, N, [r], "one")
    walk = lambda L, a, b: (L / 6) ** 0.5 * ref.EPS * torch.sqrt((a ** 2) @ (b ** 2))  # noqa: E731
    thru = lambda e, b: torch.sqrt((e ** 2) @ (b ** 2))  # noqa: E731
    x, dy, A, B, s = c.x.cpu().double(), c.dy.cpu().double(), c.A[0].cpu().double(), c.B[0].cpu().double(), float(c.scales[0])
    u, v = s * (x @ A.t()), s * (dy @ B.t())
    eu, ev = walk(K, s * x, A.t()), walk(N, s * dy, B.t())
    out = {"y": c.apply(base=None), "dx": c.backward(base=False), "dA": c.dA[0], "dB": c.dB[0]}
    want = {"y": (u @ B, walk(r, u, B) + thru(eu, B)), "dx": (v @ A, walk(r, v, A) + thru(ev, A)),
            "dA": (v.t() @ x, walk(T, v.t(), x) + thru(ev.t(), x)), "dB": (u.t() @ dy, walk(T, u.t(), dy) + thru(eu.t(), dy))}
    for name, (value, walked) in want.items():
        off = (out[name].cpu().double() - value).norm() / (4 * walked.norm())
        assert off <= 1, (name, off)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [60, 900])
def test_infinities_beside_old_values(m, dt, T):
    """In place on the base, and added to gradients that are there: what is
    beside an infinity keeps its value, and an infinity meets what it is added to."""
    inf, nan = float("inf"), float("nan")
    c = Case(m, dt, T, 72, 136, [2, 3], "mixed", R=40)
    c.A[0][0], c.A[0][1] = 1.0, 0.0
    c.ids[:6] = torch.tensor([0, 0, 1, 0, -1, 0], device="cuda")
    c.x[1, 5], c.dy[3, 7], c.x[4] = inf, -inf, nan
    c.base[1, 3], c.base[1, 4], c.base[1, 6] = nan, inf, -inf
    c.dxb[3, 3], c.dxb[3, 4], c.dxb[3, 6] = nan, inf, -inf
    y = c.apply()
    ref.close(y, *c.want(), "y")
    ok = torch.isfinite(y)
    assert torch.equal(torch.where(ok, y, 0), torch.where(ok, c.apply(inplace=True), 0)) and ok.any() and not ok.all()
    ref.close(c.apply(inplace=True), *c.want(), "y in place")
    c.check_backward(c.backward(inplace=True))
    g = torch.Generator().manual_seed(2)
    old = ([torch.randn(a.shape, generator=g).cuda() for a in c.A], [torch.randn(b.shape, generator=g).cuda() for b in c.B])
    old[0][0][0, 5], old[0][0][1, 5], old[1][0][0, 7], old[1][0][0, 8] = inf, -inf, nan, inf
    c.backward(acc=1, old=old)
    want = ref.lora_grads(c.x, c.dy, c.ids, c.A, c.B, c.scales, c.n)
    for a in range(2):
        for name, got, o, (v, e) in (("A", c.dA[a], old[0][a], want[a][0]), ("B", c.dB[a], old[1][a], want[a][1])):
            o = o.cpu().double()
            ref.close(got, v + o, e + 2 * ref.EPS * (v.abs() + o.abs()), (name, a))


@pytest.mark.parametrize("T", [9, 600])
def test_nan_of_any_bits(m, T):
    """A NaN whose bits are all in the low half of an fp32 value is one in every sum that it enters."""
    c = Case(m, "f32", T, 72, 136, [3], "one", R=40)
    c.x.view(torch.int32)[2, 9] = 0x7F800001
    c.dy.view(torch.int32)[5, 11] = -0x7FFFFF  # 0xFF800001
    assert torch.isnan(c.x[2, 9]) and torch.isnan(c.dy[5, 11])
    y, dx = c.apply(), c.backward()
    ref.close(y, *c.want(), "y")
    c.check_backward(dx)
    assert torch.isnan(y[2]).all() and torch.isnan(dx[5]).all() and torch.isnan(c.dA[0][:, 9]).all() and torch.isnan(c.dB[0][:, 11]).all()
