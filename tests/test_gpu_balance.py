"""The router's balance loss on the GPU against its definition in 64 bits
(tests/learn_ref.py, which also derives the bounds), its gradient against
differences of that definition, its refusals of bad device data, and its use
on streams and in graphs."""
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
    def __init__(self, m, T, E, k, S=1, masked=0.0, seed=0, off=None, std=1.0):
        g = torch.Generator().manual_seed(1000 * T + 10 * E + k + seed)
        self.m, self.T, self.E, self.k = m, T, E, k
        self.logits = torch.randn((T, E), generator=g) * std + torch.randn(E, generator=g)
        self.idx = (torch.topk(self.logits, k, dim=1).indices if T else torch.zeros((0, k))).to(torch.int32)
        self.mask = (torch.rand(T, generator=g) >= masked) if masked else torch.ones(T, dtype=torch.bool)
        self.has_mask = masked > 0
        cuts = sorted(torch.randint(0, T + 1, (S - 1,), generator=g).tolist())
        self.off = off if off is not None else [0, *cuts, T]
        self.S = len(self.off) - 1

    def run(self, cb=0.01, cz=0.001, up=None, grad=True, stream=None, ws=None, whole=False):
        m, T, E, S, dev = self.m, self.T, self.E, self.S, "cuda"
        self.d = m.desc(256, 64, E, self.k, "nvfp4")
        self.ld = self.logits.to(dev)
        self.idd = self.idx.to(dev)
        self.md = self.mask.to(torch.uint8).to(dev) if self.has_mask else None
        self.od = None if whole else torch.tensor(self.off, dtype=torch.int32, device=dev)
        self.ud = None if up is None else torch.tensor([up], dtype=torch.float32, device=dev)
        self.out = {"loss": torch.full((3,), 7.0, device=dev), "counts": torch.full((S, E), 7, dtype=torch.int32, device=dev),
                    "probs": torch.full((S, E), 7.0, device=dev),
                    "dlogits": torch.full((T, E), 7.0, device=dev) if grad else None}
        n = m.moe_balance_workspace_bytes(self.d, T, S)
        # junk in the workspace: nothing in it may matter
        self.ws = torch.full((n,), 0xA5, dtype=torch.uint8, device=dev) if ws is None else ws
        torch.cuda.synchronize()
        self.args = (self.d, self.ld, T, self.idd, self.md, self.od, S, cb, cz, self.ud, self.out["loss"],
                     self.out["counts"], self.out["probs"], self.out["dlogits"], self.ws)
        m.moe_balance_loss(*self.args, stream=stream)
        torch.cuda.synchronize()
        return self.out

    def check(self, out, cb=0.01, cz=0.001, up=1.0):
        want = ref.balance(self.logits, self.idx, self.mask, self.off, self.k, cb, cz, up)
        assert torch.equal(out["counts"].cpu().long(), want["counts"])
        for name in ("loss", "probs", "dlogits"):
            if out[name] is not None:
                ref.close(out[name], *want[name], name)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 512, 10), (3, 7, 7), (5, 8, 2), (17, 384, 6), (64, 64, 8), (311, 384, 6),
                                   (300, 513, 10), (130, 1023, 32), (257, 1024, 32), (1030, 256, 4), (2451, 512, 10), (40, 257, 1)])
def test_one_sequence(m, T, E, k):
    c = Case(m, T, E, k)
    c.check(c.run(up=0.75, whole=True), up=0.75)


@pytest.mark.parametrize("T,E,k,S,masked", [(1, 16, 2, 3, 0.0), (900, 1023, 2, 300, 0.1), (500, 40, 3, 1000, 0.2), (200, 64, 3, 65535, 0.0), (100, 60, 4, 5, 0.3), (777, 512, 10, 9, 0.0),
                                            (777, 130, 10, 64, 0.5), (4500, 384, 6, 2, 0.1), (33, 33, 3, 40, 0.9)])
def test_sequences_and_masks(m, T, E, k, S, masked):
    c = Case(m, T, E, k, S, masked)
    c.check(c.run())


@pytest.mark.parametrize("cb,cz", [(0.0, 0.0), (1.0, 0.0), (0.0, 1.0), (-0.5, 2.0)])
def test_coefficients(m, cb, cz):
    c = Case(m, 70, 48, 4, 3, 0.2)
    c.check(c.run(cb, cz, up=-2.0), cb, cz, up=-2.0)
    c.check(c.run(cb, cz, grad=False), cb, cz)


def test_tokens_outside_the_sequences(m):
    """Tokens before the first and behind the last sequence are not counted; their gradient rows are 0."""
    c = Case(m, 90, 64, 4, off=[7, 7, 30, 81, 81])
    c.logits[:7] = float("nan")
    c.logits[81:] = float("inf")
    want = Case(m, 90, 64, 4, off=c.off)
    out = c.run()
    assert (out["dlogits"][:7] == 0).all() and (out["dlogits"][81:] == 0).all()
    want.idx = c.idx
    want.check(out)


def test_nothing_counted(m):
    for T, off in ((0, [0, 0]), (5, [3, 3, 3]), (5, [0, 0])):
        c = Case(m, T, 24, 3, off=off)
        out = c.run()
        assert (out["loss"] == 0).all() and (out["counts"] == 0).all() and (out["probs"] == 0).all()
        assert (out["dlogits"] == 0).all()
    c = Case(m, 9, 24, 3, masked=0.5)
    c.mask[:] = False
    c.logits[:] = float("nan")
    c.idx[:] = -5
    out = c.run()
    assert (out["loss"] == 0).all() and (out["dlogits"] == 0).all()


def test_masked_rows_hold_anything(m):
    """NaN, infinities and bad indices in masked rows change nothing, bit for bit."""
    a, b = Case(m, 200, 96, 5, 4, 0.4), Case(m, 200, 96, 5, 4, 0.4)
    off = (~b.mask).nonzero()[:, 0]
    b.logits[off[::3]] = float("nan")
    b.logits[off[1::3]] = float("inf")
    b.logits[off[2::3]] = -float("inf")
    b.idx[off] = 1 << 30
    x, y = a.run(), b.run()
    for name in x:
        assert torch.equal(x[name], y[name]), name
    a.check(x)


def test_infinite_logits(m):
    """-inf excludes an expert; a row of -inf has no probabilities; a row of
    the lowest fp32 value is uniform; +inf and NaN reach the loss."""
    c = Case(m, 40, 30, 3)
    low = torch.finfo(torch.float32).min
    c.logits[3, :20] = -float("inf")
    c.logits[4] = -float("inf")
    c.logits[5, ::2] = low
    out = c.run()
    c.check(out)
    assert (out["dlogits"][4] == 0).all() and (out["dlogits"][3, :20] == 0).all()
    c.logits[6] = low
    out = c.run(cz=0.0)  # lse^2 of that row overflows; without the z term nothing else does
    c.check({**out, "loss": out["loss"][:2], "dlogits": out["dlogits"]} | {"loss": None}, cz=0.0)
    assert torch.isfinite(out["loss"][:2]).all() and torch.isinf(out["loss"][2])
    ref.close(out["probs"], *ref.balance(c.logits, c.idx, c.mask, c.off, 3, 0.01, 0.0)["probs"], "probs")
    c.logits[7, 1] = float("inf")
    assert torch.isnan(c.run()["loss"]).all()
    c.logits[7, 1] = float("nan")
    assert torch.isnan(c.run()["loss"]).all()
    c.logits[7] = -float("inf")
    c.logits[7, 1] = float("nan")
    assert torch.isnan(c.run()["loss"]).all()


@pytest.mark.parametrize("off", [[0, 5, 4, 9], [0, 10], [-1, 9], [4, 2], [0, 1 << 30]])
def test_bad_offsets(m, off):
    c = Case(m, 9, 32, 2, off=[0] * (len(off) - 1) + [9])
    c.off = off
    out = c.run()
    assert torch.isnan(out["loss"]).all() and torch.isnan(out["probs"]).all() and torch.isnan(out["dlogits"]).all()
    assert (out["counts"] == -1).all()


@pytest.mark.parametrize("bad", [-1, 32, 1 << 30, -(1 << 31)])
def test_bad_expert(m, bad):
    c = Case(m, 1200, 32, 2, 2, off=[0, 600, 1200])
    c.idx[700, 1] = bad
    out = c.run()
    assert torch.isnan(out["loss"]).all() and torch.isnan(out["dlogits"]).all() and (out["counts"] == -1).all()


def test_an_expert_named_twice(m):
    c = Case(m, 50, 16, 4)
    c.idx[:, 1] = c.idx[:, 0]
    c.check(c.run())


def test_gradient_against_differences(m):
    """Central differences of the 64-bit loss with the counts held: the third
    derivative times h^2 is below 1e-7 of the largest gradient at h = 1e-4."""
    c = Case(m, 12, 20, 3, 2, 0.2)
    out = c.run(0.7, 0.3)["dlogits"].cpu().double()
    h, scale = 1e-4, out.abs().max().item()
    for t in range(12):
        for e in range(0, 20, 3):
            v = []
            for sign in (1, -1):
                l = c.logits.double().clone()
                l[t, e] += sign * h
                v.append(ref.balance(l, c.idx, c.mask, c.off, 3, 0.7, 0.3)["loss"][0][0].item())
            assert abs((v[0] - v[1]) / (2 * h) - out[t, e].item()) <= 2e-6 * scale


def test_runs_are_identical_and_any_workspace_does(m):
    c = Case(m, 3000, 384, 6, 5, 0.1)
    a = c.run()
    b = c.run(ws=torch.full_like(c.ws, 0xFF))
    for name in a:
        assert torch.equal(a[name], b[name]), name


def test_long_batch_offsets_past_32_bits(m):
    """T * E beyond 2^31 elements: the last rows are read and written where they are."""
    E, T = 1024, (1 << 21) + 50
    dev = "cuda"
    logits = torch.zeros((T, E), device=dev)
    g = torch.Generator(device=dev).manual_seed(3)
    logits[-100:] = torch.randn((100, E), generator=g, device=dev)
    idx = torch.zeros((T, 2), dtype=torch.int32, device=dev)
    idx[-100:] = torch.topk(logits[-100:], 2, dim=1).indices.to(torch.int32)
    off = torch.tensor([T - 100, T], dtype=torch.int32, device=dev)
    d = m.desc(256, 64, E, 2, "nvfp4")
    loss, dl = torch.empty(3, device=dev), torch.empty((T, E), device=dev)
    counts = torch.empty((1, E), dtype=torch.int32, device=dev)
    ws = torch.empty(m.moe_balance_workspace_bytes(d, T, 1), dtype=torch.uint8, device=dev)
    m.moe_balance_loss(d, logits, T, idx, None, off, 1, 0.01, 0.001, None, loss, counts, None, dl, ws)
    want = ref.balance(logits[-100:].cpu(), idx[-100:].cpu(), torch.ones(100, dtype=torch.bool), [0, 100], 2, 0.01, 0.001)
    ref.close(loss, *want["loss"], "loss")
    ref.close(dl[-100:], *want["dlogits"], "dlogits")
    assert torch.equal(counts.cpu().long(), want["counts"])
    assert not dl[:T - 100].any()


def test_on_another_stream_and_two_at_once(m):
    a, b = Case(m, 800, 256, 8, 3, 0.2), Case(m, 640, 100, 4, 2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    a.run()
    b.run()
    wa, wb = {k: v.clone() for k, v in a.out.items()}, {k: v.clone() for k, v in b.out.items()}
    for _ in range(3):
        for c in (a, b):
            for v in c.out.values():
                v.fill_(9)
        torch.cuda.synchronize()
        m.moe_balance_loss(*a.args, stream=sa)
        m.moe_balance_loss(*b.args, stream=sb)
        torch.cuda.synchronize()
        for c, w in ((a, wa), (b, wb)):
            for k, v in c.out.items():
                assert torch.equal(v, w[k]), k


def test_graphs_that_share_a_workspace(m):
    a, b = Case(m, 800, 256, 8, 3, 0.2), Case(m, 640, 100, 4, 2)
    n = max(m.moe_balance_workspace_bytes(m.desc(256, 64, 256, 8, "nvfp4"), 800, 3),
            m.moe_balance_workspace_bytes(m.desc(256, 64, 100, 4, "nvfp4"), 640, 2))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    graphs, want = [], []
    for c in (a, b):
        c.run(ws=ws)
        want.append({k: v.clone() for k, v in c.out.items()})
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_balance_loss(*c.args)
        graphs.append(g)
    for turn in range(4):
        for c in (a, b):
            for v in c.out.values():
                v.fill_(9)
        for g in (graphs if turn % 2 else graphs[::-1]):
            g.replay()
        ws_use = torch.randn(1000, device="cuda").sum()  # other work between
        torch.cuda.synchronize()
        assert torch.isfinite(ws_use)
        for c, w in zip((a, b), want):
            for k, v in c.out.items():
                assert torch.equal(v, w[k]), (turn, k)
        a.ld.add_(0)
        m.moe_balance_loss(*a.args)


@pytest.mark.parametrize("T,E,k", [(37, 20, 2), (1900, 512, 10), (700, 1023, 3)])
@pytest.mark.parametrize("S", [4, 5, 7, 8, 9, 10])
def test_few_and_many_sequences(m, T, E, k, S):
    """Both sides of the number of sequences that the reducing launch is shaped by."""
    test_sequences_and_masks(m, T, E, k, S, 0.1)
