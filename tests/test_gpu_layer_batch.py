"""The layer for a few tokens on the GPU against the 64-bit reference of
tests/serve_ref.py: the chosen experts exactly (router inputs on a grid, so that
every logit is exact in fp32 in any order), weights and outputs within the
bounds of the arithmetic."""
import pytest
import torch

import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import block_scaled_fp4_route_amd as m
    return m


def grid(g, *s, step):
    return (torch.randn(s, generator=g) * 16).round().clamp(-63, 63) * step


def blocks_of(g, E, H, I, fmt, lo=None, hi=None):
    n, G = 3 * H * I, ref.GROUP[fmt]
    b = torch.empty((E, n // 2 + n // G), dtype=torch.uint8)
    b[:, :n // 2] = torch.randint(0, 256, (E, n // 2), dtype=torch.uint8, generator=g)
    lo, hi = (lo, hi) if lo is not None else (0x18, 0x49) if fmt == "nvfp4" else (121, 130)
    b[:, n // 2:] = torch.randint(lo, hi, (E, n // G), dtype=torch.uint8, generator=g)
    return b


def matrices(block, H, I, fmt):
    n, G, out = H * I, ref.GROUP[fmt], []
    for i, (r, c) in enumerate(((I, H), (I, H), (H, I))):
        at = 3 * n // 2 + i * (n // G)
        out.append(ref.decode(block[i * n // 2:(i + 1) * n // 2].view(r, c // 2), block[at:at + n // G].view(r, c // G), fmt))
    return out


def route(x, Wr, k):
    logits = (x.double() @ Wr.double().t()).tolist()
    idx = torch.tensor([sorted(range(len(l)), key=lambda e: (-l[e], e))[:k] for l in logits], dtype=torch.int64)
    l = torch.gather(torch.tensor(logits, dtype=torch.float64), 1, idx)
    return idx, torch.softmax(l, 1)


class Case:
    def __init__(self, m, T, H, I, E, k, fmt, shared=False, masked=(), seed=0, x=None, Wr=None, lo=None, hi=None):
        g = torch.Generator().manual_seed(seed + T + H + I + E)
        self.m, self.T, self.H, self.I, self.E, self.k, self.fmt = m, T, H, I, E, k, fmt
        self.x = grid(g, T, H, step=1 / 256) if x is None else x
        self.Wr = grid(g, E, H, step=1 / 64) if Wr is None else Wr
        self.blocks = blocks_of(g, E, H, I, fmt, lo, hi)
        self.sh = [torch.randn(s, generator=g).bfloat16() for s in ((I, H), (I, H), (H, I))] if shared else None
        self.on = [t for t in range(T) if t not in masked]
        self.mask = None
        if masked:
            self.mask = torch.ones(T, dtype=torch.uint8)
            self.mask[list(masked)] = 0
            self.x = self.x.clone()
            self.x[list(masked)] = float("nan")
            self.mask = self.mask.cuda()
        self.d = m.desc(H, I, E, k, fmt)
        self.gb, self.gx, self.gW = self.blocks.cuda(), self.x.cuda(), self.Wr.cuda()
        self.ptrs = m.expert_ptr_table(self.gb)
        self.gsh = tuple(t.cuda() for t in self.sh) if shared else None
        self.ws = torch.full((m.moe_workspace_bytes(self.d, T, m.MOE_MODE_DECODE_BATCH),), 0xFF, dtype=torch.uint8, device="cuda")
        self.y = torch.full((T + 1, H), 7.0, device="cuda")
        self.idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
        self.w = torch.full((T + 1, k), 7.0, device="cuda")

    def call(self, **kw):
        self.m.moe_layer_decode_batch(self.d, self.gx, self.T, self.mask, self.gW, self.ptrs, self.gsh, self.y, self.idx, self.w, self.ws, **kw)
        return self

    def check(self):
        torch.cuda.synchronize()
        on, T = self.on, self.T
        off_rows = [t for t in range(T + 1) if t not in on]
        assert (self.y[off_rows] == 7).all() and (self.idx[off_rows] == -7).all() and (self.w[off_rows] == 7).all()
        if not on:
            return self
        idx, w = route(self.x[on], self.Wr, self.k)
        assert torch.equal(self.idx.cpu()[on].long(), idx)
        # logits exact; differences, expf, a sum of k and a division, each a few roundings
        ref.close(self.w[on], w, (self.k + 20) * ref.EPS * w + 1e-38, "w")
        mats = {int(e): matrices(self.blocks[int(e)], self.H, self.I, self.fmt) for e in idx.unique()}
        sh = [t.double() for t in self.sh] if self.sh else None
        y, off = ref.layer(self.x[on].double(), mats, sh, idx, w)
        off = off + (self.k + 20) * ref.EPS * 4 * y.abs().amax(1, keepdim=True)  # the weights' own roundings
        ref.close(self.y[on], y, off, "y")
        # the fp32 bar of the single-token decode is 1e-4; an output whose hidden values are below fp32's range
        # (2^-127 twice and x: 2^-250) is 0 in fp32, and only the bound above speaks of it
        if y.abs().max() > 2.0 ** -100:
            rel = (ref.cpu64(self.y[on]) - y).abs().max() / y.abs().max()
            assert rel <= 1e-5, rel
        return self


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 15, 16, 17, 31, 33, 48, 63, 64])
def test_token_counts(m, T, fmt, shared):
    Case(m, T, 512, 96, 24, 4, fmt, shared).call().check()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("H,I,E,k", [(512, 32, 1, 1), (512, 64, 2, 2), (1024, 160, 5, 5), (2560, 640, 12, 3), (4096, 32, 9, 2), (1536, 2880, 3, 1),
                                     (512, 4096, 4, 2), (4096, 544, 3, 2), (2048, 96, 40, 32), (3584, 224, 7, 6), (512, 32, 1024, 32), (1024, 64, 700, 12)])
@pytest.mark.parametrize("T", [1, 6, 40])
def test_shapes(m, T, H, I, E, k, fmt):
    Case(m, T, H, I, E, k, fmt, shared=(H + I + T) % 2 == 1).call().check()


@pytest.mark.parametrize("I", [16, 48, 80, 112, 656])
@pytest.mark.parametrize("T", [2, 21])
def test_odd_intermediate_sizes(m, T, I):
    """NVFP4 groups are 16 wide: I need not be a multiple of 32."""
    Case(m, T, 512, I, 9, 3, "nvfp4", shared=True).call().check()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [5, 33, 64])
def test_all_tokens_choose_the_same_experts(m, T, fmt):
    """Up to 64 rows of one expert; another expert has none."""
    g = torch.Generator().manual_seed(3)
    x = grid(g, 1, 512, step=1 / 256).repeat(T, 1)
    x[::2] = -x[::2].abs()  # two kinds of tokens
    Case(m, T, 512, 96, 6, 2, fmt, x=x).call().check()


@pytest.mark.parametrize("masked", [(0,), (3, 4, 11), tuple(range(5, 12)), tuple(range(12))])
@pytest.mark.parametrize("shared", [False, True])
def test_masked_tokens(m, masked, shared):
    """Empty slots (their x NaN) leave their rows as they were; every slot may be empty."""
    Case(m, 12, 512, 96, 24, 4, "nvfp4", shared, masked).call().check()


def test_equal_logits_choose_the_lowest_experts(m):
    c = Case(m, 5, 512, 32, 100, 8, "nvfp4", Wr=torch.zeros(100, 512)).call().check()
    assert c.idx[:5].tolist() == [list(range(8))] * 5


@pytest.mark.parametrize("T", [2, 20])
def test_values_with_all_their_bits(m, T):
    """x with 24 significant bits and rows far apart in size (the router's weights on a grid keep the choice apart)."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn((T, 1024), generator=g) * torch.exp(3 * torch.randn((T, 1), generator=g)) * 0.01
    c = Case(m, T, 1024, 160, 16, 4, "nvfp4", True, x=x)
    l = (x.double() @ c.Wr.double().t()).sort(dim=1, descending=True).values
    gap = (l[:, :4] - l[:, 1:5]).amin(1)  # between the chosen ones, and to the first that is not
    err = 1026 * ref.EPS * (x.double().abs() @ c.Wr.double().abs().t()).amax(1)
    keep = (gap > 2 * err).nonzero()[:, 0].tolist()
    assert keep
    c.call()
    torch.cuda.synchronize()
    idx, w = route(x, c.Wr, 4)
    assert torch.equal(c.idx.cpu()[keep].long(), idx[keep])
    mats = {int(e): matrices(c.blocks[int(e)], 1024, 160, "nvfp4") for e in idx[keep].unique()}
    y, off = ref.layer(x[keep].double(), mats, [t.double() for t in c.sh], idx[keep], c.w.cpu()[keep].double())
    ref.close(c.y[keep], y, off, "y")


@pytest.mark.parametrize("fmt,byte", [("mxfp4", 0), ("mxfp4", 40), ("nvfp4", 0), ("nvfp4", 1)])
def test_smallest_scales(m, fmt, byte):
    Case(m, 3, 512, 64, 4, 2, fmt, lo=byte, hi=byte + 2).call().check()


def test_agrees_with_the_single_token_decode(m):
    c = Case(m, 6, 2560, 640, 32, 10, "nvfp4", True).call()
    y, idx, w = torch.empty(2560, device="cuda"), torch.empty(10, dtype=torch.int32, device="cuda"), torch.empty(10, device="cuda")
    ws = m.alloc_workspace(c.d, 1, m.MOE_MODE_DECODE)
    for t in range(6):
        m.moe_layer_decode(c.d, c.gx[t], c.gW, c.ptrs, c.gsh, y, idx, w, ws)
        assert torch.equal(idx, c.idx[t])
        assert ((y - c.y[t]).abs().max() / y.abs().max()).item() <= 1e-5


@pytest.mark.parametrize("T", [1, 9, 40])
def test_repeated_and_replayed(m, T):
    """Bit-identical from run to run, and as two graphs that share one workspace, with junk in it between replays."""
    a, b = (Case(m, T, 512, 96, 24, 4, "nvfp4", True, seed=s) for s in (0, 1))
    b.ws = a.ws
    a.call().check()
    b.call().check()
    want = [t.clone() for c in (a, b) for t in (c.y, c.idx, c.w)]
    graphs = []
    for c in (a, b):
        q = torch.cuda.CUDAGraph()
        with torch.cuda.graph(q):
            c.call()
        graphs.append(q)
    for fill in (0xFF, 0x00, 0x7F):
        for c in (a, b):
            c.y[:T].fill_(9)
        a.ws.fill_(fill)
        graphs[0].replay()
        graphs[1].replay()
        torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip([t for c in (a, b) for t in (c.y, c.idx, c.w)], want))


def test_two_streams_at_once(m):
    cs = [Case(m, 9, 512, 96, 24, 4, "mxfp4", True, seed=s) for s in (0, 1)]
    want = []
    for c in cs:
        c.call().check()
        want.append(c.y.clone())
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cs, streams):
            c.call(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(c.y, w) for c, w in zip(cs, want))
