"""4-bit quantisation and products on the GPU against the 64-bit references of
tests/serve_ref.py: codes, scales and values bit for bit, products within the
bound of one fp32 sum."""
import pytest
import torch

import serve_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import block_scaled_fp4_route_amd as m
    return m


def rule_of(m, rule):
    return {"nearest": m.MOE_SCALE_NEAREST, "floor": m.MOE_SCALE_FLOOR, "ceil": m.MOE_SCALE_CEIL}[rule]


def check_quant(m, x, fmt, rule, rows, ldv=None, inplace=False):
    """x [r][c] on the GPU, rows maybe apart in memory."""
    r, c = x.shape
    codes0, scales0, e0, val = ref.quant(x, fmt, rule, rows)
    want = ref.stored(val, x.dtype)
    G = ref.GROUP[fmt]
    codes = torch.full((r, c // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((r, c // G), 0xAA, dtype=torch.uint8, device="cuda")
    e = torch.full((r,), 77, dtype=torch.int8, device="cuda") if rows else None
    if inplace:
        v = x
    else:
        ldv = ldv or c
        v = torch.full((r, ldv), 5.0, dtype=x.dtype, device="cuda")[:, :c]
    m.moe_fp4_quant(x, x.stride(0), r, c, x.dtype, fmt, rule_of(m, rule), e, codes, scales, v, v.stride(0))
    torch.cuda.synchronize()
    assert torch.equal(scales.cpu(), scales0)
    assert torch.equal(codes.cpu(), codes0)
    if rows:
        assert torch.equal(e.cpu(), e0)
    bits = torch.int32 if x.dtype == torch.float32 else torch.int16
    g, w = v.cpu().contiguous(), want
    assert torch.equal(g.isnan(), w.isnan())
    assert torch.equal(g.nan_to_num(0, 1e4, -1e4).view(bits), w.nan_to_num(0, 1e4, -1e4).view(bits))
    return codes, scales, e


KINDS = [("nvfp4", "nearest", True), ("nvfp4", "nearest", False), ("mxfp4", "floor", False), ("mxfp4", "ceil", False)]


@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("fmt,rule,rows", KINDS)
@pytest.mark.parametrize("r,c", [(1, 32), (3, 64), (17, 2560), (5, 2080), (301, 96), (2, 8224), (1, 16416)])
def test_quant(m, r, c, fmt, rule, rows, dt):
    g = torch.Generator().manual_seed(r * c)
    x = (torch.randn((r, c), generator=g) * torch.exp(torch.randn((r, 1), generator=g))).to(DT[dt]).cuda()
    check_quant(m, x, fmt, rule, rows)


@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("fmt,rule,rows", KINDS)
def test_quant_borders_and_extremes(m, fmt, rule, rows, dt):
    """Every border between codes and between scales, one step below and above it; zeros of both signs; the type's
    largest, smallest and subnormal values; infinities and NaN."""
    t = DT[dt]
    fi = torch.finfo(t)
    g = torch.Generator().manual_seed(3)
    rows_ = []
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 2.0, 4.0, 7.0, 0.0, -0.0, 5.5], dtype=torch.float64)
    for s in (1.0, 1.125, 0.875 * 2, 2.0 ** -6, 2.0 ** -9, 3 * 2.0 ** -9, 448.0, 2.0 ** 4 * 1.875):
        v = (mids * s).to(t)
        up, down = torch.nextafter(v, torch.full_like(v, fi.max)), torch.nextafter(v, torch.full_like(v, -fi.max))
        for u in (v, up, down, -v):
            u = u.clone()
            u[-1] = torch.tensor(6 * s).to(t)  # the block's largest: the scale is s
            rows_.append(torch.cat([u, u]))
    grid = ref.e4m3(torch.arange(127))
    border = (6 * (grid[1:] + grid[:-1]) / 2).to(t)  # between two scales
    for b in (border, torch.nextafter(border, torch.full_like(border, fi.max)), torch.nextafter(border, torch.zeros_like(border))):
        for x in b:
            v = (torch.rand(32, generator=g) * float(x)).to(t)
            v = torch.minimum(v, x)
            v[3], v[20] = x, -x
            rows_.append(v)
    for top in (fi.max, fi.max / 2, fi.tiny, fi.smallest_normal, fi.smallest_normal / 4, fi.smallest_normal * 2688, 1.5 * fi.max / 2):
        v = ((torch.rand(32, generator=g).double() * 2 - 1) * top).to(t)
        v[0], v[16] = torch.tensor(top, dtype=torch.float64).to(t), -torch.tensor(top, dtype=torch.float64).to(t)
        rows_.append(v)
    rows_.append(torch.zeros(32, dtype=t))
    rows_.append(-torch.zeros(32, dtype=t))
    for bad in (float("inf"), -float("inf"), float("nan")):
        v = torch.randn(32, generator=g).to(t)
        v[5] = bad
        rows_.append(v)
    x = torch.stack(rows_)
    x = torch.cat([x, x.roll(1, 0)], dim=1).contiguous().cuda()
    check_quant(m, x, fmt, rule, rows)


@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("fmt,rule,rows", KINDS)
def test_quant_random_bits(m, fmt, rule, rows, dt):
    """Any bit patterns; then blocks of every exponent whose values lie within 2^7 of one another, with few significant
    bits (many ties)."""
    t = DT[dt]
    g = torch.Generator().manual_seed(8)
    bits = torch.int32 if t == torch.float32 else torch.int16
    x = torch.randint(torch.iinfo(bits).min, torch.iinfo(bits).max, (300, 128), dtype=torch.int64, generator=g).to(bits).view(t)
    check_quant(m, x.cuda(), fmt, rule, rows)
    lo, hi = {"f32": (-149, 127), "bf16": (-133, 127), "f16": (-24, 15)}[dt]
    e = torch.arange(lo, hi - 2).repeat_interleave(4)[:, None] + torch.randint(-5, 3, (4 * (hi - 2 - lo), 128), generator=g)
    x = torch.randint(-15, 16, e.shape, generator=g).double() / 8 * torch.exp2(e.double())
    check_quant(m, x.to(t).cuda(), fmt, rule, rows)


@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("fmt,rule,rows", KINDS)
def test_quant_strides_and_in_place(m, fmt, rule, rows, dt):
    x = torch.randn((9, 640), device="cuda").to(DT[dt])
    keep = x.clone()
    check_quant(m, x[:, :96], fmt, rule, rows, ldv=104)
    check_quant(m, x[:, 64:64 + 96], fmt, rule, rows, inplace=True)
    assert torch.equal(x[:, :64], keep[:, :64]) and torch.equal(x[:, 160:], keep[:, 160:])
    big = torch.randn((3, 9216), device="cuda").to(DT[dt])  # longer than a row's registers
    check_quant(m, big, fmt, rule, rows, inplace=True)


def test_quant_outputs_left_out(m):
    x = torch.randn((5, 64), device="cuda")
    codes, scales = torch.empty((5, 32), dtype=torch.uint8, device="cuda"), torch.empty((5, 4), dtype=torch.uint8, device="cuda")
    e = torch.empty(5, dtype=torch.int8, device="cuda")
    m.moe_fp4_quant(x, 64, 5, 64, x.dtype, "nvfp4", m.MOE_SCALE_NEAREST, e, codes, scales, None, 0)
    for part in ("codes", "scales", "values", "e"):
        c2, s2, v2, e2 = torch.zeros_like(codes), torch.zeros_like(scales), torch.zeros_like(x), torch.zeros_like(e)
        m.moe_fp4_quant(x, 64, 5, 64, x.dtype, "nvfp4", m.MOE_SCALE_NEAREST, e2, c2 if part == "codes" else None,
                        s2 if part == "scales" else None, v2 if part == "values" else None, 64)
        assert torch.equal(e, e2)
        got, want = {"codes": (c2, codes), "scales": (s2, scales), "values": (v2.cpu().double(), ref.decode(codes, scales, "nvfp4", e)), "e": (e2, e)}[part]
        assert torch.equal(got, want), part


def test_three_quantised_matrices_are_an_expert_block(m):
    """The codes and scales of gate, up and down fill a block's regions: moe_dequant_block gives the values."""
    H, I, fmt = 512, 96, "mxfp4"
    d = m.desc(H, I, 1, 1, fmt)
    off = m.moe_block_layout(d)
    block = torch.zeros(off[6], dtype=torch.uint8, device="cuda")
    vals = []
    for i, (r, c) in enumerate(((I, H), (I, H), (H, I))):
        w = (torch.randn((r, c), device="cuda") * 0.02).bfloat16()
        v = torch.empty_like(w)
        m.moe_fp4_quant(w, c, r, c, w.dtype, fmt, m.MOE_SCALE_CEIL, None, block[off[i]:off[i + 1]], block[off[3 + i]:off[4 + i]], v, c)
        vals.append(v.float())
    out = [torch.empty_like(v) for v in vals]
    m.moe_dequant_block(d, block, *out)
    assert all(torch.equal(a, b) for a, b in zip(out, vals))


# ---- products ----

def matrix(g, N, K, fmt, lo=None, hi=None, rows=True):
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g)
    lo, hi = lo if lo is not None else (0x18 if fmt == "nvfp4" else 121), hi or (0x49 if fmt == "nvfp4" else 130)
    scales = torch.randint(lo, hi, (N, K // ref.GROUP[fmt]), dtype=torch.uint8, generator=g)
    e = torch.randint(-9, 3, (N,), dtype=torch.int8, generator=g) if fmt == "nvfp4" and rows else None
    return codes.cuda(), scales.cuda(), None if e is None else e.cuda()


def padded(rows, cols, pad, dt, fill=3.0):
    """A [rows][cols] view of a wider buffer, and the buffer."""
    buf = torch.full((rows + 1, cols + pad), fill, dtype=dt, device="cuda")
    return buf[:rows, :cols], buf


def check_product(m, T, K, N, fmt, dt, rnd=False, back=False, base="other", pad=8, seed=0, x=None, w=None):
    g = torch.Generator().manual_seed(seed + T * 31 + K * 7 + N)
    t = DT[dt]
    codes, scales, e = w or matrix(g, N, K, fmt)
    W = ref.decode(codes, scales, fmt, e)
    ki, ko = (N, K) if back else (K, N)
    xin, _ = padded(T, ki, pad, t)
    xin.copy_(x if x is not None else torch.randn((T, ki), generator=g).to(t))
    out, buf = padded(T, ko, pad, t)
    b = None
    if base == "other":
        b, _ = padded(T, ko, 2 * pad, t)
        b.copy_((torch.randn((T, ko), generator=g) * 3).to(t))
    elif base == "same":
        b = out
        out.copy_((torch.randn((T, ko), generator=g) * 3).to(t))
    b0 = None if b is None else b.clone()
    f = m.fp4_desc(K, N, fmt, t)
    ws = torch.full((m.moe_fp4_workspace_bytes(f, T, back),), 0xFF, dtype=torch.uint8, device="cuda")
    ldb = 0 if b is None else b.stride(0)
    if back:
        m.moe_fp4_backward(f, xin, xin.stride(0), T, codes, scales, e, b, ldb, out, out.stride(0), ws)
    else:
        m.moe_fp4_apply(f, xin, xin.stride(0), T, codes, scales, e, rnd, b, ldb, out, out.stride(0), ws)
    torch.cuda.synchronize()
    xv = ref.cpu64(xin)
    if rnd:
        xv = ref.quant(xin, "mxfp4", "floor", False)[3]
    want, off = ref.product(xv, W.t().contiguous() if back else W, b0, t)
    ref.close(out, want, off, (T, K, N, fmt, dt, rnd, back, base))
    assert (buf[T:] == 3).all() and (buf[:, ko:] == 3).all()  # nothing behind the rows
    return out.clone()


@pytest.mark.parametrize("fmt,rnd", [("nvfp4", False), ("mxfp4", False), ("mxfp4", True)])
@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 33, 63, 64, 65, 128, 129, 300])
def test_product_token_counts(m, T, dt, fmt, rnd):
    check_product(m, T, 544, 264, fmt, dt, rnd)


@pytest.mark.parametrize("fmt,rnd", [("nvfp4", False), ("mxfp4", False), ("mxfp4", True)])
@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("K,N", [(32, 8), (64, 16), (96, 40), (2560, 640), (160, 1000), (4096, 72), (1056, 136)])
@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_product_shapes(m, T, K, N, dt, fmt, rnd):
    check_product(m, T, K, N, fmt, dt, rnd, base=("none", "same", "other")[(T + K + N) % 3])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("T", [1, 2, 16, 17, 64, 65, 129, 300])
def test_backward_token_counts(m, T, dt, fmt):
    check_product(m, T, 544, 264, fmt, dt, back=True)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("K,N", [(32, 8), (64, 16), (96, 40), (640, 2560), (160, 1000), (4096, 72), (1056, 136)])
@pytest.mark.parametrize("T", [1, 40, 200])
def test_backward_shapes(m, T, K, N, dt, fmt):
    check_product(m, T, K, N, fmt, dt, back=True, base=("none", "same", "other")[(T + K + N) % 3])


@pytest.mark.parametrize("T,K,N", [(1000, 2560, 1032), (2049, 1024, 520)])
@pytest.mark.parametrize("fmt,dt,rnd,back", [("nvfp4", "f16", False, False), ("mxfp4", "bf16", True, False), ("mxfp4", "f16", False, False),
                                             ("nvfp4", "f32", False, False), ("mxfp4", "bf16", False, True), ("nvfp4", "f16", False, True)])
def test_product_long(m, T, K, N, fmt, dt, rnd, back):
    check_product(m, T, K, N, fmt, dt, rnd, back)


@pytest.mark.parametrize("T,K,N,fmt,dt,rnd,back", [
    (40, 64, 8192, "nvfp4", "f32", False, True),      # one tile, its sum over 16 workgroups
    (1, 256, 4104, "mxfp4", "bf16", False, True),
    (130, 5600, 72, "mxfp4", "f16", False, False),    # six tiles, a sum that ends within a step
    (200, 12320, 136, "mxfp4", "bf16", True, False),
    (257, 3200, 200, "nvfp4", "f32", False, False),
    (700, 4160, 1032, "nvfp4", "f32", False, False),  # 54 tiles of 128 x 128, nine parts each
    (700, 1056, 4104, "mxfp4", "bf16", False, True),
    (800, 16416, 1000, "mxfp4", "bf16", True, False)])
def test_product_split_sums(m, T, K, N, fmt, dt, rnd, back):
    check_product(m, T, K, N, fmt, dt, rnd, back)


@pytest.mark.parametrize("fmt,dt,rnd,back", [("mxfp4", "bf16", False, True), ("nvfp4", "f16", False, False), ("mxfp4", "bf16", True, False),
                                             ("nvfp4", "f32", False, True)])
def test_product_last_round_split(m, fmt, dt, rnd, back):
    """17 x 16 tiles of 256 x 256 with ragged edges: one round of the chip and 16 tiles in several parts. Every row of the last
    tiles and some of the others against the reference."""
    T, ko, ki = 4200, 4096 - 24, 8192 if rnd else 3392
    K, N = (ko + 24, ki) if back else (ki, ko)
    g = torch.Generator().manual_seed(11)
    codes, scales, e = matrix(g, N, K, fmt)
    W = ref.decode(codes, scales, fmt, e)
    W = W.t().contiguous() if back else W
    ko = K if back else N
    x = torch.randn((T, W.shape[1]), generator=g).to(DT[dt])
    y = torch.empty((T, ko), dtype=DT[dt], device="cuda")
    f = m.fp4_desc(K, N, fmt, DT[dt])
    ws = torch.full((m.moe_fp4_workspace_bytes(f, T, back),), 0xFF, dtype=torch.uint8, device="cuda")
    if back:
        m.moe_fp4_backward(f, x.cuda(), N, T, codes, scales, e, None, 0, y, K, ws)
    else:
        m.moe_fp4_apply(f, x.cuda(), K, T, codes, scales, e, rnd, None, 0, y, N, ws)
    rows = torch.cat([torch.arange(0, 4096, 97), torch.arange(4096, T)])
    xs = ref.quant(x[rows], "mxfp4", "floor", False)[3] if rnd else x[rows].double()
    want, off = ref.product(xs, W, None, DT[dt])
    ref.close(y.cpu()[rows], want, off, (fmt, dt, rnd, back))


@pytest.mark.parametrize("T", [3, 20, 50, 200])
@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("back", [False, True])
def test_product_far_scales(m, T, dt, back):
    """MXFP4 scales down to 2^-127 (decoded values that are subnormal bf16) and up to where fp32 still holds the values;
    NVFP4's subnormal scales and row exponents at both ends."""
    g = torch.Generator().manual_seed(5)
    K, N = 96, 40
    for lo, hi in ((0, 6), (118, 137), (240, 247)):
        x = torch.randn((T, N if back else K), generator=g)
        x = x * 2.0 ** (100 if lo == 0 and dt != "f16" else -10 if lo == 240 else 0)
        if lo == 240 and dt == "f16":
            continue  # outside of fp16
        check_product(m, T, K, N, "mxfp4", dt, back=back, w=matrix(g, N, K, "mxfp4", lo, hi), x=x.to(DT[dt]), base="none")
    c, s, _ = matrix(g, N, K, "nvfp4", 1, 9)
    e = torch.tensor([-100, 60, -3, 0, 7], dtype=torch.int8).repeat(8).cuda()
    check_product(m, T, K, N, "nvfp4", dt, back=back, w=(c, s, e if dt != "f16" else e.clamp(-8, 8)), base="none")


@pytest.mark.parametrize("T", [2, 20, 200])
@pytest.mark.parametrize("fmt,rnd", [("nvfp4", False), ("mxfp4", False), ("mxfp4", True)])
@pytest.mark.parametrize("dt", sorted(DT))
def test_product_infinities_and_nan(m, T, dt, fmt, rnd):
    """Infinities and NaN among the activations reach their own token's outputs as in fp32, no other token's."""
    g = torch.Generator().manual_seed(8)
    K, N = 160, 72
    codes, scales, e = matrix(g, N, K, fmt)
    x = torch.randn((T, K), generator=g).to(DT[dt])
    x[0, 3], x[1, 40] = float("inf"), float("nan")
    t = DT[dt]
    y = torch.empty((T, N), dtype=t, device="cuda")
    f = m.fp4_desc(K, N, fmt, t)
    ws = torch.empty(m.moe_fp4_workspace_bytes(f, T, False), dtype=torch.uint8, device="cuda")
    m.moe_fp4_apply(f, x.cuda(), K, T, codes, scales, e, rnd, None, 0, y, N, ws)
    xv = ref.quant(x, "mxfp4", "floor", False)[3] if rnd else x.double()
    W = ref.decode(codes, scales, fmt, e)
    got = y.cpu().double()
    want = torch.stack([(xv[i] * W).sum(1) for i in range(T)])
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    assert torch.equal(got[got.isinf()], want[want.isinf()])
    rest, off = ref.product(xv[2:], W, None, t)
    ref.close(y[2:], rest, off, "other tokens")


@pytest.mark.parametrize("T", [2, 20, 200])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("back", [False, True])
def test_product_nan_scale(m, T, fmt, back):
    """A NaN scale makes the outputs NaN that its block enters."""
    g = torch.Generator().manual_seed(9)
    K, N = 160, 72
    codes, scales, e = matrix(g, N, K, fmt)
    scales[5, 1] = 0x7F if fmt == "nvfp4" else 0xFF
    x = torch.randn((T, N if back else K), generator=g).cuda()
    y = torch.empty((T, K if back else N), device="cuda")
    f = m.fp4_desc(K, N, fmt, torch.float32)
    ws = torch.empty(m.moe_fp4_workspace_bytes(f, T, back), dtype=torch.uint8, device="cuda")
    hit = torch.zeros(K if back else N, dtype=torch.bool, device="cuda")
    if back:
        m.moe_fp4_backward(f, x, N, T, codes, scales, e, None, 0, y, K, ws)
        G = ref.GROUP[fmt]
        hit[G:2 * G] = True
    else:
        m.moe_fp4_apply(f, x, K, T, codes, scales, e, False, None, 0, y, N, ws)
        hit[5] = True
    assert y[:, hit].isnan().all() and y[:, ~hit].isfinite().all()


@pytest.mark.parametrize("T", [1, 48, 200])
@pytest.mark.parametrize("kind", ["kept", "rounded", "back"])
def test_product_graphs_share_a_workspace(m, T, kind):
    """Two captured calls on one workspace, replayed in turn with junk in it between: bit for bit the eager results."""
    g = torch.Generator().manual_seed(T)
    K, N = 544, 264
    codes, scales, _ = matrix(g, N, K, "mxfp4")
    f = m.fp4_desc(K, N, "mxfp4", torch.bfloat16)
    back = kind == "back"
    ws = torch.empty(m.moe_fp4_workspace_bytes(f, T, back), dtype=torch.uint8, device="cuda")
    xs = [torch.randn((T, N if back else K), generator=g).bfloat16().cuda() for _ in range(2)]
    ys = [torch.empty((T, K if back else N), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def call(i):
        if back:
            m.moe_fp4_backward(f, xs[i], N, T, codes, scales, None, None, 0, ys[i], K, ws)
        else:
            m.moe_fp4_apply(f, xs[i], K, T, codes, scales, None, kind == "rounded", None, 0, ys[i], N, ws)

    call(0)
    call(1)
    want = [y.clone() for y in ys]
    graphs = []
    for i in range(2):
        q = torch.cuda.CUDAGraph()
        with torch.cuda.graph(q):
            call(i)
        graphs.append(q)
    for _ in range(3):
        for y in ys:
            y.fill_(9)
        ws.fill_(0xFF)
        graphs[0].replay()
        graphs[1].replay()
        torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want))


@pytest.mark.parametrize("T", [4, 40, 300])
def test_two_streams_at_once(m, T):
    g = torch.Generator().manual_seed(1)
    K, N = 1056, 264
    codes, scales, e = matrix(g, N, K, "nvfp4")
    f = m.fp4_desc(K, N, "nvfp4", torch.float32)
    xs = [torch.randn((T, K), generator=g).cuda() for _ in range(2)]
    ws = [torch.empty(m.moe_fp4_workspace_bytes(f, T, 0), dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = []
    for i in range(2):
        y = torch.empty((T, N), device="cuda")
        m.moe_fp4_apply(f, xs[i], K, T, codes, scales, e, False, None, 0, y, N, ws[0])
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty((T, N), device="cuda") for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for j in range(20):
        for i in range(2):
            m.moe_fp4_apply(f, xs[i], K, T, codes, scales, e, False, None, 0, got[i][j], N, ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
