"""4-bit quantisation and products at the ends of what their arguments allow:
the most rows, the longest strides, addresses without alignment, scale bytes
that no quantisation writes."""
import pytest
import torch

import serve_ref as ref
from test_gpu_fp4 import check_product, check_quant, m, matrix  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1 << 26, (1 << 26) + 5])
def test_quant_of_many_short_rows_with_exponents(m, rows):  # noqa: F811
    """64 threads a row: 2^26 rows are 2^32 threads, more than one launch may have. Every row as in a call of its part of
    the matrix, some of them against the definition."""
    c, dt = 16, torch.bfloat16
    x = torch.randn((rows, c), dtype=dt, device="cuda")
    x *= torch.exp2(torch.randint(-20, 20, (rows, 1), device="cuda").float()).to(dt)
    kinds = (c // 2, torch.uint8), (c // 16, torch.uint8), (1, torch.int8), (c, dt)

    def quant(v):
        codes, scales, e, val = (torch.full((v.shape[0], n), 77, dtype=t, device="cuda") for n, t in kinds)
        m.moe_fp4_quant(v, c, v.shape[0], c, dt, "nvfp4", m.MOE_SCALE_NEAREST, e, codes, scales, val, c)
        return codes, scales, e, val

    got, step = quant(x), 1 << 23
    for at in range(0, rows, step):
        part = x[at:at + step]
        assert all(torch.equal(a[at:at + step], b) for a, b in zip(got, quant(part)))
    pick = torch.tensor([0, (1 << 25) - 1, 1 << 25, (1 << 25) + 1, rows - 2, rows - 1], device="cuda")
    codes0, scales0, e0, val = ref.quant(x[pick], "nvfp4", "nearest", True)
    for g, w in zip(got, (codes0, scales0, e0[:, None], ref.stored(val, dt))):
        assert torch.equal(g[pick].cpu(), w)


def call(m, f, back, rnd, x, T, w, base, y, ws):  # noqa: F811
    codes, scales, e = w
    ldb = 0 if base is None else base.stride(0)
    if back:
        m.moe_fp4_backward(f, x, x.stride(0), T, codes, scales, e, base, ldb, y, y.stride(0), ws)
    else:
        m.moe_fp4_apply(f, x, x.stride(0), T, codes, scales, e, rnd, base, ldb, y, y.stride(0), ws)


@pytest.mark.parametrize("T,K,N,fmt,dt,rnd,back", [
    (1, 544, 264, "nvfp4", "f32", False, False), (4, 544, 264, "mxfp4", "bf16", True, False),
    (20, 544, 264, "nvfp4", "bf16", False, False), (20, 544, 264, "mxfp4", "f32", False, False), (64, 544, 264, "mxfp4", "bf16", True, False),
    (65, 544, 264, "nvfp4", "f32", False, False), (300, 544, 264, "mxfp4", "bf16", True, False), (130, 5600, 72, "mxfp4", "f16", False, False),
    (1, 544, 264, "nvfp4", "f32", False, True), (300, 544, 264, "mxfp4", "bf16", False, True)])
def test_workspace_of_exactly_the_size(m, T, K, N, fmt, dt, rnd, back):  # noqa: F811
    """Nothing behind the size asked for is written, nor the first 4096 bytes of the workspace."""
    t = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dt]
    g = torch.Generator().manual_seed(T)
    f = m.fp4_desc(K, N, fmt, t)
    need = m.moe_fp4_workspace_bytes(f, T, back)
    buf = torch.randint(0, 256, (need + (1 << 20),), dtype=torch.uint8, generator=g).cuda()
    keep = buf.clone()
    x = torch.randn((T, N if back else K), generator=g).to(t).cuda()
    y = torch.empty((T, K if back else N), dtype=t, device="cuda")
    call(m, f, back, rnd, x, T, matrix(g, N, K, fmt), None, y, buf[:need])
    assert torch.equal(buf[need:], keep[need:])
    assert torch.equal(buf[:4096], keep[:4096])


def workspace(m, f, T, back):  # noqa: F811
    return torch.full((m.moe_fp4_workspace_bytes(f, T, back),), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("T", [2, 20, 50, 200])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_nan_scale_beside_rounded_activations(m, T, dt):  # noqa: F811
    """A NaN scale of W makes the outputs NaN that its block enters, whatever it meets (here also a block of zeros)."""
    g = torch.Generator().manual_seed(9)
    K, N, t = 160, 72, {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dt]
    codes, scales, _ = matrix(g, N, K, "mxfp4")
    scales[5, 1] = 0xFF
    codes[5, 16:32] = 0
    x = torch.randn((T, K), generator=g).to(t).cuda()
    x[1, 32:64] = 0
    y = torch.empty((T, N), dtype=t, device="cuda")
    f = m.fp4_desc(K, N, "mxfp4", t)
    call(m, f, False, True, x, T, (codes, scales, None), None, y, workspace(m, f, T, False))
    hit = torch.arange(N, device="cuda") == 5
    assert y[:, hit].isnan().all() and y[:, ~hit].isfinite().all()


@pytest.mark.parametrize("T", [2, 20, 50, 200])
def test_weights_above_fp32_beside_rounded_activations(m, T):  # noqa: F811
    """Scale byte 254 (2^127): codes of 2 and more stand for values above the largest fp32: their outputs are
    infinite or NaN or the definition's, the others as always."""
    g = torch.Generator().manual_seed(7)
    K, N = 96, 40
    codes, scales, _ = matrix(g, N, K, "mxfp4")
    scales[5, 1] = 254
    codes[5, 16:32] = 0x77  # 6 2^127
    x = torch.randn((T, K), generator=g) * 2.0 ** -20
    y = torch.empty((T, N), device="cuda")
    f = m.fp4_desc(K, N, "mxfp4", torch.float32)
    call(m, f, False, True, x.cuda(), T, (codes, scales, None), None, y, workspace(m, f, T, False))
    W = ref.decode(codes, scales, "mxfp4")
    want, off = ref.product(ref.quant(x, "mxfp4", "floor", False)[3], W, None, torch.float32)
    y = y.cpu()
    hit = torch.arange(N) == 5
    as_it_is = (y[:, 5].double() - want[:, 5]).abs() <= off[:, 5]
    assert (as_it_is | ~y[:, 5].isfinite()).all()
    ref.close(y[:, ~hit], want[:, ~hit], off[:, ~hit], "other outputs")


@pytest.mark.parametrize("T,K,N,fmt,dt,rnd,back", [
    (4, 544, 264, "nvfp4", "f32", False, False), (3, 96, 40, "mxfp4", "bf16", True, False),
    (64, 544, 264, "nvfp4", "bf16", False, False), (64, 544, 264, "mxfp4", "f32", False, False), (61, 544, 264, "mxfp4", "f16", True, False),
    (300, 544, 264, "nvfp4", "f16", False, False), (257, 96, 40, "nvfp4", "f32", False, False), (300, 544, 264, "mxfp4", "bf16", True, False),
    (300, 544, 264, "mxfp4", "bf16", False, True), (260, 544, 264, "nvfp4", "f32", False, True),
    (300, 128, 24600, "mxfp4", "bf16", False, False), (300, 24608, 128, "mxfp4", "bf16", False, True)])
def test_longest_strides(m, T, K, N, fmt, dt, rnd, back):  # noqa: F811
    """Rows 2^22 elements apart on every side: the last row of a tile of 256 lies 2^31 bytes less 8 MiB (16-bit values)
    behind its first, or its parts do. Bit for bit as with rows side by side."""
    t, ld = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dt], 1 << 22
    ki, ko = (N, K) if back else (K, N)
    g = torch.Generator().manual_seed(T + K + N)
    w = matrix(g, N, K, fmt)
    f = m.fp4_desc(K, N, fmt, t)
    ws = workspace(m, f, T, back)
    x, base, y = torch.randn((T, ki), generator=g).to(t).cuda(), torch.randn((T, ko), generator=g).to(t).cuda(), torch.empty((T, ko), dtype=t, device="cuda")
    call(m, f, back, rnd, x, T, w, base, y, ws)
    far = []
    for v in (x, base, y):
        buf = torch.empty((T - 1) * ld + v.shape[1], dtype=t, device="cuda")
        far.append(buf.as_strided(v.shape, (ld, 1)))
    far[0].copy_(x)
    far[1].copy_(base)
    call(m, f, back, rnd, far[0], T, w, far[1], far[2], ws)
    assert torch.equal(far[2], y)


@pytest.mark.parametrize("fmt,rule,rows", [("nvfp4", "nearest", True), ("nvfp4", "nearest", False), ("mxfp4", "floor", False)])
def test_quant_of_rows_past_31_bits(m, fmt, rule, rows):  # noqa: F811
    """Rows whose offsets pass 2^31 elements, on both sides."""
    c, ld = 96, (1 << 30) + 8
    buf = torch.empty(2 * ld + c, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, c), (ld, 1))
    x.copy_(torch.randn((3, c), device="cuda"))
    check_quant(m, x, fmt, rule, rows, inplace=True)


@pytest.mark.parametrize("fmt,rnd,back", [("nvfp4", False, False), ("mxfp4", False, False), ("mxfp4", True, False), ("nvfp4", False, True),
                                          ("mxfp4", False, True)])
@pytest.mark.parametrize("T", [1, 20, 50, 200])
def test_scales_at_odd_addresses(m, T, fmt, rnd, back):  # noqa: F811
    """Scale bytes may lie anywhere: bit for bit as from an aligned address; and a quantisation writes them there."""
    g = torch.Generator().manual_seed(T)
    K, N = 544, 264
    codes, scales, e = matrix(g, N, K, fmt)
    odd = torch.full((scales.numel() + 2,), 0xAB, dtype=torch.uint8, device="cuda")[1:-1].view(scales.shape)
    assert odd.data_ptr() % 2 == 1
    odd.copy_(scales)
    f = m.fp4_desc(K, N, fmt, torch.bfloat16)
    ws = workspace(m, f, T, back)
    x = torch.randn((T, N if back else K), generator=g).bfloat16().cuda()
    y = [torch.empty((T, K if back else N), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for s, o in ((scales, y[0]), (odd, y[1])):
        call(m, f, back, rnd, x, T, (codes, s, e), None, o, ws)
    assert torch.equal(*y)
    v = torch.randn((N, K), generator=g).cuda()
    rule = m.MOE_SCALE_NEAREST if fmt == "nvfp4" else m.MOE_SCALE_FLOOR
    for s in (scales, odd):
        m.moe_fp4_quant(v, K, N, K, v.dtype, fmt, rule, None, None, s, None, 0)
    assert torch.equal(odd, scales)


@pytest.mark.parametrize("T", [2, 20, 50, 200])
def test_far_scales_beside_rounded_activations(m, T):  # noqa: F811
    """Scale bytes from 2^-127 up to where fp32 still holds the values."""
    g = torch.Generator().manual_seed(5)
    K, N = 96, 40
    for lo, hi, p in ((0, 6, 100), (118, 137, 0), (240, 247, -10)):
        x = torch.randn((T, K), generator=g) * 2.0 ** p
        check_product(m, T, K, N, "mxfp4", "f32", True, w=matrix(g, N, K, "mxfp4", lo, hi), x=x, base="none")


@pytest.mark.parametrize("base", ["none", "same", "other"])
@pytest.mark.parametrize("fmt,dt,rnd,back", [("nvfp4", "f16", False, False), ("nvfp4", "f32", False, False), ("mxfp4", "bf16", True, False),
                                             ("mxfp4", "f32", False, True), ("nvfp4", "bf16", False, True)])
def test_whole_tiles_of_128(m, fmt, dt, rnd, back, base):  # noqa: F811
    """20 x 21 tiles of 128 x 128 with ragged edges, 110 of 256 x 256: each workgroup writes its tile itself, with row
    exponents and base."""
    T, ki, ko = 2451, 544, 2568
    if back:
        check_product(m, T, ko + 24, ki, fmt, dt, back=True, base=base)
    else:
        check_product(m, T, ki, ko, fmt, dt, rnd, base=base)


@pytest.mark.parametrize("T,K,N,fmt,dt,rnd,back", [
    (1, 65536, 65536, "nvfp4", "f32", False, False), (17, 65536, 65536, "nvfp4", "bf16", False, False), (40, 65536, 65536, "mxfp4", "bf16", True, False),
    (65, 65536, 65536, "nvfp4", "f32", False, False), (70, 65536, 65536, "mxfp4", "bf16", True, False),
    (2, 65536, 65536, "nvfp4", "f32", False, True), (90, 65536, 65536, "mxfp4", "f16", False, True),
    (1 << 20, 32, 8, "nvfp4", "f32", False, False), (1 << 20, 96, 40, "mxfp4", "bf16", True, False), (1 << 20, 32, 8, "mxfp4", "f16", False, True)])
def test_largest_sizes(m, T, K, N, fmt, dt, rnd, back):  # noqa: F811
    """The ends of every range: some tokens and outputs, the first and last among them, against the definition."""
    t = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dt]
    torch.manual_seed(T)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    lo, hi = (0x18, 0x39) if fmt == "nvfp4" else (114, 123)
    scales = torch.randint(lo, hi, (N, K // ref.GROUP[fmt]), dtype=torch.uint8, device="cuda")
    e = torch.randint(-9, 1, (N,), dtype=torch.int8, device="cuda") if fmt == "nvfp4" else None
    f = m.fp4_desc(K, N, fmt, t)
    ki, ko = (N, K) if back else (K, N)
    x, y = (torch.randn((T, ki), device="cuda") / 16).to(t), torch.empty((T, ko), dtype=t, device="cuda")
    call(m, f, back, rnd, x, T, (codes, scales, e), None, y, workspace(m, f, T, back))
    rows = torch.tensor(sorted({0, 1, T // 2, T - 2, T - 1} & set(range(T))), device="cuda")
    xv = x[rows].cpu()
    xv = ref.quant(xv, "mxfp4", "floor", False)[3] if rnd else xv.double()
    G = ref.GROUP[fmt]
    if back:  # whole groups of columns
        for c in (0, K - G):
            W = ref.decode(codes[:, c // 2:(c + G) // 2], scales[:, c // G:c // G + 1], fmt, e)
            want, off = ref.product(xv, W.t().contiguous(), None, t)
            ref.close(y[rows][:, c:c + G], want, off, (T, K, N, c))
    else:
        n = torch.tensor(sorted({0, 1, N // 2, N - 2, N - 1}), device="cuda")
        want, off = ref.product(xv, ref.decode(codes[n], scales[n], fmt, None if e is None else e[n]), None, t)
        ref.close(y[rows][:, n], want, off, (T, K, N))
