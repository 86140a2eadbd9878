"""4-bit quantisation and products at the ends of what their arguments allow:
the most rows, the longest strides, addresses without alignment, scale bytes
that no quantisation writes."""
import pytest
import torch

import serve_ref as ref
from test_gpu_fp4 import m, matrix  # noqa: F401

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
