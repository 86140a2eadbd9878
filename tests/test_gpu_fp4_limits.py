"""4-bit quantisation and products at the ends of what their arguments allow:
the most rows, the longest strides, addresses without alignment, scale bytes
that no quantisation writes."""
import pytest
import torch

import serve_ref as ref
from test_gpu_fp4 import m  # noqa: F401

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
