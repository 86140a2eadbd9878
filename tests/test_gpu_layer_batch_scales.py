"""The layer for a few tokens at the ends of the scales, with inputs whose
outputs fp32 can hold, against a bound of the batched kernels' own arithmetic:
an output of zeros, or one that lost its subnormal weights, is far outside."""
import pytest
import torch

import serve_ref as ref
from test_gpu_layer_batch import Case, grid, m, matrices, route  # noqa: F401

pytestmark = pytest.mark.gpu
EPS = ref.EPS


def dot(w, v, ev):
    """w v in fp32 from three bf16 parts of v, and its bound: the parts hold 24 bits (what they cut off lies below 2^-133), a
    product of two of at most 8 bits is exact, and a sum of 3 K of them in any order is off by (3 K + 2) EPS of the magnitudes, and
    by half the smallest step of fp32 for each addition below its normal range."""
    K = w.shape[1]
    return w @ v, (3 * K + 2) * EPS * (w.abs() @ v.abs()) + w.abs() @ (ev + 2.0 ** -133) + 3 * K * 2.0 ** -150


def layer(x, mats, shared, idx, w):
    """y and its bound, token by token."""
    y, off = torch.zeros(x.shape, dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64)

    def ffn(g, u, d, v):
        a, ea = dot(g, v, torch.zeros_like(v))
        b, eb = dot(u, v, torch.zeros_like(v))
        s = torch.sigmoid(a)
        h = a * s * b
        # silu's slope at most 1.1; expf (which takes a with all its bits), an addition, a division and a product, each a few
        # roundings; where e^-a overflows (a < -88) 0 stands for a value of at most 89 e^-88 < 1e-36 before the product with b
        eh = 1.1 * ea * (b.abs() + eb) + (a * s).abs() * eb + 16 * EPS * h.abs() + 1e-36 * b.abs() + 2.0 ** -148
        return dot(d, h, eh)

    for t in range(x.shape[0]):
        for j in range(idx.shape[1]):
            v, e = ffn(*mats[int(idx[t, j])], x[t])
            wt = float(w[t, j])
            y[t] += wt * v
            # a weight is a quotient of a sum of k exponentials, the product with it rounded once
            off[t] += wt * e + (idx.shape[1] + 24) * EPS * wt * v.abs()
        if shared is not None:
            v, e = ffn(*shared, x[t])
            y[t] += v
            off[t] += e
        off[t] += (idx.shape[1] + 2) * EPS * y[t].abs()
    return y, off


def run(m, T, H, I, E, k, fmt, shared, p, gate_up, down, seed=0):  # noqa: F811
    """x of about 2^p; scale bytes of gate and up, and of down, drawn from [lo, hi)."""
    g = torch.Generator().manual_seed(100 + T + seed)
    x, Wr = grid(g, T, H, step=1 / 256) * 2.0 ** p, grid(g, E, H, step=1 / 64) * 2.0 ** -p  # the logits are exact
    c = Case(m, T, H, I, E, k, fmt, shared, x=x, Wr=Wr)
    n, G = H * I, ref.GROUP[fmt]
    for at, rows, (lo, hi) in ((3 * n // 2, 2 * n // G, gate_up), (3 * n // 2 + 2 * n // G, n // G, down)):
        c.blocks[:, at:at + rows] = torch.randint(lo, hi, (E, rows), dtype=torch.uint8, generator=g)
    c.gb.copy_(c.blocks)
    c.call()
    idx, w = route(c.x, c.Wr, k)
    assert torch.equal(c.idx.cpu()[:T].long(), idx)
    mats = {int(e): matrices(c.blocks[int(e)], H, I, fmt) for e in idx.unique()}
    y, off = layer(c.x.double(), mats, [t.double() for t in c.sh] if shared else None, idx, w)
    top = y.abs().amax(1)
    assert (top > 2.0 ** -100).all() and (top < 2.0 ** 100).all()
    assert (off.amax(1) < 0.1 * top).all()  # zeros, or halves, are far outside
    ref.close(c.y[:T], y, off, "y")
    rel = ((ref.cpu64(c.y[:T]) - y).abs().amax(1) / top).max()
    assert rel <= 1e-5, rel  # the bar of the single-token decode is 1e-4


@pytest.mark.parametrize("T", [2, 3, 20, 50])
@pytest.mark.parametrize("gate_up,down,p", [
    ((0, 2), (121, 130), 100),     # subnormal bf16 weights in gate and up
    ((121, 130), (0, 2), 40),      # and in down
    ((40, 42), (121, 130), 70),
    ((121, 130), (40, 42), 30),
    ((240, 246), (121, 130), -110)])
def test_mxfp4_scales_at_the_ends(m, T, gate_up, down, p):  # noqa: F811
    run(m, T, 512, 64, 4, 2, "mxfp4", False, p, gate_up, down)


@pytest.mark.parametrize("T", [2, 3, 20, 50])
@pytest.mark.parametrize("gate_up,down,p", [
    ((0, 2), (0x18, 0x49), 0),     # 0 and the smallest E4M3 value
    ((0x18, 0x49), (0, 2), 0),
    ((1, 9), (1, 9), 0),
    ((0x7D, 0x7F), (0x7D, 0x7F), -4)])
def test_nvfp4_scales_at_the_ends(m, T, gate_up, down, p):  # noqa: F811
    run(m, T, 512, 64, 4, 2, "nvfp4", False, p, gate_up, down)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,H,I,E,k", [(2, 512, 96, 24, 4), (7, 1024, 160, 5, 5), (33, 512, 96, 24, 4), (64, 512, 32, 12, 3)])
def test_ordinary_scales(m, T, H, I, E, k, fmt):  # noqa: F811
    run(m, T, H, I, E, k, fmt, True, 0, *(2 * [(0x18, 0x49) if fmt == "nvfp4" else (121, 130)]))
