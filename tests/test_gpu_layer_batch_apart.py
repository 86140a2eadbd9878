"""Tokens of one call of the layer for a few tokens do not touch one another:
infinities and NaN in one token's x leave the others' results bit for bit."""
import pytest
import torch

from test_gpu_layer_batch import Case, grid, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,I", [("nvfp4", 96), ("nvfp4", 48), ("mxfp4", 96)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("T,E,k", [(2, 24, 4), (20, 24, 4), (50, 6, 2)])
def test_bad_values_of_one_token(m, T, E, k, I, bad, fmt):  # noqa: F811
    g = torch.Generator().manual_seed(T)
    x = grid(g, T, 512, step=1 / 256)
    x[1] = x[0]  # the same experts as a good token
    good = Case(m, T, 512, I, E, k, fmt, True, x=x).call()
    torch.cuda.synchronize()
    x2 = x.clone()
    x2[1, 5] = bad
    if T > 2:
        x2[7] = bad
    c = Case(m, T, 512, I, E, k, fmt, True, x=x2).call()
    torch.cuda.synchronize()
    on = [t for t in range(T) if t != 1 and (T == 2 or t != 7)]
    for a, b in ((good.y, c.y), (good.w, c.w), (good.idx, c.idx)):
        assert torch.equal(a[on], b[on])
    assert (c.idx[:T] >= 0).all() and (c.idx[:T] < E).all()
    if bad != 3e38:
        assert not c.y[1].isfinite().any()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("E,k", [(1024, 32), (700, 32), (32, 32)])
def test_most_tokens_and_choices(m, E, k, fmt):  # noqa: F811
    """64 tokens of 32 experts each, an empty slot among them: items of 5 and of 15 assignments."""
    Case(m, 64, 512, 32, E, k, fmt, True, (9,)).call().check()
