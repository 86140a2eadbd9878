"""The norms around a block: more tokens than the backward pass has workgroups
for short rows, workspaces of exactly the size asked for, an empty batch."""
import pytest
import torch

from test_gpu_norm import check, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(9001, 264), (5003, 1032), (20011, 8)])
@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("acc", [False, True])
def test_many_tokens(m, T, H, gate, acc):  # noqa: F811
    """More than 512 workgroups, each with several rows."""
    check(m, T, H, ("bf16", "f32", "f32"), gate, mask="mixed", acc=acc)


@pytest.mark.parametrize("T", [1, 700, 9001])
def test_workspace_of_exactly_the_size(m, T):  # noqa: F811
    """Nothing behind the size asked for is written, nor the first 4096 bytes of the workspace."""
    H = 264
    g = torch.Generator().manual_seed(T)
    n = m.norm_desc(H, torch.float32, torch.float32, torch.float32, "channel", 1.0, 1e-6)
    need = m.moe_block_norm_workspace_bytes(n, T)
    buf = torch.randint(0, 256, (need + (1 << 20),), dtype=torch.uint8, generator=g).cuda()
    keep = buf.clone()
    r, y, dx = (torch.randn((T, H), generator=g).cuda() for _ in range(3))
    w = torch.ones(H, device="cuda")
    dr, dy = torch.empty_like(r), torch.empty_like(y)
    out = [torch.empty(H, device="cuda") for _ in range(3)]
    m.moe_block_norm_backward(n, r, H, y, H, T, None, w, w, w, None, 0, dx, H, dr, H, dy, H, *out, 0, buf[:need])
    assert torch.equal(buf[need:], keep[need:])
    assert torch.equal(buf[:4096], keep[:4096])


def test_no_tokens_and_a_workspace_of_the_size_asked_for(m):  # noqa: F811
    """An empty batch writes zeros with the workspace that its size asks for."""
    H = 64
    n = m.norm_desc(H, torch.float32, torch.float32, torch.float32, "channel", 1.0, 1e-6)
    w = torch.ones(H, device="cuda")
    out = [torch.full((H,), 5.0, device="cuda") for _ in range(3)]
    e = torch.empty((0, H), device="cuda")
    ws = torch.empty(m.moe_block_norm_workspace_bytes(n, 0), dtype=torch.uint8, device="cuda")
    m.moe_block_norm_backward(n, e, H, e, H, 0, None, w, w, w, None, 0, e, H, None, 0, None, 0, *out, 0, ws)
    assert all((o == 0).all() for o in out)


def test_most_tokens(m):  # noqa: F811
    """2^20 rows of 8 channels."""
    check(m, 1 << 20, 8, ("bf16", "f32", "f32"), "token", mask="mixed", pad=0)


@pytest.mark.parametrize("kinds", [("bf16", "f16", "f32"), ("f32", "bf16", "bf16"), ("f16", "f32", "bf16"), ("bf16", "bf16", "bf16")])
@pytest.mark.parametrize("H", [4104, 8192, 8200, 16384])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_long_rows(m, H, kinds, gate):  # noqa: F811
    """Rows above 4096 channels in each type, masked, several to a workgroup."""
    check(m, 601, H, kinds, gate, mask="mixed", acc=H % 512 != 0)


@pytest.mark.parametrize("gate", ["channel", "token"])
def test_masked_in_place(m, gate):  # noqa: F811
    """dr over dr_out: rows left out become zeros there too."""
    check(m, 65, 264, ("bf16", "f32", "f32"), gate, mask="mixed", inplace=True)
