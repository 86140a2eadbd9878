"""Workspace sizes of the norms and the 4-bit products, on the CPU."""
import block_scaled_fp4_route_amd as m

F32, BF16, F16 = m.MOE_ACT_F32, m.MOE_ACT_BF16, m.MOE_ACT_F16


def test_norm_workspace_of_an_empty_batch():
    """Also T = 0 asks for some bytes: a buffer of the size asked for has an address."""
    for H in (8, 2560, 16384):
        assert m.moe_block_norm_workspace_bytes(m.norm_desc(H, BF16, BF16, BF16, "channel", 1.0, 1e-6), 0) >= 4096
