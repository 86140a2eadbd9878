"""Workspace sizes of the norms and the 4-bit products, on the CPU."""
import block_scaled_fp4_route_amd as m

F32, BF16, F16 = m.MOE_ACT_F32, m.MOE_ACT_BF16, m.MOE_ACT_F16


def test_norm_workspace_of_an_empty_batch():
    """Also T = 0 asks for some bytes: a buffer of the size asked for has an address."""
    for H in (8, 2560, 16384):
        assert m.moe_block_norm_workspace_bytes(m.norm_desc(H, BF16, BF16, BF16, "channel", 1.0, 1e-6), 0) >= 4096


def test_product_workspace_of_few_tokens():
    """Nothing for a widened matrix where none is made: up to 64 tokens forward, the activations' parts or codes at most."""
    for fmt in ("nvfp4", "mxfp4"):
        for dt in (F32, BF16, F16):
            f = m.fp4_desc(2560, 8192, fmt, dt)
            assert m.moe_fp4_workspace_bytes(f, 1, 0) == m.moe_fp4_workspace_bytes(f, 4, 0) <= 4096
            for T in (5, 64):
                assert m.moe_fp4_workspace_bytes(f, T, 0) <= 4096 + 2 * 256 + T * 2560 * 6
            assert m.moe_fp4_workspace_bytes(f, 65, 0) >= 2 * 2560 * 8192 and m.moe_fp4_workspace_bytes(f, 1, 1) >= 2 * 2560 * 8192
