"""Argument checks of the router-training and adapter entry points, on the
CPU: every refusal has its documented status and launches nothing."""
import pytest

import block_scaled_fp4_route_amd as m

FAKE = 1 << 20          # an aligned, never dereferenced address
OTHER = 1 << 21
THIRD = 3 << 20
ODD = FAKE + 4          # misaligned for 16-byte arguments
BIG = 1 << 42


def status(fn, *a):
    with pytest.raises(m.MoeError) as ei:
        fn(*a)
    return ei.value.status


D = m.desc(2560, 640, 512, 10, "nvfp4")


def balance(d=D, logits=FAKE, T=100, idx=FAKE, mask=None, off=None, S=1, cb=0.01, cz=0.0, dloss=None, loss=FAKE,
            counts=None, probs=None, dl=OTHER, ws=FAKE, wsb=BIG):
    return status(m.moe_balance_loss, d, logits, T, idx, mask, off, S, cb, cz, dloss, loss, counts, probs, dl, ws, wsb, 0)


def test_balance_errors():
    assert balance(d=m.desc(2560, 640, 8, 9, "nvfp4")) == m.MOE_ERR_ARG
    assert balance(T=-1) == m.MOE_ERR_ARG
    assert balance(S=0) == m.MOE_ERR_ARG
    assert balance(S=2) == m.MOE_ERR_ARG                  # several sequences without offsets
    assert balance(logits=None) == m.MOE_ERR_ARG
    assert balance(logits=ODD) == m.MOE_ERR_ARG
    assert balance(idx=None) == m.MOE_ERR_ARG
    assert balance(idx=FAKE + 2) == m.MOE_ERR_ARG
    assert balance(off=FAKE + 1) == m.MOE_ERR_ARG
    assert balance(dloss=FAKE + 1) == m.MOE_ERR_ARG
    assert balance(loss=None) == m.MOE_ERR_ARG
    assert balance(counts=FAKE + 1) == m.MOE_ERR_ARG
    assert balance(probs=FAKE + 1) == m.MOE_ERR_ARG
    assert balance(dl=ODD) == m.MOE_ERR_ARG
    assert balance(dl=FAKE) == m.MOE_ERR_ARG              # in place
    assert balance(cb=float("nan")) == m.MOE_ERR_ARG
    assert balance(cz=float("inf")) == m.MOE_ERR_ARG
    assert balance(d=m.desc(2560, 640, 1025, 10, "nvfp4")) == m.MOE_ERR_UNSUPPORTED
    assert balance(d=m.desc(2560, 640, 512, 33, "nvfp4")) == m.MOE_ERR_UNSUPPORTED
    assert balance(off=FAKE, S=65536) == m.MOE_ERR_UNSUPPORTED
    assert balance(T=(1 << 24) + 1) == m.MOE_ERR_UNSUPPORTED
    need = m.moe_balance_workspace_bytes(D, 100, 1)
    assert need > 0
    assert balance(ws=None, wsb=0) == m.MOE_ERR_WORKSPACE
    assert balance(ws=FAKE + 16) == m.MOE_ERR_WORKSPACE
    assert balance(wsb=need - 1) == m.MOE_ERR_WORKSPACE


def route_backward(d=D, x=FAKE, T=100, Wr=FAKE, idx=FAKE, w=FAKE, dw=FAKE, mask=None, din=FAKE, dout=None, dx=OTHER,
                   dWr=THIRD, acc=0, ws=FAKE, wsb=BIG):
    return status(m.moe_route_backward, d, x, T, Wr, idx, w, dw, mask, din, dout, dx, dWr, acc, ws, wsb, 0)


def test_route_backward_errors():
    assert route_backward(T=-1) == m.MOE_ERR_ARG
    assert route_backward(acc=4) == m.MOE_ERR_ARG
    assert route_backward(dw=None, din=None) == m.MOE_ERR_ARG
    assert route_backward(dx=None, dWr=None) == m.MOE_ERR_ARG
    assert route_backward(idx=None) == m.MOE_ERR_ARG
    assert route_backward(w=None) == m.MOE_ERR_ARG
    assert route_backward(din=FAKE + 2) == m.MOE_ERR_ARG
    assert route_backward(dout=FAKE + 2) == m.MOE_ERR_ARG
    assert route_backward(Wr=None) == m.MOE_ERR_ARG
    assert route_backward(x=None) == m.MOE_ERR_ARG
    assert route_backward(x=ODD) == m.MOE_ERR_ARG
    assert route_backward(Wr=ODD) == m.MOE_ERR_ARG
    assert route_backward(dx=ODD) == m.MOE_ERR_ARG
    assert route_backward(dWr=ODD) == m.MOE_ERR_ARG
    assert route_backward(d=m.desc(2560 + 128, 640, 512, 10, "nvfp4")) == m.MOE_ERR_UNSUPPORTED
    assert route_backward(d=m.desc(8192 + 256, 640, 512, 10, "nvfp4")) == m.MOE_ERR_UNSUPPORTED
    assert route_backward(T=(1 << 20) + 1) == m.MOE_ERR_UNSUPPORTED
    need = m.moe_route_backward_workspace_bytes(D, 100)
    assert need >= 100 * 512 * 4
    assert route_backward(ws=None, wsb=0) == m.MOE_ERR_WORKSPACE
    assert route_backward(wsb=need - 1) == m.MOE_ERR_WORKSPACE
    # outputs that are inputs, or each other
    own = dict(x=4 << 20, Wr=5 << 20, w=6 << 20, dw=7 << 20, din=8 << 20, dout=9 << 20)
    assert route_backward(**own, wsb=0) == m.MOE_ERR_WORKSPACE
    for out in ("dx", "dWr", "dout"):
        for name in ("x", "Wr", "w", "dw", "din"):
            if (out, name) != ("dout", "din"):
                assert route_backward(**{**own, out: own[name]}) == m.MOE_ERR_ARG, (out, name)
    assert route_backward(**{**own, "dout": own["din"]}, wsb=0) == m.MOE_ERR_WORKSPACE
    assert route_backward(dx=THIRD) == m.MOE_ERR_ARG
    assert route_backward(dout=OTHER) == m.MOE_ERR_ARG
    assert route_backward(dout=THIRD) == m.MOE_ERR_ARG


def test_fewer_tokens_never_need_more_workspace():
    """A workspace made for the longest batch serves the shorter ones."""
    Ts = [*range(0, 700), *range(700, 9000, 37), 8191, 8192, 8193, 16384, 32768, 40000, 1 << 17, 1 << 20]
    Ts.sort()
    for H, E in ((256, 8), (256, 1024), (1024, 64), (2560, 512), (4096, 384), (8192, 129)):
        d = m.desc(H, 64, E, 4, "nvfp4")
        sizes = [m.moe_route_backward_workspace_bytes(d, T) for T in Ts]
        assert sizes == sorted(sizes), (H, E)
        for S in (1, 7, 1000):
            sizes = [m.moe_balance_workspace_bytes(d, T, S) for T in Ts]
            assert sizes == sorted(sizes), (E, S)
    for K, N in ((256, 256), (2560, 8192), (4096, 2880), (8192, 512)):
        for n, R in ((1, 1), (4, 64), (8, 16), (300, 8), (2, 128)):
            for back in (False, True):
                sizes = [m.moe_lora_workspace_bytes(m.lora_desc(K, N, n, R, m.MOE_ACT_BF16), T, back) for T in Ts]
                assert sizes == sorted(sizes), (K, N, n, R, back)


L = m.lora_desc(2560, 8192, 4, 16, m.MOE_ACT_BF16)


def lora(l=L, x=FAKE, ldx=2560, T=100, ids=FAKE, a=FAKE, b=FAKE, ranks=FAKE, scales=FAKE, base=None, ldb=8192, y=OTHER,
         ldy=8192, ws=FAKE, wsb=BIG):
    return status(m.moe_lora_apply, l, x, ldx, T, ids, a, b, ranks, scales, base, ldb, y, ldy, ws, wsb, 0)


BAD_DESCS = [(0, 8192, 4, 16, 0), (2560, -8, 4, 16, 0), (2560, 8192, 0, 16, 0), (2560, 8192, 4, 0, 0),
             (2564, 8192, 4, 16, 0), (2560, 8190, 4, 16, 0), (2560, 8192, 4, 16, 3), (2560, 8192, 4, 16, -1)]
FAR_DESCS = [(65544, 8192, 4, 16, 0), (2560, 65544, 4, 16, 0), (2560, 8192, 1025, 16, 0), (2560, 8192, 4, 129, 0)]


def test_lora_errors():
    for bad in BAD_DESCS:
        assert lora(l=m.lora_desc(*bad)) == m.MOE_ERR_ARG
        assert m.moe_lora_workspace_bytes(m.lora_desc(*bad), 1, False) == 0
    for far in FAR_DESCS:
        assert lora(l=m.lora_desc(*far), ldx=1 << 17, ldy=1 << 17) == m.MOE_ERR_UNSUPPORTED
    assert lora(T=-1) == m.MOE_ERR_ARG
    assert lora(T=(1 << 20) + 1) == m.MOE_ERR_UNSUPPORTED
    for name in ("x", "ids", "a", "b", "ranks", "scales", "y"):
        assert lora(**{name: None}) == m.MOE_ERR_ARG, name
    for name in ("x", "a", "b", "y", "base"):
        assert lora(**{name: ODD}) == m.MOE_ERR_ARG, name
    assert lora(ldx=2552) == m.MOE_ERR_ARG                # shorter than a row
    assert lora(ldx=2564) == m.MOE_ERR_ARG                # not a multiple of 8
    assert lora(ldy=-8192) == m.MOE_ERR_ARG
    assert lora(base=FAKE, ldb=8184) == m.MOE_ERR_ARG
    assert lora(base=OTHER, ldb=8200) == m.MOE_ERR_ARG    # y itself, other rows
    assert lora(y=FAKE) == m.MOE_ERR_ARG                  # y is x
    for T in (1, 64, 65, 4096):
        need = m.moe_lora_workspace_bytes(L, T, False)
        assert need > 0 and lora(T=T, wsb=need - 1) == m.MOE_ERR_WORKSPACE
    assert lora(ws=None, wsb=0) == m.MOE_ERR_WORKSPACE
    assert lora(ws=FAKE + 16) == m.MOE_ERR_WORKSPACE
    m.moe_lora_apply(L, None, 0, 0, None, None, None, None, None, None, 0, None, 0, None, 0, 0)  # no tokens: nothing


def lora_backward(l=L, x=FAKE, ldx=2560, dy=FAKE, lddy=8192, T=100, ids=FAKE, a=FAKE, b=FAKE, ranks=FAKE, scales=FAKE,
                  dxb=None, lddxb=2560, dx=OTHER, lddx=2560, da=FAKE, db=OTHER, acc=0, ws=FAKE, wsb=BIG):
    return status(m.moe_lora_backward, l, x, ldx, dy, lddy, T, ids, a, b, ranks, scales, dxb, lddxb, dx, lddx, da, db,
                  acc, ws, wsb, 0)


def test_lora_backward_errors():
    for bad in BAD_DESCS:
        assert lora_backward(l=m.lora_desc(*bad)) == m.MOE_ERR_ARG
    for far in FAR_DESCS:
        assert lora_backward(l=m.lora_desc(*far)) == m.MOE_ERR_UNSUPPORTED
    assert lora_backward(T=-1) == m.MOE_ERR_ARG
    assert lora_backward(dx=None, da=None, db=None) == m.MOE_ERR_ARG
    for name in ("x", "dy", "ids", "a", "b", "ranks", "scales"):
        assert lora_backward(**{name: None}) == m.MOE_ERR_ARG, name
    for name in ("x", "dy", "dx", "dxb"):
        assert lora_backward(**{name: ODD}) == m.MOE_ERR_ARG, name
    assert lora_backward(da=FAKE + 4) == m.MOE_ERR_ARG
    assert lora_backward(db=FAKE + 4) == m.MOE_ERR_ARG
    assert lora_backward(lddy=8184) == m.MOE_ERR_ARG
    assert lora_backward(lddx=2564) == m.MOE_ERR_ARG
    assert lora_backward(dxb=OTHER, lddxb=2568) == m.MOE_ERR_ARG
    assert lora_backward(dx=FAKE) == m.MOE_ERR_ARG        # dx is an input
    assert lora_backward(db=FAKE) == m.MOE_ERR_ARG        # the tables of dA and dB are one
    need = m.moe_lora_workspace_bytes(L, 100, True)
    assert need > m.moe_lora_workspace_bytes(L, 100, False)
    assert lora_backward(wsb=need - 1) == m.MOE_ERR_WORKSPACE
    assert lora_backward(T=0, ranks=None) == m.MOE_ERR_ARG


def test_tensors_off_the_gpu_are_refused():
    import torch
    t = torch.zeros(64)
    assert status(m.moe_balance_loss, D, t, 1, t, None, None, 1, 1.0, 0.0, None, t, None, None, None, t, None, 0) == m.MOE_ERR_ARG


def test_descs_by_dtype():
    import torch
    assert m.lora_desc(8, 8, 1, 1, torch.float32).dtype == m.MOE_ACT_F32
    assert m.lora_desc(8, 8, 1, 1, torch.bfloat16).dtype == m.MOE_ACT_BF16
    assert m.lora_desc(8, 8, 1, 1, torch.float16).dtype == m.MOE_ACT_F16


def test_fp32_products_is_a_flag_of_its_own():
    assert m.MOE_FP32_PRODUCTS not in (m.MOE_ACC_DX, m.MOE_ACC_DWR, 4)
    for acc in range(4):  # accepted up to the workspace
        assert route_backward(acc=acc + m.MOE_FP32_PRODUCTS, wsb=0) == m.MOE_ERR_WORKSPACE
    assert route_backward(acc=2 * m.MOE_FP32_PRODUCTS) == m.MOE_ERR_ARG
    assert route_backward(acc=-1) == m.MOE_ERR_ARG
