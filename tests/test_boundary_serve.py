"""Argument checks of the 4-bit, few-token and norm entry points, on the CPU:
every refusal has its documented status and launches nothing."""
import pytest

import block_scaled_fp4_route_amd as m
from test_boundary_learn import BIG, FAKE, ODD, OTHER, THIRD, status

FOURTH = 1 << 23
F32, BF16, F16 = m.MOE_ACT_F32, m.MOE_ACT_BF16, m.MOE_ACT_F16
NEAR, FLOOR, CEIL = m.MOE_SCALE_NEAREST, m.MOE_SCALE_FLOOR, m.MOE_SCALE_CEIL


def quant(x=FAKE, ldx=64, rows=3, cols=64, dtype=F32, fmt="mxfp4", rule=FLOOR, row_exp=None, codes=OTHER, scales=THIRD,
          values=None, ldv=0):
    return status(m.moe_fp4_quant, x, ldx, rows, cols, dtype, fmt, rule, row_exp, codes, scales, values, ldv, 0)


def test_quant_errors():
    A = m.MOE_ERR_ARG
    assert quant(fmt=7) == A
    assert quant(dtype=3) == A
    assert quant(rows=-1) == A
    assert quant(cols=0) == A and quant(cols=48) == A
    assert quant(rule=NEAR) == A and quant(fmt="nvfp4", rule=FLOOR) == A and quant(rule=9) == A
    assert quant(row_exp=FOURTH) == A                      # MXFP4 has no row exponents
    assert quant(codes=None, scales=None) == A             # no output
    assert quant(x=None) == A and quant(x=ODD) == A
    assert quant(ldx=60) == A and quant(ldx=68) == A
    assert quant(codes=OTHER + 2) == A
    assert quant(values=FOURTH, ldv=32) == A and quant(values=ODD, ldv=64) == A
    assert quant(values=FAKE, ldv=72) == A                 # in place with another stride
    assert quant(codes=FAKE) == A and quant(scales=OTHER) == A and quant(values=OTHER, ldv=64) == A
    assert quant(rows=1 << 28, cols=64) == m.MOE_ERR_UNSUPPORTED
    m.moe_fp4_quant(None, 0, 0, 64, F32, "mxfp4", FLOOR, None, OTHER, THIRD, None, 0, 0)  # no rows: nothing to do


FD = m.fp4_desc(64, 40, "nvfp4", BF16)


def apply(f=FD, x=FAKE, ldx=64, T=3, codes=OTHER, scales=THIRD, row_exp=None, round_x=False, base=None, ldb=0, y=FOURTH, ldy=40,
          ws=FAKE << 4, wsb=BIG):
    return status(m.moe_fp4_apply, f, x, ldx, T, codes, scales, row_exp, round_x, base, ldb, y, ldy, ws, wsb, 0)


def back(f=FD, dy=FAKE, lddy=40, T=3, codes=OTHER, scales=THIRD, row_exp=None, base=None, ldb=0, dx=FOURTH, lddx=64,
         ws=FAKE << 4, wsb=BIG):
    return status(m.moe_fp4_backward, f, dy, lddy, T, codes, scales, row_exp, base, ldb, dx, lddx, ws, wsb, 0)


@pytest.mark.parametrize("call,out", [(apply, "y"), (back, "dx")])
def test_product_errors(call, out):
    A, U = m.MOE_ERR_ARG, m.MOE_ERR_UNSUPPORTED
    for f in (m.fp4_desc(48, 40, "nvfp4", BF16), m.fp4_desc(64, 36, "nvfp4", BF16), m.fp4_desc(0, 40, "nvfp4", BF16),
              m.fp4_desc(64, 40, 5, BF16), m.fp4_desc(64, 40, "nvfp4", 4)):
        assert call(f=f) == A
    assert call(T=-1) == A
    assert call(f=m.fp4_desc(65536 + 32, 40, "nvfp4", BF16)) == U
    assert call(f=m.fp4_desc(64, 65536 + 8, "nvfp4", BF16)) == U
    assert call(T=(1 << 20) + 1) == U
    assert call(codes=None) == A and call(codes=OTHER + 8) == A and call(scales=None) == A
    assert call(f=m.fp4_desc(64, 40, "mxfp4", BF16), row_exp=FAKE) == A
    inp, ld = ("x", "ldx") if call is apply else ("dy", "lddy")
    assert call(**{inp: None}) == A and call(**{inp: ODD}) == A
    assert call(**{ld: 32}) == A and call(**{ld: 68}) == A and call(**{ld: (1 << 22) + 8}) == U
    assert call(**{out: None}) == A and call(**{out: ODD}) == A and call(**{"ld" + out: 32}) == A
    assert call(base=ODD, ldb=64) == A and call(base=FOURTH, ldb=128) == A
    assert call(**{out: FAKE}) == A and call(**{out: OTHER}) == A and call(**{out: THIRD}) == A
    need = m.moe_fp4_workspace_bytes(FD, 3, call is back)
    assert need > 0
    assert call(ws=None, wsb=0) == m.MOE_ERR_WORKSPACE
    assert call(ws=FAKE + 16) == m.MOE_ERR_WORKSPACE
    assert call(wsb=need - 1) == m.MOE_ERR_WORKSPACE


def test_product_corner_arguments():
    assert apply(round_x=True) == m.MOE_ERR_ARG            # only beside MXFP4
    m.moe_fp4_apply(FD, None, 0, 0, None, None, None, False, None, 0, None, 0, None, 0, 0)   # T = 0
    m.moe_fp4_backward(FD, None, 0, 0, None, None, None, None, 0, None, 0, None, 0, 0)
    assert m.moe_fp4_workspace_bytes(m.fp4_desc(48, 40, "nvfp4", BF16), 3, 0) == 0


def test_rounded_product_of_too_many_activations():
    """The quantisation counts its pieces in 32 bits: up to 2^33 elements."""
    for K, want in ((8192, m.MOE_ERR_WORKSPACE), (8224, m.MOE_ERR_UNSUPPORTED), (65536, m.MOE_ERR_UNSUPPORTED)):
        f = m.fp4_desc(K, 40, "mxfp4", BF16)
        assert apply(f=f, ldx=65536, T=1 << 20, round_x=True, ws=None, wsb=0) == want
        assert apply(f=f, ldx=65536, T=1 << 20, round_x=False, ws=None, wsb=0) == m.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("backward", [0, 1])
def test_product_workspace_never_falls(fmt, dtype, backward):
    f = m.fp4_desc(2560, 640, fmt, dtype)
    sizes = [m.moe_fp4_workspace_bytes(f, T, backward) for T in list(range(0, 700)) + [1000, 5000, 8191, 8192, 70000, 1 << 20]]
    assert all(b >= a for a, b in zip(sizes, sizes[1:]))


D = m.desc(2560, 640, 512, 10, "nvfp4")


def batch(d=D, x=FAKE, T=4, mask=None, Wr=FAKE, ptrs=FAKE, shared=None, y=OTHER, idx=THIRD, w=FOURTH, ws=FAKE << 4, wsb=BIG):
    return status(m.moe_layer_decode_batch, d, x, T, mask, Wr, ptrs, shared, y, idx, w, ws, wsb, 0)


def test_batch_errors():
    A, U = m.MOE_ERR_ARG, m.MOE_ERR_UNSUPPORTED
    assert batch(d=m.desc(2560, 640, 8, 9, "nvfp4")) == A
    assert batch(T=-1) == A
    assert batch(T=65) == U
    assert batch(d=m.desc(2560 + 256, 640, 512, 10, "nvfp4")) == U
    assert batch(d=m.desc(4096 + 512, 640, 512, 10, "nvfp4")) == U
    assert batch(d=m.desc(2560, 4096 + 16, 512, 10, "nvfp4")) == U
    assert batch(d=m.desc(2560, 640, 1025, 10, "nvfp4")) == U
    assert batch(d=m.desc(2560, 640, 512, 33, "nvfp4")) == U
    for name in ("x", "Wr", "ptrs", "y", "idx", "w"):
        assert batch(**{name: None}) == A, name
    assert batch(x=ODD) == A and batch(Wr=ODD) == A and batch(ptrs=FAKE + 2) == A
    assert batch(shared=(FAKE, None, FAKE)) == A and batch(shared=(FAKE, FAKE, ODD)) == A
    assert batch(y=FAKE) == A and batch(idx=OTHER) == A and batch(w=OTHER) == A and batch(w=THIRD) == A
    need = m.moe_workspace_bytes(D, 4, m.MOE_MODE_DECODE_BATCH)
    assert need > 0
    assert batch(ws=None, wsb=0) == m.MOE_ERR_WORKSPACE
    assert batch(ws=(FAKE << 4) + 16) == m.MOE_ERR_WORKSPACE
    assert batch(wsb=need - 1) == m.MOE_ERR_WORKSPACE
    m.moe_layer_decode_batch(D, None, 0, None, None, None, None, None, None, None, None, 0, 0)  # T = 0
    assert m.moe_workspace_bytes(D, 65, m.MOE_MODE_DECODE_BATCH) == 0


@pytest.mark.parametrize("d", [D, m.desc(4096, 2880, 384, 6, "mxfp4"), m.desc(512, 16, 1, 1, "nvfp4"), m.desc(4096, 4096, 1024, 32, "mxfp4")])
def test_batch_workspace_never_falls(d):
    sizes = [m.moe_workspace_bytes(d, T, m.MOE_MODE_DECODE_BATCH) for T in range(65)]
    assert all(b >= a for a, b in zip(sizes, sizes[1:]))


N = m.norm_desc(64, BF16, F32, F32, "none", 1.0, 1e-6)
NC = m.norm_desc(64, BF16, F32, F32, "channel", 1.0, 1e-6)
NT = m.norm_desc(64, BF16, F32, F32, "token", 1.0, 1e-6)
P = [i << 20 for i in range(1, 16)]


def fwd(n=N, r=P[0], ldr=64, y=P[1], ldy=64, T=3, mask=None, post=P[2], gate=None, pre=P[3], ro=P[4], ldro=64, x=P[5], ldx=64):
    return status(m.moe_block_norm, n, r, ldr, y, ldy, T, mask, post, gate, pre, ro, ldro, x, ldx, 0)


def bwd(n=N, r=P[0], ldr=64, y=P[1], ldy=64, T=3, mask=None, post=P[2], gate=None, pre=P[3], dro=P[4], lddro=64, dx=P[5], lddx=64,
        dr=P[6], lddr=64, dy=P[7], lddy=64, dpost=P[8], dgate=None, dpre=P[9], acc=0, ws=P[10], wsb=BIG):
    return status(m.moe_block_norm_backward, n, r, ldr, y, ldy, T, mask, post, gate, pre, dro, lddro, dx, lddx, dr, lddr, dy, lddy,
                  dpost, dgate, dpre, acc, ws, wsb, 0)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_norm_errors(call):
    A, U = m.MOE_ERR_ARG, m.MOE_ERR_UNSUPPORTED
    for n in (m.norm_desc(60, BF16, F32, F32, "none", 1.0, 1e-6), m.norm_desc(0, BF16, F32, F32, "none", 1.0, 1e-6),
              m.norm_desc(64, 3, F32, F32, "none", 1.0, 1e-6), m.norm_desc(64, BF16, 3, F32, "none", 1.0, 1e-6),
              m.norm_desc(64, BF16, F32, -1, "none", 1.0, 1e-6), m.norm_desc(64, BF16, F32, F32, 3, 1.0, 1e-6),
              m.norm_desc(64, BF16, F32, F32, "none", 1.0, 0.0), m.norm_desc(64, BF16, F32, F32, "none", 1.0, float("nan")),
              m.norm_desc(64, BF16, F32, F32, "none", float("inf"), 1e-6)):
        assert call(n=n) == A
    assert call(T=-1) == A
    assert call(n=m.norm_desc(16392, BF16, F32, F32, "none", 1.0, 1e-6)) == U
    assert call(T=(1 << 20) + 1) == U
    assert call(r=None) == A and call(r=ODD) == A and call(ldr=56) == A and call(ldr=68) == A
    assert call(y=ODD) == A and call(ldy=56) == A
    assert call(post=ODD) == A and call(pre=ODD) == A
    assert call(gate=P[11]) == A                           # MOE_GATE_NONE
    assert call(n=NC, gate=None) == A and call(n=NC, gate=P[11] + 4) == A and call(n=NT, gate=P[11] + 2) == A
    assert call(y=None) == A                               # post without y


def test_norm_forward_errors():
    A = m.MOE_ERR_ARG
    assert fwd(x=None) == A and fwd(pre=None) == A         # x and pre go together
    assert fwd(pre=None, x=None, ro=None) == A             # no output
    assert fwd(ro=ODD) == A and fwd(ldro=32) == A and fwd(x=ODD) == A and fwd(ldx=32) == A
    assert fwd(ro=P[0], ldro=72) == A                      # in place with another stride
    assert fwd(x=P[0]) == A and fwd(x=P[4]) == A and fwd(ro=P[1]) == A
    m.moe_block_norm(N, None, 0, None, 0, 0, None, None, None, FAKE, None, 0, OTHER, 0, 0)  # T = 0


def test_norm_backward_errors():
    A = m.MOE_ERR_ARG
    assert bwd(dr=None, dy=None, dpost=None, dpre=None) == A
    assert bwd(y=None, post=None, dpost=None) == A         # dy without y
    assert bwd(post=None) == A and bwd(pre=None) == A      # dpost, dpre without their vectors
    assert bwd(pre=None, dpre=None) == A                   # dx without pre
    assert bwd(dx=None) == A                               # dpre without dx
    assert bwd(dgate=P[12]) == A                           # no gate
    assert bwd(n=NC, gate=P[11], dgate=P[12] + 4) == A and bwd(n=NT, gate=P[11], dgate=P[12] + 2) == A
    assert bwd(dpost=ODD) == A and bwd(dpre=ODD) == A
    assert bwd(dro=ODD) == A and bwd(lddro=32) == A and bwd(dx=ODD) == A and bwd(dr=ODD) == A and bwd(dy=ODD) == A and bwd(lddy=8) == A
    assert bwd(dr=P[4], lddr=72) == A                      # in place with another stride
    assert bwd(dr=P[5]) == A and bwd(dy=P[1]) == A and bwd(dy=P[6]) == A and bwd(dpre=P[8]) == A and bwd(dpost=P[2]) == A
    need = m.moe_block_norm_workspace_bytes(N, 3)
    assert need > 0
    assert bwd(ws=None, wsb=0) == m.MOE_ERR_WORKSPACE
    assert bwd(ws=P[10] + 16) == m.MOE_ERR_WORKSPACE
    assert bwd(wsb=need - 1) == m.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("H", [8, 264, 2560, 16384])
def test_norm_workspace_never_falls(H):
    n = m.norm_desc(H, BF16, BF16, BF16, "channel", 1.0, 1e-6)
    sizes = [m.moe_block_norm_workspace_bytes(n, T) for T in list(range(0, 2000)) + [8191, 70000, 1 << 20]]
    assert all(b >= a for a, b in zip(sizes, sizes[1:]))
