"""The 64-bit references of the 4-bit and norm operators, on the CPU: against
torch's own conversions, autograd and differences."""
import pytest
import torch

import serve_ref as ref


def test_decoders_match_torch():
    b = torch.arange(256).to(torch.uint8)
    assert torch.equal(ref.e4m3(b).nan_to_num(1e9), b.view(torch.float8_e4m3fn).double().nan_to_num(1e9))
    assert torch.equal(ref.ue8m0(b)[1:255], b.view(torch.float8_e8m0fnu).float().double()[1:255])


@pytest.mark.parametrize("fmt,rule,rows", [("nvfp4", "nearest", True), ("nvfp4", "nearest", False), ("mxfp4", "floor", False), ("mxfp4", "ceil", False)])
def test_quant_is_nearest_and_decodes_to_its_values(fmt, rule, rows):
    g = torch.Generator().manual_seed(1)
    x = torch.randn((6, 96), generator=g) * torch.exp(2 * torch.randn((6, 1), generator=g))
    codes, scales, e, val = ref.quant(x, fmt, rule, rows)
    assert torch.equal(ref.decode(codes, scales, fmt, e), val)
    G = ref.GROUP[fmt]
    s = (val * 0 + 1).view(6, -1, G) * ((ref.e4m3 if fmt == "nvfp4" else ref.ue8m0)(scales) * ref.two(e)[:, None])[..., None]
    grid = torch.cat([-ref.MAGS, ref.MAGS])
    best = (x.double().view(6, -1, G, 1) - grid * s[..., None]).abs().amin(-1)
    assert torch.equal((x.double() - val).abs().view(6, -1, G), best)  # no other code is nearer
    if rule == "floor":  # what saturates is above 6 times the scale, below 8
        assert ((x.double().abs().view(6, -1, G) / s).amax() < 8)
    if rule == "ceil":
        assert ((x.double().abs().view(6, -1, G) / s).amax() <= 6)
    if rows:
        top = x.double().abs().amax(1) / ref.two(e)
        assert (top <= 2688).all() and (top > 1344).all()


def test_quant_hand_cases():
    x = torch.zeros((1, 32))
    x[0, :8] = torch.tensor([6.0, 5.0, 2.5, -0.25, 0.25, 0.75, 3.5, 1.25])  # ties to the even code
    codes, scales, _, val = ref.quant(x, "mxfp4", "floor", False)
    assert scales.tolist() == [[127]]
    assert val[0, :8].tolist() == [6, 4, 2, 0, 0, 1, 4, 1]
    assert codes[0, :4].tolist() == [0x67, 0x84, 0x20, 0x26]
    x = torch.zeros((1, 16))
    x[0, 0] = 6 * 1.0625  # the middle between the E4M3 values 1 and 1.125: to the even one
    assert ref.quant(x, "nvfp4", "nearest", False)[1].tolist() == [[0x38]]
    x[0, 0] = 6 * 1.1875
    assert ref.quant(x, "nvfp4", "nearest", False)[1].tolist() == [[0x3A]]


@pytest.mark.parametrize("gate_kind", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_norm_gradients_against_autograd_and_differences(gate_kind, post, pre):
    g = torch.Generator().manual_seed(2)

    def rnd(*s):
        return torch.randn(s, generator=g, dtype=torch.float64).requires_grad_()

    T, H, scale, eps = 3, 8, 0.75, 1e-3
    r, y = rnd(T, H), rnd(T, H)
    gate = {"none": None, "channel": rnd(H), "token": rnd(T)}[gate_kind]
    po, pr = (rnd(H) if post else None), (rnd(H) if pre else None)
    dr, dx = torch.randn((T, H), generator=g, dtype=torch.float64), torch.randn((T, H), generator=g, dtype=torch.float64)

    def fwd(r, y, *rest):
        rest = list(rest)
        ga = rest.pop(0) if gate is not None else None
        p1 = rest.pop(0) if post else None
        p2 = rest.pop(0) if pre else None
        s, _, x, _ = ref.norm_forward(r, y, p1, ga, p2, scale, eps, gate_kind)
        return (s, x) if pre else (s,)

    leaves = [t for t in (r, y, gate, po, pr) if t is not None]
    assert torch.autograd.gradcheck(fwd, leaves)  # autograd's against differences
    out = fwd(*leaves)
    (sum((o * d).sum() for o, d in zip(out, (dr, dx)))).backward()
    with torch.no_grad():
        s = out[0].detach()
        got = ref.norm_backward(s, y, po, gate, pr, dr, dx if pre else None, scale, eps, gate_kind)
    # dr is the gradient of r; the others are the leaves'
    for name, leaf in (("dr", r), ("dy", y), ("dgate", gate), ("dpost", po), ("dpre", pr)):
        if leaf is not None:
            assert torch.allclose(got[name][0], leaf.grad, rtol=1e-9, atol=1e-12), name
