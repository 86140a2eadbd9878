"""64-bit references of 4-bit quantisation and products, of the layer for a few
tokens and of the norms around a block, with the error that the kernels'
arithmetic may make beside each value. All on the CPU.

EPS = 2^-24 is the largest relative error of one fp32 rounding. A sum of n
terms in any order is off by at most (n + 2) EPS times the sum of their
magnitudes (each product rounded once, each partial sum at most n times, first
order); a stored 16-bit value adds half a step of its type."""
from __future__ import annotations

import torch

from learn_ref import EPS, HALF, TINY, close, cpu64  # noqa: F401

GROUP = {"nvfp4": 16, "mxfp4": 32}
MAGS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def two(e):
    """2^e in fp64 for whole e, exactly."""
    return torch.ldexp(torch.ones((), dtype=torch.float64), torch.as_tensor(e).to(torch.int64))


def e4m3(b):
    b = b.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * two(e - 7))
    v = torch.where(b & 0x7F == 0x7F, torch.full_like(v, float("nan")), v)
    return torch.where(b >= 128, -v, v)


def ue8m0(b):
    b = b.to(torch.int64)
    return torch.where(b == 255, torch.full(b.shape, float("nan"), dtype=torch.float64), two(b - 127))


def decode(codes, scales, fmt, row_exp=None):
    """codes [rows][cols / 2], scales [rows][cols / G] (uint8) -> fp64 [rows][cols]."""
    codes, scales = codes.cpu(), scales.cpu()
    n = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(codes.shape[0], -1).to(torch.int64)
    v = MAGS[n & 7] * torch.where(n >= 8, -1.0, 1.0)
    v = v * (e4m3 if fmt == "nvfp4" else ue8m0)(scales).repeat_interleave(GROUP[fmt], dim=1)
    return v if row_exp is None else v * two(row_exp.cpu())[:, None]


def _nearest_code(t):
    """t >= 0 -> the code of the nearest magnitude, ties to the even code."""
    d = (t.clamp(max=8)[..., None] - MAGS).abs()  # far above 6, fp64 would see all distances alike
    even, odd = d[..., 0::2].min(-1), d[..., 1::2].min(-1)
    return torch.where(even.values <= odd.values, 2 * even.indices, 2 * odd.indices + 1)


def quant(x, fmt, rule, rows):
    """x (any dtype) [r][c] -> codes, scales (uint8), row exponents (rows: wanted) and values in fp64.
    rule: "nearest" (nvfp4), "floor" or "ceil" (mxfp4)."""
    v = cpu64(x)
    r, c = v.shape
    G = GROUP[fmt]
    fine = v.isfinite()
    e = torch.zeros(r, dtype=torch.int64)
    if rows:
        top = torch.where(fine, v, torch.zeros_like(v)).abs().amax(1)
        m, p = torch.frexp(top / 2688)  # m 2^p, m in [0.5, 1): the next power of two is 2^p but for m = 0.5
        e = torch.where(top == 0, 0, (p - (m == 0.5).int()).clamp(-100, 116)).to(torch.int64)
    b = (v * two(-e)[:, None]).view(r, c // G, G)
    bad = ~fine.view(r, c // G, G).all(-1)
    top = torch.where(bad, torch.zeros(()).double(), b.abs().amax(-1))
    if fmt == "nvfp4":
        grid = e4m3(torch.arange(127))
        want = top / 6
        up = torch.searchsorted(grid, want).clamp(max=126)
        lo = (up - 1).clamp(min=0)
        a, z = want - grid[lo], grid[up] - want
        byte = torch.where((a < z) | ((a == z) & (lo % 2 == 0)), lo, up)
        s = grid[byte]
        byte = torch.where(bad, 0x7F, byte)
    else:
        m, p = torch.frexp(top)
        X = p - 3 + ((m > 0.75).int() if rule == "ceil" else 0)
        X = X.clamp(-127, 125).to(torch.int64)
        s = two(X)
        byte = torch.where(bad, 255, torch.where(top == 0, 0, X + 127))
    code = _nearest_code(torch.where(s > 0, b.abs().nan_to_num(0, 0, 0).permute(2, 0, 1) / s.clamp(min=2.0 ** -140), 0.0).permute(1, 2, 0))
    code = torch.where((s > 0)[..., None] & ~bad[..., None], code, 0)
    neg = torch.signbit(cpu64(x)).view(r, c // G, G) & ~bad[..., None]
    val = MAGS[code] * torch.where(neg, -1.0, 1.0) * s[..., None] * two(e)[:, None, None]
    val = torch.where(bad[..., None], torch.full_like(val, float("nan")), val).view(r, c)
    n = (code + 8 * neg.int()).view(r, c).to(torch.uint8)
    return n[:, 0::2] | (n[:, 1::2] << 4), byte.to(torch.uint8), e.to(torch.int8), val


def stored(v, dt):
    """fp64 values as moe_fp4_quant stores them in dt."""
    top = torch.finfo(dt).max
    return v.clamp(-top, top).to(dt) if dt == torch.float16 else v.to(torch.float32).to(dt)


def product(x, w, base, dt):
    """x [T][K] fp64 times w [N][K] fp64, and the bound of one fp32 sum of at most 3 K exact products of
    parts, rounded once to dt."""
    y = x @ w.t()
    off = (3 * x.shape[1] + 2) * EPS * (x.abs() @ w.t().abs())
    if base is not None:
        y = y + cpu64(base)
        off = off + EPS * y.abs()
    return y, off * (1 + HALF[dt]) + HALF[dt] * y.abs() + TINY[dt]


# ---- the layer ----

def layer(x, mats, shared, idx, w):
    """x [T][H] fp64; mats[e] = (gate, up, down) fp64; idx, w [T][k]: y and the bound.

    Products of 4-bit weights with fp32 values taken as parts are exact to 2^-22 of each product, and
    2^-39 of the row's largest value (parts of fp16 under one power of two); three bf16 parts are exact.
    A sum of up to 3 K such products: (3 K + 2) EPS + 3 2^-22 of the magnitudes. Below fp32's normal range
    a result is off by half its smallest step, 2^-150, at most, whatever its size."""
    T, H = x.shape
    y, off = torch.zeros((T, H), dtype=torch.float64), torch.zeros((T, H), dtype=torch.float64)

    def dot(m, v, ev):
        K = m.shape[1]
        out, mag = m @ v, m.abs() @ v.abs()
        return out, ((3 * K + 2) * EPS + 3 * 2.0 ** -22) * mag + 2.0 ** -39 * v.abs().max() * m.abs().sum(1) + m.abs() @ ev + 3 * K * 2.0 ** -149

    def ffn(g, u, d, v):
        zero = torch.zeros_like(v)
        a, ea = dot(g, v, zero)
        b, eb = dot(u, v, zero)
        sg = torch.sigmoid(a)
        h = a * sg * b
        slope = (sg * (1 + a * (1 - sg))).abs()  # of silu
        # silu in fp32: expf, an addition, a division and two products, each a few roundings; an e^-a that
        # overflows leaves 0 for a value below 1e-36
        eh = slope * ea * b.abs() + (a * sg).abs() * eb + ea * eb + 16 * EPS * h.abs() * (1 + a.abs() * EPS) + 1e-36 * b.abs() + 2.0 ** -148
        return dot(d, h, eh)

    for t in range(T):
        for j in range(idx.shape[1]):
            v, e = ffn(*mats[int(idx[t, j])], x[t])
            wt = float(w[t, j])
            y[t] += wt * v
            off[t] += abs(wt) * e + 4 * EPS * abs(wt) * v.abs()
        if shared is not None:
            v, e = ffn(*shared, x[t])
            y[t] += v
            off[t] += e
        off[t] += (idx.shape[1] + 2) * EPS * y[t].abs()
    return y, off


# ---- the norms ----

def norm_forward(r, y, post, gate, pre, scale, eps, gate_kind):
    """All fp64. s, x (None without pre) and their bounds before a rounding to 16 bits."""
    H = r.shape[1]
    es = torch.zeros_like(r)
    s = r
    if y is not None:
        g = scale * _gate(gate, gate_kind)
        v, rel = y, 0.0
        if post is not None:
            v = y / ((y * y).mean(1, keepdim=True) + eps).sqrt() * post
            rel = (H + 2) / 2 * EPS + 4 * EPS  # of the root of a sum of squares, the root, the reciprocal
        s = r + g * v
        es = (rel + 4 * EPS) * (g * v).abs() + EPS * (s.abs() + r.abs())
    if pre is None:
        return s, es, None, None
    ms = (s * s).mean(1, keepdim=True) + eps
    x = s / ms.sqrt() * pre
    rel = (H + 2) / 2 * EPS + 6 * EPS + (s.abs() * es).mean(1, keepdim=True) / ms
    return s, es, x, rel * x.abs() + es * (pre.abs() / ms.sqrt())


def _gate(gate, kind):
    if kind == "none":
        return 1.0
    return gate[None, :] if kind == "channel" else gate[:, None]


def norm_backward(r, y, post, gate, pre, dr_out, dx, scale, eps, gate_kind):
    """All fp64 (None where absent). {name: (value, bound)} of dr, dy, dpost, dgate, dpre."""
    T, H = r.shape
    out = {}
    root = (H + 2) / 2 * EPS + 4 * EPS
    d = torch.zeros_like(r) if dr_out is None else dr_out
    ed = torch.zeros_like(r)
    if dx is not None:
        S = ((r * r).mean(1, keepdim=True) + eps).sqrt()
        n, a = r / S, dx * pre
        m = (a * n).mean(1, keepdim=True)
        em = ((H + 4) * EPS + root) * (a * n).abs().mean(1, keepdim=True)
        d = d + (a - n * m) / S
        ed = (n.abs() * em + (2 * root + 4 * EPS) * (n * m).abs() + 2 * EPS * a.abs()) / S + (root + 4 * EPS) * ((a - n * m) / S).abs() + EPS * d.abs()
        p = dx * n
        out["dpre"] = (p.sum(0), (T + 4) * EPS * p.abs().sum(0) + root * p.abs().sum(0))
    out["dr"] = (d, ed)
    if y is None:
        return out
    g = scale * _gate(gate, gate_kind)
    if post is not None:
        Y = ((y * y).mean(1, keepdim=True) + eps).sqrt()
        q, p, rel = y / Y, post, root
    else:
        Y, q, p, rel = torch.ones((T, 1), dtype=torch.float64), y, torch.ones(H, dtype=torch.float64), 0.0
    u = g * d
    eu = (g.abs() if torch.is_tensor(g) else abs(g)) * ed + 3 * EPS * u.abs()
    if post is not None:
        out["dpost"] = ((u * q).sum(0), (eu * q.abs() + (rel + (T + 4) * EPS) * (u * q).abs()).sum(0))
    dq = scale * d * q * p
    edq = abs(scale) * ed * (q * p).abs() + (rel + 6 * EPS) * dq.abs()
    if gate_kind == "channel":
        out["dgate"] = (dq.sum(0), (edq + (T + 2) * EPS * dq.abs()).sum(0))
    elif gate_kind == "token":
        out["dgate"] = (dq.sum(1), (edq + (H + 2) * EPS * dq.abs()).sum(1))
    if post is not None:
        b = u * p
        eb = eu * p.abs() + EPS * b.abs()
        m = (b * q).mean(1, keepdim=True)
        em = (eb * q.abs()).mean(1, keepdim=True) + ((H + 6) * EPS + 2 * rel) * (b * q).abs().mean(1, keepdim=True)
        dy = (b - q * m) / Y
        out["dy"] = (dy, (eb + q.abs() * em + (rel + 4 * EPS) * (q * m).abs() + EPS * b.abs()) / Y + (rel + 4 * EPS) * dy.abs())
    else:
        out["dy"] = (u, eu)
    return out


def rounded(ref, off, dt):
    """A value and its bound after one rounding to dt."""
    return ref, off * (1 + HALF[dt]) + HALF[dt] * ref.abs() + TINY[dt]
