"""64-bit references of the router-training and adapter operators, with the
error that fp32 arithmetic may make beside each value.

EPS = 2^-24 is the largest relative error of one fp32 rounding. A sum of K
products in any order is off by at most (K + 2) EPS sum|a b| (each product
rounded once, each partial sum at most K times, first order); a stored 16-bit
value adds half a step of its type. All on the CPU."""
from __future__ import annotations

import torch

EPS = 2.0 ** -24
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
# the smallest step of a type: a value below its normal range is off by half of it
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def cpu64(t):
    return t.detach().cpu().double()


def close(got, ref, tol, what):
    """|got - ref| <= tol element by element; NaN and infinities where ref has them."""
    got, ref = cpu64(got), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = (got == ref) | (got.isnan() & ref.isnan())
    d = torch.where(same, torch.zeros_like(ref), (got - ref).abs())
    bad = ~(same | (d <= tol))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist(),
                           (d / tol)[bad].max().item())


def mm(a, b, ea=None, eb=None, pairs=False):
    """a @ b and what fp32 may be off by, with errors ea, eb already in the operands.

    pairs: the operands are sums of two fp16 parts h + l, scaled so that the
    largest of a row of a (a column of b) is in [2^14, 2^15). h rounds to
    2^-11 of the value and l to 2^-11 of what is left, so h + l is off by at
    most 2^-22 of it, or by half the smallest fp16 step, 2^-25, which is 2^-39
    of the largest at most; the product of the two l, 2^-22 of the product, is
    left out: 3 * 2^-22 of each product, and 2^-39 of the largest times the
    other operand. A product of three sums has 3 K terms to add."""
    K = a.shape[1]
    off = ((3 * K if pairs else K) + 2) * EPS * (a.abs() @ b.abs())
    if pairs:
        off = off + 3 * 2.0 ** -22 * (a.abs() @ b.abs())
        off = off + 2.0 ** -39 * (a.abs().amax(1, keepdim=True) * b.abs().sum(0, keepdim=True) +
                                  a.abs().sum(1, keepdim=True) * b.abs().amax(0, keepdim=True))
    if ea is not None:
        off = off + ea @ b.abs()
    if eb is not None:
        off = off + a.abs() @ eb
    return a @ b, off


# ---- balance loss ----

def balance(logits, idx, mask, off, k, cb, cz, up=1.0):
    """Values and bounds of loss, probs, dlogits; counts exactly. logits
    [T][E] fp32, mask bool [T], off a list of S + 1 offsets."""
    l = cpu64(logits)
    T, E = l.shape
    S = len(off) - 1
    counts = torch.zeros((S, E), dtype=torch.int64)
    probs, eprobs = torch.zeros((S, E), dtype=torch.float64), torch.zeros((S, E), dtype=torch.float64)
    grad, egrad = torch.zeros((T, E), dtype=torch.float64), torch.zeros((T, E), dtype=torch.float64)
    rows = [[t for t in range(off[s], off[s + 1]) if mask[t]] for s in range(S)]
    live, N = sum(len(r) > 0 for r in rows), sum(len(r) for r in rows)
    bal = ebal = z = ez = 0.0
    for s, r in enumerate(rows):
        if not r:
            continue
        v = l[r]
        top = v.amax(1, keepdim=True)
        dead = (top == -torch.inf)
        top = torch.where(dead, torch.zeros_like(top), top)
        ex = torch.exp(v - top)
        zz = ex.sum(1, keepdim=True)
        p = torch.where(zz == 0, torch.zeros_like(ex), ex / zz)
        lse = torch.where(zz == 0, torch.zeros_like(zz), top + torch.log(zz))
        # v - top rounds once (relative to its size, which is an absolute error
        # of the exponent), exp 2 units, the sum of E values E / 64 + 6 lanes'
        # roundings, the quotient and the product 3 more
        far = torch.where(p > 0, (v - top).abs(), torch.zeros_like(p)).amax(1, keepdim=True)
        rel = (2 * far + 4 + E / 64 + 6 + 4) * EPS
        n = len(r)
        hits = torch.bincount(idx[r].reshape(-1).cpu().long(), minlength=E)
        counts[s] = hits
        probs[s] = p.mean(0)
        depth = n + 8  # additions that a probability's sum passes at most
        eprobs[s] = (rel * p).mean(0) + depth * EPS * probs[s] + 2.0 ** -120
        f = hits.double() / (n * k)
        bal += float(E * (f * probs[s]).sum()) / live
        ebal += float(E * (f * (eprobs[s] + (E + S + 8) * EPS * probs[s])).sum()) / live
        elz = (lse.abs() + top.abs()) * 2 * EPS + rel + 4 * EPS  # of lse: log z and the sum with the maximum
        z += float((lse ** 2).sum())
        ez += float((2 * lse.abs() * elz + (n + 8) * EPS * lse ** 2).sum())
        c = cb * f * E / (live * n)
        dot = (p * c).sum(1, keepdim=True)
        zf = cz * 2 / N
        g = p * (c - dot + zf * lse)
        eg = p * (8 * EPS * c.abs() + (rel + (E / 64 + 10) * EPS) * (p * c.abs()).sum(1, keepdim=True) +
                  abs(zf) * (elz + 8 * EPS * lse.abs())) + (rel + 4 * EPS) * g.abs()
        if zf == 0:
            g, eg = p * (c - dot), p * (8 * EPS * c.abs() + (rel + (E / 64 + 10) * EPS) * (p * c.abs()).sum(1, keepdim=True)) + (rel + 4 * EPS) * (p * (c - dot)).abs()
        grad[r], egrad[r] = up * g, abs(up) * eg + 2.0 ** -120
    z, ez = (z / N, ez / N) if N else (0.0, 0.0)
    total = (cb * bal if cb else 0.0) + (cz * z if cz else 0.0)
    etotal = (abs(cb) * ebal if cb else 0.0) + (abs(cz) * ez if cz else 0.0) + 4 * EPS * (abs(cb * bal) + (abs(cz * z) if cz else 0.0))
    loss = torch.tensor([total, bal, z], dtype=torch.float64)
    eloss = torch.tensor([etotal, ebal + 4 * EPS * abs(bal), ez + 4 * EPS * abs(z)], dtype=torch.float64) + 2.0 ** -120
    return {"loss": (loss, eloss), "counts": counts, "probs": (probs, eprobs), "dlogits": (grad, egrad)}


# ---- routing gradient ----

def route_backward(x, Wr, idx, w, dw, mask, din, T, E, k):
    G, eG = torch.zeros((T, E), dtype=torch.float64), torch.zeros((T, E), dtype=torch.float64)
    if din is not None:
        G += cpu64(din)
    if dw is not None:
        w, dw = cpu64(w), cpu64(dw)
        dot = (w * dw).sum(1, keepdim=True)
        ds = w * (dw - dot)
        eds = w * ((k + 6) * EPS * (w * dw).abs().sum(1, keepdim=True) + 3 * EPS * dw.abs())
        at = idx.cpu().long()
        G.scatter_add_(1, at, ds)
        hits = torch.zeros_like(G).scatter_add_(1, at, torch.ones_like(ds))
        mag = G.abs() if din is None else cpu64(din).abs()
        mag = mag.scatter_add(1, at, ds.abs())
        eG.scatter_add_(1, at, eds)
        eG += hits * EPS * mag
    if mask is not None:
        off = ~mask
        G[off], eG[off] = 0.0, 0.0
    out = {"dlogits": (G, eG + 2.0 ** -140)}
    pairs = Wr is not None and T * E * Wr.shape[1] >= 1 << 29  # the sizes that multiply pairs of fp16 parts
    if Wr is not None:
        v, e = mm(G, cpu64(Wr), ea=eG, pairs=pairs)
        out["dx"] = (v, e + 2.0 ** -140)
    if x is not None:
        x = cpu64(x)
        if mask is not None:
            x[~mask] = 0.0
        v, e = mm(G.t().contiguous(), x, ea=eG.t().contiguous(), pairs=pairs)
        out["dWr"] = (v, e + 2.0 ** -140)
    return out


# ---- adapters ----

def _stored(v, e, dtype):
    """The value as stored in dtype, and the bound: half a step of the type at most."""
    return v, e + HALF[dtype] * (v.abs() + e) + TINY[dtype]


def lora(x, ids, A, B, scales, base, dtype, n):
    """A, B: lists of [r][K], [r][N]; x, base CPU or GPU tensors, base may be None."""
    T, N = x.shape[0], B[0].shape[1]
    y = torch.zeros((T, N), dtype=torch.float64) if base is None else cpu64(base)
    ey = torch.zeros_like(y)
    ids = ids.cpu()
    for a in range(n):
        rows = (ids == a).nonzero()[:, 0]
        if not len(rows) or not A[a].shape[0]:
            continue
        u, eu = mm(cpu64(x)[rows], cpu64(A[a]).t().contiguous())
        s = float(scales[a])
        u, eu = s * u, abs(s) * eu + 2 * EPS * (s * u).abs()
        v, ev = mm(u, cpu64(B[a]), ea=eu)
        ey[rows] += ev + EPS * (v.abs() + y[rows].abs())
        y[rows] += v
    y[ids >= n] = torch.nan
    return _stored(y, ey, dtype)


def lora_grads(x, dy, ids, A, B, scales, n):
    """dA, dB with bounds, per adapter."""
    ids, out = ids.cpu(), []
    for a in range(n):
        rows = (ids == a).nonzero()[:, 0]
        xr, dr = cpu64(x)[rows], cpu64(dy)[rows]
        s = float(scales[a])
        u, eu = mm(xr, cpu64(A[a]).t().contiguous())
        v, ev = mm(dr, cpu64(B[a]).t().contiguous())
        u, eu = s * u, abs(s) * eu + 2 * EPS * (s * u).abs()
        v, ev = s * v, abs(s) * ev + 2 * EPS * (s * v).abs()
        dA, eA = mm(v.t().contiguous(), xr, ea=ev.t().contiguous())
        dB, eB = mm(u.t().contiguous(), dr, ea=eu.t().contiguous())
        out.append(((dA, eA + 2.0 ** -140), (dB, eB + 2.0 ** -140)))
    return out
