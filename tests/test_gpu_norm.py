"""The norms around a block on the GPU, forward and backward, against the
64-bit references of tests/serve_ref.py, element by element."""
import itertools

import pytest
import torch

import serve_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import block_scaled_fp4_route_amd as m
    return m


def rows(T, H, pad, dt, g, std=1.0):
    buf = torch.full((T + 1, H + pad), 3.0, dtype=dt, device="cuda")
    buf[:T, :H] = (torch.randn((T, H), generator=g) * std).to(dt).cuda()
    return buf[:T, :H], buf


def check(m, T, H, kinds=("f32", "f32", "f32"), gate="channel", y=True, post=True, pre=True, mask="none", pad=8, scale=0.75, eps=1e-5,
          dr_out=True, acc=False, inplace=False, ystd=20.0):
    g = torch.Generator().manual_seed(T * 13 + H)
    rt, yt, xt = (DT[k] for k in kinds)
    r, rbuf = rows(T, H, pad, rt, g, 2.0)
    yv = rows(T, H, 2 * pad, yt, g, ystd)[0] if y else None
    po = (1 + 0.2 * torch.randn(H, generator=g)).cuda() if y and post else None
    pr = (1 + 0.2 * torch.randn(H, generator=g)).cuda() if pre else None
    ga = None if gate == "none" else torch.randn(H if gate == "channel" else T, generator=g).cuda()
    mk = torch.ones(T, dtype=torch.bool)
    if mask == "tail":
        mk[T - T // 3:] = False
    elif mask == "all":
        mk[:] = False
    elif mask == "mixed":
        mk = torch.rand(T, generator=g) < 0.6
    if mask != "none":
        for v in (r, yv):
            if v is not None:
                v[~mk.cuda()] = float("nan")  # not read
    md = None if mask == "none" else mk.to(torch.uint8).cuda()
    n = m.norm_desc(H, rt, yt, xt, gate, scale, eps)
    r0 = r.clone()
    if inplace:
        ro, robuf = r, rbuf
    else:
        ro, robuf = rows(T, H, 3 * pad, rt, g)
    x, xbuf = rows(T, H, pad, xt, g) if pre else (None, None)
    before = [None if b is None else b.clone() for b in (robuf, xbuf)]
    ldy = 0 if yv is None else yv.stride(0)
    m.moe_block_norm(n, r, r.stride(0), yv, ldy, T, md, po, ga, pr, ro, ro.stride(0), x, x.stride(0) if pre else 0)
    torch.cuda.synchronize()
    w64 = lambda t: None if t is None else ref.cpu64(t)  # noqa: E731
    on = mk.nonzero()[:, 0]
    gsel = None if ga is None else w64(ga) if gate == "channel" else w64(ga)[on]
    s, es, xr, ex = ref.norm_forward(w64(r0)[on], None if yv is None else w64(yv)[on], w64(po), gsel, w64(pr), scale, eps, gate)
    ref.close(ro.cpu()[on], *ref.rounded(s, es, rt), "r_out")
    if pre:
        ref.close(x.cpu()[on], *ref.rounded(xr, ex, xt), "x")
    for b, now, outv in ((before[0], robuf, ro), (before[1], xbuf, x)):  # rows left out and all that lies beside
        if b is not None:
            same = (b == now) | (b.isnan() & now.isnan())
            same[:T, :H][mk.cuda()] = True
            assert same.all()
    # backward
    dro = rows(T, H, pad, rt, g, 0.1)[0] if dr_out else None
    dx = rows(T, H, 2 * pad, xt, g, 0.1)[0] if pre else None
    if mask != "none":
        for v in (dro, dx):
            if v is not None:
                v[~mk.cuda()] = float("inf")
    rin = ro.clone()
    rin[~mk.cuda()] = float("nan")
    dro0 = None if dro is None else dro.clone()
    dr, drb = (dro, None) if inplace and dr_out else rows(T, H, pad, rt, g)
    dy = rows(T, H, pad, yt, g)[0] if y else None
    old = {k: torch.randn(H if k != "dgate" or gate == "channel" else T, generator=g).cuda() for k in ("dpost", "dgate", "dpre")}
    got = {k: v.clone() for k, v in old.items()}
    ws = torch.full((m.moe_block_norm_workspace_bytes(n, T),), 0xFF, dtype=torch.uint8, device="cuda")
    m.moe_block_norm_backward(n, rin, H, yv, ldy, T, md, po, ga, pr, dro, 0 if dro is None else dro.stride(0), dx, dx.stride(0) if pre else 0,
                              dr, dr.stride(0), dy, dy.stride(0) if y else 0, got["dpost"] if po is not None else None,
                              got["dgate"] if ga is not None and y else None, got["dpre"] if pre else None, acc, ws)
    torch.cuda.synchronize()
    want = ref.norm_backward(w64(rin)[on], None if yv is None else w64(yv)[on], w64(po), gsel, w64(pr),
                             None if dro0 is None else w64(dro0)[on], None if dx is None else w64(dx)[on], scale, eps, gate)
    ref.close(dr.cpu()[on], *ref.rounded(*want["dr"], rt), "dr")
    assert (dr.cpu()[~mk] == 0).all()
    if y:
        ref.close(dy.cpu()[on], *ref.rounded(*want["dy"], yt), "dy")
        assert (dy.cpu()[~mk] == 0).all()
    for k in ("dpost", "dgate", "dpre"):
        if k not in want:
            assert torch.equal(got[k], old[k])
            continue
        v, off = want[k]
        if k == "dgate" and gate == "token":
            full, o = torch.zeros(T, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
            full[on], o[on] = v, off
            v, off = full, o
        if acc:
            v = v + w64(old[k])
            off = off + ref.EPS * v.abs() + ref.EPS * w64(old[k]).abs()
        ref.close(got[k], v, off + ref.TINY[torch.float32], k)
    return ro.clone(), got


@pytest.mark.parametrize("T,H", [(1, 8), (1, 2560), (3, 2048), (5, 2056), (7, 4096), (4, 4104), (2, 8200), (2, 16384), (600, 264), (1300, 64), (513, 1032)])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_sizes(m, T, H, gate):
    check(m, T, H, gate=gate)


@pytest.mark.parametrize("kinds", list(itertools.product(sorted(DT), repeat=3)))
def test_types(m, kinds):
    check(m, 37, 520, kinds=kinds, gate="token")


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("y,post,pre", [(True, False, True), (True, True, False), (True, False, False), (False, False, True)])
@pytest.mark.parametrize("dr_out", [True, False])
def test_parts_left_out(m, gate, y, post, pre, dr_out):
    check(m, 19, 264, ("bf16", "f32", "f32"), gate, y, post, pre, dr_out=dr_out)


@pytest.mark.parametrize("mask", ["tail", "all", "mixed"])
@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("acc", [False, True])
def test_masks(m, mask, gate, acc):
    check(m, 700, 136, ("bf16", "f16", "f32"), gate, mask=mask, acc=acc)


@pytest.mark.parametrize("kinds", [("f32", "f32", "f32"), ("bf16", "f32", "f32"), ("f16", "bf16", "f16")])
def test_in_place_and_accumulation(m, kinds):
    check(m, 65, 1032, kinds, "channel", inplace=True, acc=True)


def test_zero_rows(m):
    """A block output of zeros leaves the stream as it is, and a stream of zeros gives x = 0; gradients stay finite."""
    H = 256
    n = m.norm_desc(H, torch.float32, torch.float32, torch.float32, "none", 1.0, 1e-6)
    r, y = torch.zeros((2, H), device="cuda"), torch.zeros((2, H), device="cuda")
    r[0] = 1.5
    w = torch.ones(H, device="cuda")
    ro, x = torch.empty_like(r), torch.empty_like(r)
    m.moe_block_norm(n, r, H, y, H, 2, None, w, None, w, ro, H, x, H)
    assert torch.equal(ro, r) and (x[1] == 0).all()
    dx, dr, dy = torch.ones_like(r), torch.empty_like(r), torch.empty_like(r)
    dpost, dpre = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    ws = torch.empty(m.moe_block_norm_workspace_bytes(n, 2), dtype=torch.uint8, device="cuda")
    m.moe_block_norm_backward(n, ro, H, y, H, 2, None, w, None, w, None, 0, dx, H, dr, H, dy, H, dpost, None, dpre, 0, ws)
    assert all(t.isfinite().all() for t in (dr, dy, dpost, dpre))


def test_no_tokens(m):
    H = 64
    n = m.norm_desc(H, torch.float32, torch.float32, torch.float32, "channel", 1.0, 1e-6)
    w = torch.ones(H, device="cuda")
    out = [torch.full((H,), 5.0, device="cuda") for _ in range(3)]
    e = torch.empty((0, H), device="cuda")
    ws = torch.empty(max(256, m.moe_block_norm_workspace_bytes(n, 0)), dtype=torch.uint8, device="cuda")
    args = (n, e, H, e, H, 0, None, w, w, w, None, 0, e, H, None, 0, None, 0)
    m.moe_block_norm_backward(*args, *out, 1, ws)
    assert all((o == 5).all() for o in out)
    m.moe_block_norm_backward(*args, *out, 0, ws)
    assert all((o == 0).all() for o in out)


def test_rows_past_31_bits(m):
    """Rows whose offsets pass 2^31 elements."""
    H, T, ld = 64, 3, (1 << 30) + 8
    buf = torch.empty(2 * ld + H, dtype=torch.bfloat16, device="cuda")
    r = buf.as_strided((T, H), (ld, 1))
    v = torch.randn((T, H), device="cuda").bfloat16()
    r.copy_(v)
    n = m.norm_desc(H, torch.bfloat16, torch.bfloat16, torch.float32, "none", 1.0, 1e-6)
    w = torch.ones(H, device="cuda")
    x, x2 = torch.empty((T, H), device="cuda"), torch.empty((T, H), device="cuda")
    m.moe_block_norm(n, r, ld, None, 0, T, None, None, None, w, None, 0, x, H)
    m.moe_block_norm(n, v, H, None, 0, T, None, None, None, w, None, 0, x2, H)
    assert torch.equal(x, x2)


@pytest.mark.parametrize("T", [1, 900])
def test_repeated_and_replayed(m, T):
    """Run to run and captured: bit-identical, with junk in the workspace."""
    H = 520
    g = torch.Generator().manual_seed(4)
    n = m.norm_desc(H, torch.bfloat16, torch.float32, torch.float32, "channel", 0.5, 1e-6)
    mk = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    r, y, dr_out, dx = mk(T, H).bfloat16(), mk(T, H), mk(T, H).bfloat16(), mk(T, H)
    post, gate, pre = mk(H), mk(H), mk(H)
    outs = [torch.empty_like(r), torch.empty_like(y), torch.empty_like(r), torch.empty_like(y), torch.empty_like(post), torch.empty_like(post), torch.empty_like(post)]
    ws = torch.empty(m.moe_block_norm_workspace_bytes(n, T), dtype=torch.uint8, device="cuda")

    def step():
        ro, x, dr, dy, dpost, dgate, dpre = outs
        m.moe_block_norm(n, r, H, y, H, T, None, post, gate, pre, ro, H, x, H)
        m.moe_block_norm_backward(n, ro, H, y, H, T, None, post, gate, pre, dr_out, H, dx, H, dr, H, dy, H, dpost, dgate, dpre, 0, ws)

    step()
    want = [t.clone() for t in outs]
    q = torch.cuda.CUDAGraph()
    with torch.cuda.graph(q):
        step()
    for _ in range(3):
        for t in outs:
            t.fill_(9)
        ws.fill_(0xFF)
        q.replay()
        torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
