"""The operators around a routed layer as a program strings them together, each
checked on what the one before left on the GPU, against the references of
tests/serve_ref.py, and the whole run captured and replayed:

* serving: moe_block_norm -> moe_layer_decode_batch -> moe_block_norm, twice,
  then moe_fp4_apply as the head, with empty slots in the batch;
* training: moe_fp4_quant once; moe_block_norm -> moe_fp4_apply and
  moe_lora_apply onto it -> moe_fp4_backward and moe_lora_backward onto it ->
  moe_block_norm_backward;
* a layer's and a product's graph over one workspace.
"""
import pytest
import torch

import learn_ref
import serve_ref as ref
from test_gpu_layer_batch import blocks_of, matrices
from test_gpu_learn_together import replayed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import block_scaled_fp4_route_amd as m
    return m


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,masked", [(1, ()), (4, ()), (1, (0,)), (7, (2, 6)), (33, (0, 20, 21))])
def test_serving_two_layers_and_a_head(m, T, masked, fmt):
    H, I, E, k, V, eps = 512, 96, 24, 4, 1032, 1e-5
    g = torch.Generator().manual_seed(T)
    blocks = [blocks_of(g, E, H, I, fmt) for _ in range(2)]
    gblocks = [b.cuda() for b in blocks]
    tables = [m.expert_ptr_table(b) for b in gblocks]
    Wr = [(torch.randn((E, H), generator=g) * 0.1) for _ in range(2)]
    gWr = [w.cuda() for w in Wr]
    pre, post, gate = ([(torch.randn(H, generator=g) * s + c) for _ in range(3)] for s, c in ((0.1, 1.0), (0.1, 0.01), (0.5, 1.0)))
    gpre, gpost, ggate = ([t.cuda() for t in ts] for ts in (pre, post, gate))
    Wh = (torch.randn((V, H), generator=g) * 0.05).cuda()
    codes, scales = torch.empty((V, H // 2), dtype=torch.uint8, device="cuda"), torch.empty((V, H // ref.GROUP[fmt]), dtype=torch.uint8, device="cuda")
    e = torch.empty(V, dtype=torch.int8, device="cuda") if fmt == "nvfp4" else None
    m.moe_fp4_quant(Wh, H, V, H, Wh.dtype, fmt, m.MOE_SCALE_NEAREST if e is not None else m.MOE_SCALE_FLOOR, e, codes, scales, None, 0)
    on = [t for t in range(T) if t not in masked]
    mask = None
    r0 = torch.randn((T, H), generator=g)
    if masked:
        mask = torch.ones(T, dtype=torch.uint8)
        mask[list(masked)] = 0
        r0[list(masked)] = float("nan")
        mask = mask.cuda()
    r0 = r0.cuda()
    n = m.norm_desc(H, torch.float32, torch.float32, torch.float32, "channel", 0.5, eps)
    n0 = m.norm_desc(H, torch.float32, torch.float32, torch.float32, "none", 1.0, eps)
    d, f = m.desc(H, I, E, k, fmt), m.fp4_desc(H, V, fmt, torch.float32)
    ws = torch.empty(max(m.moe_workspace_bytes(d, T, m.MOE_MODE_DECODE_BATCH), m.moe_fp4_workspace_bytes(f, T, False)), dtype=torch.uint8, device="cuda")
    x, r, y = ([torch.zeros((T, H), device="cuda") for _ in range(c)] for c in (3, 3, 2))
    idx, w = [torch.zeros((T, k), dtype=torch.int32, device="cuda") for _ in range(2)], [torch.zeros((T, k), device="cuda") for _ in range(2)]
    out = torch.zeros((T, V), device="cuda")

    def step():
        m.moe_block_norm(n0, r0, H, None, 0, T, mask, None, None, gpre[0], r[0], H, x[0], H)
        for i in range(2):
            m.moe_layer_decode_batch(d, x[i], T, mask, gWr[i], tables[i], None, y[i], idx[i], w[i], ws)
            m.moe_block_norm(n, r[i], H, y[i], H, T, mask, gpost[i], ggate[i], gpre[i + 1], r[i + 1], H, x[i + 1], H)
        m.moe_fp4_apply(f, x[2], H, T, codes, scales, e, False, None, 0, out, V, ws)

    step()
    torch.cuda.synchronize()
    c64 = lambda t: t.cpu().double()  # noqa: E731
    _, _, v, off = ref.norm_forward(c64(r0)[on], None, None, None, c64(pre[0]), 1.0, eps, "none")
    ref.close(x[0][on], *ref.rounded(v, off, torch.float32), "x0")
    assert torch.equal(r[0][on], r0[on])
    for i in range(2):
        X, W = c64(x[i])[on], Wr[i].double()
        logits, el = learn_ref.mm(X, W.t().contiguous())
        ii = idx[i].cpu()[on].long()
        chosen, ec = logits.gather(1, ii), el.gather(1, ii)
        left = torch.ones_like(logits, dtype=torch.bool).scatter(1, ii, False)
        # in order, and none left out that is larger, but for the logits' errors
        assert (chosen[:, :-1] - chosen[:, 1:] >= -(ec[:, :-1] + ec[:, 1:])).all()
        for t in range(len(on)):
            assert len(set(ii[t].tolist())) == k
            assert (logits[t][left[t]] - el[t][left[t]]).max() <= chosen[t, -1] + ec[t, -1]
        p = torch.softmax(chosen, 1)
        # a logit off by e moves every weight by a factor of exp(2 e) at most
        ref.close(w[i][on], p, (1.01 * 2 * ec.amax(1, keepdim=True) + (k + 20) * ref.EPS) * p + 1e-38, ("w", i))
        mats = {int(a): matrices(blocks[i][int(a)], H, I, fmt) for a in ii.unique()}
        v, off = ref.layer(X, mats, None, ii, c64(w[i])[on])
        ref.close(y[i][on], v, off, ("y", i))
        s, es, v, off = ref.norm_forward(c64(r[i])[on], c64(y[i])[on], c64(post[i]), c64(gate[i]), c64(pre[i + 1]), 0.5, eps, "channel")
        ref.close(r[i + 1][on], *ref.rounded(s, es, torch.float32), ("r", i + 1))
        ref.close(x[i + 1][on], *ref.rounded(v, off, torch.float32), ("x", i + 1))
    v, off = ref.product(c64(x[2])[on], ref.decode(codes, scales, fmt, e), None, torch.float32)
    ref.close(out[on], v, off, "head")
    for t in (*x, *y, *r[1:]):
        assert (t[list(masked)] == 0).all()
    replayed_rows(step, [out, *y, *w, *idx, r[2]], on)


def replayed_rows(fn, outs, on):
    """fn captured gives the rows that it gave eagerly, on every replay. What it does not write stays as it was, also
    what the program put there between the replays."""
    want = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    for _ in range(3):
        for t in outs:
            t[on] = 9
        g.replay()
        torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [2, 33, 200])
def test_training_step_over_a_frozen_matrix(m, T, fmt, dt):
    """h = rms(r + gate rms(y) post) pre; z = W4 h + adapters(h), W4 frozen in 4 bits; the gradients of everything that learns
    and of the residual stream."""
    K, N, eps, scale = 512, 264, 1e-5, 0.7
    g = torch.Generator().manual_seed(T)
    W = torch.randn((N, K), generator=g).cuda() * 0.05
    codes, scales = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda"), torch.empty((N, K // ref.GROUP[fmt]), dtype=torch.uint8, device="cuda")
    e = torch.empty(N, dtype=torch.int8, device="cuda") if fmt == "nvfp4" else None
    W4 = torch.empty_like(W)
    m.moe_fp4_quant(W, K, N, K, W.dtype, fmt, m.MOE_SCALE_NEAREST if e is not None else m.MOE_SCALE_FLOOR, e, codes, scales, W4, K)
    assert torch.equal(W4.cpu().double(), ref.decode(codes, scales, fmt, e))
    # off by one scale at most (half the step between 4 and 6), and where the largest value saturates (MXFP4: below 8
    # scales, so 6/8 of it are left; NVFP4: above 6 scales by the scale's own 2^-4 at most) by a quarter of it
    assert (W4 - W).abs().max() <= 0.25 * W.abs().max()
    r, y = (torch.randn((T, K), generator=g).to(dt).cuda() for _ in range(2))
    post, gate, pre = ((torch.randn(K, generator=g) * 0.2 + 1).cuda() for _ in range(3))
    ranks = [8, 4]
    A = [(torch.randn((q, K), generator=g) * K ** -0.5).bfloat16().cuda() for q in ranks]
    B = [(torch.randn((q, N), generator=g) * 0.1).bfloat16().cuda() for q in ranks]
    ids = (torch.arange(T) % 3 - 1).to(torch.int32).cuda()
    ptrs = lambda ts: torch.tensor([t.data_ptr() for t in ts], dtype=torch.int64).cuda()  # noqa: E731
    lsc = torch.tensor([2.0, 0.5]).cuda()
    tab = (ids, ptrs(A), ptrs(B), torch.tensor(ranks, dtype=torch.int32).cuda(), lsc)
    dA, dB = [torch.empty(a.shape, device="cuda") for a in A], [torch.empty(b.shape, device="cuda") for b in B]
    grads = ptrs(dA), ptrs(dB)
    n, f, l = m.norm_desc(K, dt, dt, dt, "channel", scale, eps), m.fp4_desc(K, N, fmt, dt), m.lora_desc(K, N, 2, 8, dt)
    ws = torch.empty(max(m.moe_fp4_workspace_bytes(f, T, False), m.moe_fp4_workspace_bytes(f, T, True), m.moe_lora_workspace_bytes(l, T, True),
                         m.moe_block_norm_workspace_bytes(n, T)), dtype=torch.uint8, device="cuda")
    ro, h, dh4, dh, dr, dy = (torch.empty((T, K), dtype=dt, device="cuda") for _ in range(6))
    z4, z = (torch.empty((T, N), dtype=dt, device="cuda") for _ in range(2))
    dz, dro = torch.randn((T, N), generator=g).to(dt).cuda(), torch.randn((T, K), generator=g).to(dt).cuda()
    dpost, dgate, dpre = (torch.empty(K, device="cuda") for _ in range(3))

    def step():
        m.moe_block_norm(n, r, K, y, K, T, None, post, gate, pre, ro, K, h, K)
        m.moe_fp4_apply(f, h, K, T, codes, scales, e, False, None, 0, z4, N, ws)
        m.moe_lora_apply(l, h, K, T, *tab, z4, N, z, N, ws)
        m.moe_fp4_backward(f, dz, N, T, codes, scales, e, None, 0, dh4, K, ws)
        m.moe_lora_backward(l, h, K, dz, N, T, *tab, dh4, K, dh, K, *grads, 0, ws)
        m.moe_block_norm_backward(n, ro, K, y, K, T, None, post, gate, pre, dro, K, dh, K, dr, K, dy, K, dpost, dgate, dpre, 0, ws)

    step()
    torch.cuda.synchronize()
    c = ref.cpu64
    s, es, v, off = ref.norm_forward(c(r), c(y), c(post), c(gate), c(pre), scale, eps, "channel")
    ref.close(ro, *ref.rounded(s, es, dt), "r_out")
    ref.close(h, *ref.rounded(v, off, dt), "h")
    ref.close(z4, *ref.product(c(h), c(W4), None, dt), "z4")
    ref.close(z, *learn_ref.lora(h, ids, A, B, lsc, z4, dt, 2), "z")
    ref.close(dh4, *ref.product(c(dz), c(W4).t().contiguous(), None, dt), "dh4")
    ref.close(dh, *learn_ref.lora(dz, ids, B, A, lsc, dh4, dt, 2), "dh")
    for a, (wa, wb) in enumerate(learn_ref.lora_grads(h, dz, ids, A, B, lsc, 2)):
        ref.close(dA[a], *wa, ("dA", a))
        ref.close(dB[a], *wb, ("dB", a))
    want = ref.norm_backward(c(ro), c(y), c(post), c(gate), c(pre), c(dro), c(dh), scale, eps, "channel")
    for name, got in (("dr", dr), ("dy", dy)):
        ref.close(got, *ref.rounded(*want[name], dt), name)
    for name, got in (("dpost", dpost), ("dgate", dgate), ("dpre", dpre)):
        ref.close(got, *want[name], name)
    if dt == torch.float32:
        # the step as a whole against autograd in 64 bits: 2^-10 of each gradient's largest value. Every value that
        # enters a sum is off by at most (3 K + 2) 2^-24 < 2^-13 of the magnitudes that made it, four sums follow one
        # another (norm, product or adapter, its gradient, the norm's), and sums of values of both signs are smaller
        # than their magnitudes' by no more than the square root of the terms' number here: 4 2^-13 at the outside
        # from each, and fp32 sums of random signs stay far below their bounds
        p = [t.cpu().double().requires_grad_() for t in (r, y, post, gate, pre)]
        fac = [t.cpu().double().requires_grad_() for t in (*A, *B)]
        rms = lambda t: t / ((t * t).mean(1, keepdim=True) + eps).sqrt()  # noqa: E731
        S = p[0] + scale * p[3] * (rms(p[1]) * p[2])
        hh = rms(S) * p[4]
        zz = hh @ c(W4).t()
        for a in range(2):
            zz = zz + (ids.cpu() == a)[:, None] * float(lsc[a]) * (hh @ fac[a].t() @ fac[2 + a])
        ((zz * c(dz)).sum() + (S * c(dro)).sum()).backward()
        for name, got, w in zip(("dr", "dy", "dpost", "dgate", "dpre", "dA0", "dA1", "dB0", "dB1"), (dr, dy, dpost, dgate, dpre, *dA, *dB), p + fac):
            assert (c(got) - w.grad).abs().max() <= 2.0 ** -10 * w.grad.abs().max(), name
    replayed(step, [ro, h, z, dh, dr, dy, dpost, dgate, dpre, *dA, *dB])


def test_two_graphs_share_a_workspace(m):
    """A product's and a layer's graph, replayed in turn over one workspace, and eager calls of both between them."""
    H, I, E, k, T, N = 512, 96, 24, 4, 9, 520
    g = torch.Generator().manual_seed(2)
    blocks = blocks_of(g, E, H, I, "mxfp4").cuda()
    ptrs, Wr, x = m.expert_ptr_table(blocks), (torch.randn((E, H), generator=g) * 0.1).cuda(), torch.randn((T, H), generator=g).cuda()
    codes = torch.randint(0, 256, (N, H // 2), dtype=torch.uint8, generator=g).cuda()
    scales = torch.randint(121, 130, (N, H // 32), dtype=torch.uint8, generator=g).cuda()
    d, f = m.desc(H, I, E, k, "mxfp4"), m.fp4_desc(H, N, "mxfp4", torch.float32)
    dz = torch.randn((T, N), generator=g).cuda()
    ws = torch.full((max(m.moe_workspace_bytes(d, T, m.MOE_MODE_DECODE_BATCH), m.moe_fp4_workspace_bytes(f, T, True)),), 0xFF, dtype=torch.uint8, device="cuda")
    y, idx, w, dx = torch.empty((T, H), device="cuda"), torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda"), torch.empty((T, H), device="cuda")
    fns = [lambda: m.moe_layer_decode_batch(d, x, T, None, Wr, ptrs, None, y, idx, w, ws),
           lambda: m.moe_fp4_backward(f, dz, N, T, codes, scales, None, None, 0, dx, H, ws)]
    for fn in fns:
        fn()
    torch.cuda.synchronize()
    want, graphs = [t.clone() for t in (y, idx, w, dx)], []
    for fn in fns:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fn()
    for i in range(4):
        for t in (y, idx, w, dx):
            t.fill_(9)
        (graphs[0].replay, fns[0])[i // 2 % 2]()
        (graphs[1].replay, fns[1])[i % 2]()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, idx, w, dx), want))
