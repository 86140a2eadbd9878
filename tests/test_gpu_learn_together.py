"""The router's training operators and the adapters as a program strings them
together, each on the outputs of the one before, against autograd in 64 bits:

* moe_route -> expert outputs (moe_expert_prefill, one expert a row) -> dw,
  moe_balance_loss -> moe_route_backward, over padded sequences;
* moe_gemv_fp8 -> moe_lora_apply onto its output -> moe_lora_backward onto
  the projection's own gradient.

The tolerances are those of the single operators (tests/learn_ref.py) with
the errors of what they start from carried through; each test says how.
"""
import pytest
import torch

import learn_ref as ref
import synthgen as sg
from gpu_helpers import layer_blocks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import block_scaled_fp4_route_amd as m
    return m


def replayed(fn, outs):
    """fn captured in a graph gives what it gave eagerly, on every replay."""
    want = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    for _ in range(3):
        for t in outs:
            t.fill_(9)
        g.replay()
        torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("T,E", [(150, 32), (1, 32), (1100, 64)])
def test_a_training_step_of_the_router(m, T, E):
    H, I, k, cb, cz = 512, 128, 4, 0.01, 0.001
    wl = sg.Workload("learn_small", 95, H, I, E, k, "nvfp4", 1, T, False, "zipf", 1.1, 0x18, 0x48, False)
    g = torch.Generator().manual_seed(T)
    d, d1 = m.desc(H, I, E, k, "nvfp4"), m.desc(H, I, E, 1, "nvfp4")
    blocks = layer_blocks(wl)
    ptrs = m.expert_ptr_table(blocks)
    x, Wr = torch.randn((T, H), generator=g).cuda(), (torch.randn((E, H), generator=g) * 0.05).cuda()
    dy = torch.randn((T, H), generator=g).cuda()
    mask = torch.ones(T, dtype=torch.uint8)
    mask[T // 3:T // 3 + T // 10] = 0  # padding within the first sequence
    off = [0, T // 2, T // 2, T]
    maskd, offd = mask.cuda(), torch.tensor(off, dtype=torch.int32).cuda()
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    logits, dl, G = (torch.empty((T, E), device="cuda") for _ in range(3))
    o, dw = torch.empty((T * k, H), device="cuda"), torch.empty((T, k), device="cuda")
    loss, counts = torch.empty(3, device="cuda"), torch.empty((3, E), dtype=torch.int32, device="cuda")
    dx, dWr = torch.empty((T, H), device="cuda"), torch.empty((E, H), device="cuda")
    rows, ones = torch.empty((T * k, H), device="cuda"), torch.ones(T * k, device="cuda")
    ws = m.alloc_workspace(d1, T * k, m.MOE_MODE_PREFILL)
    wr = m.alloc_workspace(d, T, m.MOE_MODE_ROUTE)
    # one workspace for the loss and the gradient, which follow one another
    wl_ = torch.empty(max(m.moe_balance_workspace_bytes(d, T, 3), m.moe_route_backward_workspace_bytes(d, T)),
                      dtype=torch.uint8, device="cuda")

    rows.view(T, k, H).copy_(x[:, None, :].expand(T, k, H))

    def forward():
        m.moe_route(d, x, T, Wr, idx, w, logits, wr)
        m.moe_expert_prefill(d1, rows, T * k, ptrs, idx, ones, o, m.MOE_OUT_F32, ws)

    def backward():
        m.moe_balance_loss(d, logits, T, idx, maskd, offd, 3, cb, cz, None, loss, counts, None, dl, wl_)
        m.moe_route_backward(d, x, T, Wr, idx, w, dw, maskd, dl, G, dx, dWr, 0, wl_)

    forward()
    dw.copy_((o.view(T, k, H) * dy[:, None, :]).sum(2))
    backward()
    torch.cuda.synchronize()
    # the same in 64 bits: the experts' outputs (through dw) and the choice of
    # experts are given, the logits and everything behind them are not
    X, W, DW = x.cpu().double().requires_grad_(), Wr.cpu().double().requires_grad_(), dw.cpu().double()
    ii, on = idx.cpu().long(), mask.bool()
    L = X @ W.t()
    L.retain_grad()
    ws64, p, lse = torch.softmax(L.gather(1, ii), 1), torch.softmax(L, 1), torch.logsumexp(L, 1)
    live = [[t for t in range(off[s], off[s + 1]) if on[t]] for s in range(3)]
    nlive, N = sum(len(r) > 0 for r in live), sum(len(r) for r in live)
    bal, coef = 0.0, torch.zeros((T, E), dtype=torch.float64)  # coef: what multiplies p[t][e] in the balance term
    for s, r in enumerate(live):
        c = torch.bincount(ii[r].flatten(), minlength=E).double()
        assert torch.equal(counts[s].cpu().double(), c)
        if r:
            coef[r] = cb * E * c / (nlive * len(r) * k * len(r))
            bal = bal + (coef[r] * p[r]).sum() / cb
    z = (lse[on] ** 2).sum() / N
    total = cb * bal + cz * z
    (total + (ws64 * DW)[on].sum()).backward()
    # A logit is off by el; softmaxes by a factor of exp(2 el) and their own
    # rounding (8 EPS), so w and p by rho of themselves, and a gradient of the
    # form w (c - sum w c) by rho (w |c| + 2 w sum w |c|); lse by el.
    el = (ref.mm(X.detach(), W.detach().t().contiguous())[1]).amax(1, keepdim=True)
    rho = 1.01 * (2 * el + 8 * ref.EPS)
    ew = rho * (ws64 * DW.abs() + 2 * ws64 * (ws64 * DW.abs()).sum(1, keepdim=True)).detach()
    eb = rho * (p * coef + 2 * p * (p * coef).sum(1, keepdim=True)).detach()
    ez = (2 * cz / N * p * (rho * lse.abs()[:, None] + el)).detach()
    eG = (eb + ez).scatter_add(1, ii, ew) * on[:, None]
    own = ref.route_backward(x, Wr, idx, w, dw, mask.bool(), dl, T, E, k)  # from the values that it was given
    bl = ref.balance(logits, idx.cpu(), on, off, k, cb, cz)
    ref.close(loss[0], total.detach(), bl["loss"][1][0] + (2 * rho.amax() * total + 2 * cz * el.amax() * lse.abs().amax()).detach(), "loss")
    eGl = bl["dlogits"][1] + eG
    ref.close(G, L.grad, own["dlogits"][1] + eGl, "G")
    ref.close(dx, X.grad, own["dx"][1] + eGl @ W.detach().abs(), "dx")
    ref.close(dWr, W.grad, own["dWr"][1] + eGl.t() @ X.detach().abs(), "dWr")
    replayed(lambda: (forward(), backward()), [logits, idx, w, o, loss, G, dx, dWr])


@pytest.mark.parametrize("T", [1, 3])
def test_adapters_beside_the_fp8_projection(m, T):
    K, N, ranks = 2560, 1024, [16, 8, 4]
    Wq, s = sg.fp8_matrix(N, K, 5).cuda(), sg.fp8_row_scales(N, 5).cuda()
    g = torch.Generator().manual_seed(T)
    x, dy = torch.randn((T, K), generator=g).cuda(), torch.randn((T, N), generator=g).cuda()
    A = [(torch.randn((r, K), generator=g) * K ** -0.5).bfloat16().cuda() for r in ranks]
    B = [(torch.randn((r, N), generator=g) * 0.1).bfloat16().cuda() for r in ranks]
    ids = torch.tensor([2, -1, 0][:T], dtype=torch.int32).cuda()
    ptrs = lambda ts: torch.tensor([t.data_ptr() for t in ts], dtype=torch.int64).cuda()  # noqa: E731
    scales = torch.tensor([2.0, 0.5, 1.5]).cuda()
    dA, dB = [torch.empty(a.shape, device="cuda") for a in A], [torch.empty(b.shape, device="cuda") for b in B]
    tab = (ids, ptrs(A), ptrs(B), torch.tensor(ranks, dtype=torch.int32).cuda(), scales)
    grads = ptrs(dA), ptrs(dB)
    l = m.lora_desc(K, N, 3, 16, torch.float32)
    ws = torch.empty(m.moe_lora_workspace_bytes(l, T, True), dtype=torch.uint8, device="cuda")
    y, dx = torch.empty((T, N), device="cuda"), torch.empty((T, K), device="cuda")
    W64 = Wq.view(torch.float8_e4m3fn).float().cpu().double() * s.cpu().double()[:, None]
    dxb = (dy.cpu().double() @ W64).float().cuda()

    def step():
        for t in range(T):
            m.moe_gemv_fp8(Wq, s, x[t], N, K, y[t])
        m.moe_lora_apply(l, x, K, T, *tab, y, N, y, N, ws)
        dx.copy_(dxb)
        m.moe_lora_backward(l, x, K, dy, N, T, *tab, dx, K, dx, K, *grads, 0, ws)

    step()
    torch.cuda.synchronize()
    base, eb = ref.mm(x.cpu().double(), W64.t().contiguous())
    # the projection's sums round like any of K terms, its row scale once more
    eb = eb + 2 * ref.EPS * base.abs()
    v, e = ref.lora(x, ids, A, B, scales, base, torch.float32, 3)
    ref.close(y, v, e + eb, "y")
    ref.close(dx, *ref.lora(dy, ids, B, A, scales, dxb, torch.float32, 3), "dx")
    for a, (wa, wb) in enumerate(ref.lora_grads(x, dy, ids, A, B, scales, 3)):
        ref.close(dA[a], *wa, ("dA", a))
        ref.close(dB[a], *wb, ("dB", a))
    replayed(step, [y, dx, *dA, *dB])
