"""Cases of the operators that train a routed layer's router and carry low-rank adapters beside its projections.

Four operators, each in its plain form (elementary torch operations in fp32) and as the framework's call:

balance        the balance loss of a router (and its z loss), the per-expert counts, and the logits' gradient
route_backward the gradients of the routing: logits, router weights and layer input
lora           low-rank adapters of many requests added to a shared projection's output
lora_backward  the gradients of those adapters and of their input
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a 311-token prompt through a 384-expert, top-6 router: one step of a small fine-tuning batch
        {"name": "balance_311x384", "op": "balance", "T": 311, "E": 384, "k": 6, "S": 1, "masked": 0.0},
        # a 2451-token prompt through a 512-expert, top-10 router
        {"name": "balance_2451x512", "op": "balance", "T": 2451, "E": 512, "k": 10, "S": 1, "masked": 0.0},
        # a packed training batch: 37 ragged sequences, balanced one by one, some of their tokens padding
        {"name": "balance_32768x512_s37", "op": "balance", "T": 32768, "E": 512, "k": 10, "S": 37, "masked": 0.12},
        # the router's backward pass of the small batch, hidden size 4096
        {"name": "route_backward_311x384", "op": "route_backward", "T": 311, "E": 384, "k": 6, "H": 4096, "masked": 0.0},
        # the router's backward pass of a long batch with padding, hidden size 2560
        {"name": "route_backward_8191x512", "op": "route_backward", "T": 8191, "E": 512, "k": 10, "H": 2560, "masked": 0.1},
        # one decoded token of one request beside the 8192 x 2560 FP8 projection
        {"name": "lora_1_f32", "op": "lora", "T": 1, "K": 2560, "N": 8192, "n": 8, "r": 16, "runs": 0, "ragged": False, "dtype": "f32"},
        # a decode batch: 64 requests over 32 adapters of unequal ranks
        {"name": "lora_64_bf16", "op": "lora", "T": 64, "K": 2560, "N": 8192, "n": 32, "r": 16, "runs": 0, "ragged": True, "dtype": "bf16"},
        # prompts of several requests, 2451 tokens in 8 runs, larger ranks
        {"name": "lora_2451_f16", "op": "lora", "T": 2451, "K": 2560, "N": 2560, "n": 4, "r": 64, "runs": 8, "ragged": False, "dtype": "f16"},
        # a long prefill batch over 16 adapters
        {"name": "lora_8192_bf16", "op": "lora", "T": 8192, "K": 2560, "N": 8192, "n": 16, "r": 16, "runs": 24, "ragged": False, "dtype": "bf16"},
        # a small training step of three adapters in fp32 activations
        {"name": "lora_backward_300_f32", "op": "lora_backward", "T": 300, "K": 2560, "N": 640, "n": 3, "r": 8, "runs": 5, "ragged": True, "dtype": "f32"},
        # a training step of four adapters side by side
        {"name": "lora_backward_4096_f16", "op": "lora_backward", "T": 4096, "K": 4096, "N": 2880, "n": 4, "r": 16, "runs": 9, "ragged": False, "dtype": "f16"},
        # a long training step of one adapter of rank 64
        {"name": "lora_backward_8192_bf16", "op": "lora_backward", "T": 8192, "K": 2560, "N": 8192, "n": 1, "r": 64, "runs": 1, "ragged": False, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "route_backward", "lora", "lora", "lora_backward"])
    if op == "balance":
        E = _spread(rng, 8, 1024)
        T = _spread(rng, 1, 32768 * 512 // max(E, 512))
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(E, 16)), "S": _spread(rng, 1, 64), "masked": rng.choice([0.0, 0.0, 0.1, 0.5])}
    if op == "route_backward":
        E, H = _spread(rng, 8, 512), 256 * rng.randint(1, 16)
        T = min(_spread(rng, 1, 8191), 8191 * 512 * 2560 // (E * H))
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(E, 16)), "H": H, "masked": rng.choice([0.0, 0.1])}
    K, N, r = 8 * _spread(rng, 32, 512), 8 * _spread(rng, 32, 1024), _spread(rng, 1, 128)
    # the adapters' ranks together stay in what the plain form's two dense products pay for
    n = max(1, min(_spread(rng, 1, 32), 512 // r))
    T = _spread(rng, 1, 8192)
    if op == "lora_backward":
        r = min(r, 64)
    case = {"op": op, "T": T, "K": K, "N": N, "n": n, "r": r, "runs": rng.choice([0, 1, 7]), "ragged": rng.random() < 0.5, "dtype": rng.choice(sorted(DTYPES))}
    big = next(c for c in listed() if c["name"] == "lora_backward_8192_bf16")
    while case["T"] > 1 and (work(case)["flops"] > work(big)["flops"] or work(case)["bytes"] > work(big)["bytes"]):
        case["T"] = (case["T"] + 1) // 2
    return case


def _ranks(case):
    r, n = case["r"], case["n"]
    return [max(1, r - (a * 5) % r) if case["ragged"] else r for a in range(n)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.RandomState(seed % (1 << 31))
    dev = {"device": "cuda"}

    def normal(*size, std=1.0, dtype=torch.float32):
        return torch.empty(size, dtype=dtype, **dev).normal_(0, std, generator=g)

    T, st = case["T"], {"case": dict(case)}
    if case["op"] in ("balance", "route_backward"):
        E, k = case["E"], case["k"]
        # logits of a router whose experts are not used alike; the routing is what the router itself chooses
        lift = normal(E, std=0.7)
        st["logits"] = normal(T, E) + lift
        top = torch.sort(st["logits"], dim=1, descending=True, stable=True)
        st["idx"] = top.indices[:, :k].to(torch.int32).contiguous()
        st["w"] = torch.softmax(top.values[:, :k], dim=1).contiguous()
        del top
        st["mask"] = None
        if case["masked"]:
            st["mask"] = (torch.rand(T, generator=g, **dev) >= case["masked"]).to(torch.uint8)
    if case["op"] == "balance":
        S = case["S"]
        cuts = np.sort(host.randint(0, T + 1, S - 1))  # sequences without tokens among them
        st["seq_off"] = torch.tensor(np.concatenate([[0], cuts, [T]]), dtype=torch.int32, **dev)
        st["coef"] = (0.01, 0.001)
        st["dloss"] = torch.full((1,), 0.5, **dev)
        st["out"] = {"loss": torch.empty(3, **dev), "counts": torch.empty((S, E), dtype=torch.int32, **dev),
                     "probs": torch.empty((S, E), **dev), "dlogits": torch.empty((T, E), **dev)}
    elif case["op"] == "route_backward":
        H = case["H"]
        st["x"] = normal(T, H)
        st["Wr"] = normal(E, H, std=0.02)
        st["dw"] = normal(T, k, std=0.1)
        st["dlogits"] = normal(T, E, std=1e-3)
        st["out"] = {"dlogits": torch.empty((T, E), **dev), "dx": torch.empty((T, H), **dev), "dWr": torch.empty((E, H), **dev)}
        del st["logits"]
    else:
        K, N, n, dt = case["K"], case["N"], case["n"], DTYPES[case["dtype"]]
        wt = torch.float16 if dt == torch.float16 else torch.bfloat16
        ranks = _ranks(case)
        st["A"] = normal(sum(ranks), K, std=K ** -0.5, dtype=wt)
        st["B"] = normal(sum(ranks), N, std=0.05, dtype=wt)
        first = np.concatenate([[0], np.cumsum(ranks)[:-1]]).astype(np.int64)
        st["owner"] = torch.tensor(np.repeat(np.arange(n), ranks), dtype=torch.int64, **dev)
        st["ranks"] = torch.tensor(ranks, dtype=torch.int32, **dev)
        st["scales"] = torch.tensor(2.0 ** host.randint(-1, 2, n) * 1.25, dtype=torch.float32, **dev)
        st["a_ptrs"] = torch.tensor(st["A"].data_ptr() + first * (2 * K), dtype=torch.int64, **dev)
        st["b_ptrs"] = torch.tensor(st["B"].data_ptr() + first * (2 * N), dtype=torch.int64, **dev)
        order = host.permutation(n)
        if case["runs"]:  # whole sequences, one after the other
            cuts = np.sort(host.randint(0, T + 1, case["runs"] - 1))
            ids = order[np.searchsorted(cuts, np.arange(T), side="right") % n]
        else:  # a token of each request, some requests without an adapter
            ids = order[np.arange(T) % n]
            ids[7::8] = -1
        st["ids"] = torch.tensor(ids, dtype=torch.int32, **dev)
        st["x"] = normal(T, K, dtype=dt)
        if case["op"] == "lora":
            st["base"] = normal(T, N, dtype=dt)
            st["out"] = {"y": torch.empty((T, N), dtype=dt, **dev)}
        else:
            st["dy"] = normal(T, N, std=0.1, dtype=dt)
            st["base"] = normal(T, K, std=0.1, dtype=dt)
            st["out"] = {"dx": torch.empty((T, K), dtype=dt, **dev), "dA": torch.empty((sum(ranks), K), **dev), "dB": torch.empty((sum(ranks), N), **dev)}
            st["da_ptrs"] = torch.tensor(st["out"]["dA"].data_ptr() + first * (4 * K), dtype=torch.int64, **dev)
            st["db_ptrs"] = torch.tensor(st["out"]["dB"].data_ptr() + first * (4 * N), dtype=torch.int64, **dev)
    return st


def run(state):
    if own:
        return _own(state)
    return {"balance": _balance, "route_backward": _route_backward, "lora": _lora, "lora_backward": _lora_backward}[state["case"]["op"]](state)


# ---- the framework's calls ----


def _own(st):
    import block_scaled_fp4_route_amd as m

    c, o = st["case"], st["out"]
    T = c["T"]
    if c["op"] == "balance":
        if "ws" not in st:
            st["d"] = m.desc(256, 64, c["E"], c["k"], "nvfp4")
            st["ws"] = torch.empty(m.moe_balance_workspace_bytes(st["d"], T, c["S"]), dtype=torch.uint8, device="cuda")
        m.moe_balance_loss(st["d"], st["logits"], T, st["idx"], st["mask"], st["seq_off"], c["S"], *st["coef"], st["dloss"],
                           o["loss"], o["counts"], o["probs"], o["dlogits"], st["ws"])
    elif c["op"] == "route_backward":
        if "ws" not in st:
            st["d"] = m.desc(c["H"], 64, c["E"], c["k"], "nvfp4")
            st["ws"] = torch.empty(m.moe_route_backward_workspace_bytes(st["d"], T), dtype=torch.uint8, device="cuda")
        m.moe_route_backward(st["d"], st["x"], T, st["Wr"], st["idx"], st["w"], st["dw"], st["mask"], st["dlogits"],
                             o["dlogits"], o["dx"], o["dWr"], 0, st["ws"])
    else:
        K, N, back = c["K"], c["N"], c["op"] == "lora_backward"
        if "ws" not in st:
            st["l"] = m.lora_desc(K, N, c["n"], c["r"], st["x"].dtype)
            st["ws"] = torch.empty(m.moe_lora_workspace_bytes(st["l"], T, back), dtype=torch.uint8, device="cuda")
        table = (st["ids"], st["a_ptrs"], st["b_ptrs"], st["ranks"], st["scales"])
        if back:
            m.moe_lora_backward(st["l"], st["x"], K, st["dy"], N, T, *table, st["base"], K, o["dx"], K, st["da_ptrs"], st["db_ptrs"], 0, st["ws"])
        else:
            m.moe_lora_apply(st["l"], st["x"], K, T, *table, st["base"], N, o["y"], N, st["ws"])
    return o


# ---- the plain forms ----


def _balance(st):
    c = st["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    logits, off, (cb, cz) = st["logits"], st["seq_off"], st["coef"]
    t = torch.arange(T, device="cuda")
    member = (t >= off[:-1, None]) & (t < off[1:, None])  # [S][T]
    if st["mask"] is not None:
        member = member & (st["mask"] != 0)
    m32 = member.float()
    n = m32.sum(1)
    chosen = torch.zeros((T, E), device="cuda").scatter_add_(1, st["idx"].long(), torch.ones((T, k), device="cuda"))
    counts = m32 @ chosen
    top = logits.amax(1, keepdim=True)
    ex = torch.exp(logits - top)
    z = ex.sum(1, keepdim=True)
    p = ex / z
    lse = (top + torch.log(z))[:, 0]
    used = (n > 0).float()
    nn = n.clamp(min=1)[:, None]
    probs = (m32 @ p) / nn
    share = used.sum().clamp(min=1)
    coef = counts * (E / k) / nn / share  # d balance / d mean probability
    balance = (coef * probs).sum()
    counted = m32.sum(0)
    total = counted.sum().clamp(min=1)
    zloss = (counted * lse * lse).sum() / total
    per = m32.t() @ (coef / nn)  # [T][E]
    grad = cb * p * (per - (p * per).sum(1, keepdim=True)) + cz * (2 / total) * (counted * lse)[:, None] * p
    loss = torch.stack([cb * balance + cz * zloss, balance, zloss])
    return {"loss": loss, "counts": counts.to(torch.int32), "probs": probs, "dlogits": grad * st["dloss"]}


def _route_backward(st):
    keep = 1.0 if st["mask"] is None else (st["mask"] != 0).float()[:, None]
    w, dw = st["w"], st["dw"]
    dsel = w * (dw - (w * dw).sum(1, keepdim=True))
    g = (st["dlogits"].clone().scatter_add_(1, st["idx"].long(), dsel)) * keep
    return {"dlogits": g, "dx": g @ st["Wr"], "dWr": g.t() @ (st["x"] * keep)}


def _low(st, v, M):
    """scale * (M v) of each token's own adapter, zero in the columns of the others: [T][sum of ranks]."""
    u = v.float() @ M.float().t()
    mine = st["ids"][:, None] == st["owner"][None, :]
    return torch.where(mine, u * st["scales"][st["owner"]], torch.zeros((), device="cuda"))


def _lora(st):
    u = _low(st, st["x"], st["A"])
    return {"y": (st["base"].float() + u @ st["B"].float()).to(st["x"].dtype)}


def _lora_backward(st):
    u, v = _low(st, st["x"], st["A"]), _low(st, st["dy"], st["B"])
    dx = (st["base"].float() + v @ st["A"].float()).to(st["x"].dtype)
    return {"dx": dx, "dA": v.t() @ st["x"].float(), "dB": u.t() @ st["dy"].float()}


# ---- what a pass cannot do without ----


def work(case):
    T = case["T"]
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        return {"bytes": 8 * T * E + 4 * T * k + (T if case["masked"] else 0) + 4 * (S + 1) + 8 * S * E + 16, "flops": 12 * T * E}
    if case["op"] == "route_backward":
        E, k, H = case["E"], case["k"], case["H"]
        return {"bytes": 8 * T * E + 12 * T * k + 8 * E * H + 8 * T * H + (T if case["masked"] else 0), "flops": 4 * T * E * H + 5 * T * k}
    K, N, size = case["K"], case["N"], 4 if case["dtype"] == "f32" else 2
    ranks = _ranks(case)
    per = sum(ranks) / len(ranks)
    used = sum(ranks) * min(1.0, T / len(ranks))
    if case["op"] == "lora":
        return {"bytes": size * T * (K + 2 * N) + 2 * used * (K + N) + 4 * T, "flops": 2 * T * per * (K + N)}
    return {"bytes": size * T * (3 * K + N) + 2 * used * (K + N) + 4 * sum(ranks) * (K + N) + 4 * T, "flops": 2 * T * per * (3 * K + 2 * N)}


# ---- the definitions in 64 bits ----


def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        on = np.ones(T, bool) if st["mask"] is None else st["mask"].cpu().numpy() != 0
        off, idx, (cb, cz), up = st["seq_off"].tolist(), st["idx"].long(), st["coef"], float(st["dloss"][0])
        logp = torch.log_softmax(st["logits"].double(), 1)
        lse = torch.logsumexp(st["logits"].double(), 1)
        rows = [torch.from_numpy(off[s] + np.flatnonzero(on[off[s]:off[s + 1]])).cuda() for s in range(S)]
        live, every = sum(len(r) > 0 for r in rows), sum(len(r) for r in rows)
        counts, probs = torch.zeros((S, E), dtype=torch.int32, device="cuda"), torch.zeros((S, E), dtype=f8, device="cuda")
        grad, balance, zsum = torch.zeros((T, E), dtype=f8, device="cuda"), 0.0, 0.0
        for s, r in enumerate(rows):
            if not len(r):
                continue
            p = logp[r].exp()
            hits = torch.bincount(idx[r].reshape(-1), minlength=E)
            f = hits.to(f8) / (len(r) * k)
            counts[s], probs[s] = hits.to(torch.int32), p.mean(0)
            balance += float(E * (f * probs[s]).sum()) / live
            zsum += float((lse[r] ** 2).sum())
            bal = (E / (live * len(r))) * p * (f - (p @ f)[:, None])
            grad[r] = up * (cb * bal + cz * (2 / every) * lse[r][:, None] * p)
        z = zsum / every if every else 0.0
        return {"loss": torch.tensor([cb * balance + cz * z, balance, z], dtype=f8), "counts": counts, "probs": probs, "dlogits": grad}
    if case["op"] == "route_backward":
        T, k = case["T"], case["k"]
        w, dw = st["w"].double(), st["dw"].double()
        g = st["dlogits"].double()
        at, tok = st["idx"].long(), torch.arange(T, device="cuda")
        jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]  # of a softmax over the chosen
        sel = (jac * dw[:, None, :]).sum(2)
        for j in range(k):
            g[tok, at[:, j]] += sel[:, j]
        x = st["x"].double()
        if st["mask"] is not None:
            off = st["mask"] == 0
            g[off], x[off] = 0.0, 0.0
        return {"dlogits": g, "dx": torch.mm(g, st["Wr"].double()), "dWr": torch.mm(g.t().contiguous(), x)}
    ranks, ids, scales = _ranks(case), st["ids"].cpu().numpy(), st["scales"].tolist()
    out = {"dx" if case["op"] == "lora_backward" else "y": st["base"].double()}
    if case["op"] == "lora_backward":
        out["dA"], out["dB"] = torch.zeros_like(st["A"], dtype=f8), torch.zeros_like(st["B"], dtype=f8)
    first = 0
    for a, r in enumerate(ranks):
        mine = torch.from_numpy(np.flatnonzero(ids == a)).cuda()
        A, B = st["A"][first:first + r].double(), st["B"][first:first + r].double()
        x = st["x"][mine].double()
        if case["op"] == "lora":
            out["y"][mine] += scales[a] * torch.mm(torch.mm(x, A.t().contiguous()), B)
        else:
            dy = st["dy"][mine].double()
            out["dx"][mine] += scales[a] * torch.mm(torch.mm(dy, B.t().contiguous()), A)
            out["dA"][first:first + r] = scales[a] * torch.mm(torch.mm(dy, B.t().contiguous()).t().contiguous(), x)
            out["dB"][first:first + r] = scales[a] * torch.mm(torch.mm(x, A.t().contiguous()).t().contiguous(), dy)
        first += r
    return out
