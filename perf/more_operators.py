"""Cases of the operators around a routed layer that serves a few tokens, and of 4-bit matrices beside it.

Five operators, each in its plain form (elementary torch operations in fp32) and as the framework's call:

quant             a matrix to block-scaled e2m1 codes (NVFP4 or MXFP4), with the values that the codes stand for
product           activations times a matrix stored in 4 bits, the activations kept or rounded to MXFP4
product_backward  the gradient of that product's activations
layer             a whole mixture-of-experts layer for a few tokens: router, chosen experts, shared expert
norm              the norm behind a block, its gate and residual scale, and the norm before the next one; in training their gradients too
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
RES_SCALE = 0.75


def listed():
    return [
        # one expert's gate matrix, stored in 4 bits with a power of two for each row
        {"name": "quant_640x2560_nv", "op": "quant", "rows": 640, "cols": 2560, "fmt": "nvfp4", "dtype": "bf16", "ceil": False},
        # a batch of activations, rounded as a scaled product takes them
        {"name": "quant_8192x2560_mx", "op": "quant", "rows": 8192, "cols": 2560, "fmt": "mxfp4", "dtype": "f32", "ceil": False},
        # one decoded token through the 8192 x 2560 projection
        {"name": "product_1_nv_f32", "op": "product", "T": 1, "K": 2560, "N": 8192, "fmt": "nvfp4", "dtype": "f32", "round": False},
        # a 2451-token prompt, activations kept in their 16 bits
        {"name": "product_2451_nv_f16", "op": "product", "T": 2451, "K": 2560, "N": 2560, "fmt": "nvfp4", "dtype": "f16", "round": False},
        # a long prompt, both operands in 4 bits
        {"name": "product_8192_mx_bf16", "op": "product", "T": 8192, "K": 2560, "N": 8192, "fmt": "mxfp4", "dtype": "bf16", "round": True},
        # a small training batch through a frozen 640 x 2560 matrix, back to its input
        {"name": "product_backward_311_nv_f32", "op": "product_backward", "T": 311, "K": 2560, "N": 640, "fmt": "nvfp4", "dtype": "f32"},
        # a long training batch beside adapters of the 8192 x 2560 projection
        {"name": "product_backward_8192_mx_bf16", "op": "product_backward", "T": 8192, "K": 2560, "N": 8192, "fmt": "mxfp4", "dtype": "bf16"},
        # four sequences decoded side by side: 512 NVFP4 experts, ten for each token, a shared expert
        {"name": "layer_4_nv", "op": "layer", "T": 4, "H": 2560, "I": 640, "E": 512, "k": 10, "fmt": "nvfp4", "shared": True, "masked": 0},
        # a draft of 13 tokens checked at once: 384 MXFP4 experts, six for each token
        {"name": "layer_13_mx", "op": "layer", "T": 13, "H": 4096, "I": 2880, "E": 384, "k": 6, "fmt": "mxfp4", "shared": False, "masked": 0},
        # a serving batch of 48 slots, some of them empty
        {"name": "layer_48_nv", "op": "layer", "T": 48, "H": 2560, "I": 640, "E": 512, "k": 10, "fmt": "nvfp4", "shared": True, "masked": 5},
        # one decoded token between two blocks
        {"name": "norm_1", "op": "norm", "T": 1, "H": 2560, "r": "bf16", "y": "f32", "x": "f32", "gate": "token", "train": False, "masked": 0},
        # a long training step: both directions, a learned gate for each channel
        {"name": "norm_8191_train", "op": "norm", "T": 8191, "H": 4096, "r": "bf16", "y": "bf16", "x": "bf16", "gate": "channel", "train": True, "masked": 700},
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "product_backward", "layer", "layer", "norm"])
    fmt, dtype = rng.choice(["nvfp4", "mxfp4"]), rng.choice(sorted(DTYPES))
    if op == "quant":
        cols = (16 if fmt == "nvfp4" else 32) * _spread(rng, 4, 128)
        return {"op": op, "rows": min(_spread(rng, 1, 8192), 8192 * 2560 // cols), "cols": cols, "fmt": fmt, "dtype": dtype, "ceil": fmt == "mxfp4" and rng.random() < 0.5}
    if op in ("product", "product_backward"):
        case = {"op": op, "T": _spread(rng, 1, 8192), "K": 32 * _spread(rng, 8, 128), "N": 8 * _spread(rng, 32, 1024), "fmt": fmt, "dtype": dtype}
        if op == "product":
            case["round"] = fmt == "mxfp4" and rng.random() < 0.5
        big = next(c for c in listed() if c["name"] == "product_8192_mx_bf16")
        while case["T"] > 1 and (work(case)["flops"] > work(big)["flops"] or work(case)["bytes"] > work(big)["bytes"]):
            case["T"] = (case["T"] + 1) // 2
        return case
    if op == "layer":
        E = _spread(rng, 8, 512)
        case = {"op": op, "T": _spread(rng, 1, 64), "H": 512 * rng.randint(1, 8), "I": 32 * _spread(rng, 2, 40), "E": E, "k": rng.randint(1, min(E, 12)), "fmt": fmt, "shared": rng.random() < 0.5}
        while case["E"] > case["k"] and case["E"] * case["H"] * case["I"] > 512 * 2560 * 640:
            case["E"] -= 1
        while case["T"] > 1 and case["T"] * case["k"] * case["H"] * case["I"] > 48 * 10 * 2560 * 640:
            case["T"] -= 1
        case["masked"] = rng.choice([0, 0, min(3, case["T"] - 1)])
        return case
    H = 8 * _spread(rng, 32, 1024)
    T = min(_spread(rng, 1, 8191), 8191 * 4096 // max(H, 4096))
    kinds = {k: rng.choice(sorted(DTYPES)) for k in ("r", "y", "x")}
    train = rng.random() < 0.5
    if "f32" in kinds.values():
        T = (T + 1) // 2
    return {"op": op, "T": T, "H": H, **kinds, "gate": rng.choice(["none", "channel", "token"]), "train": train, "masked": rng.choice([0, T // 7])}


# ---- what a program has in hand ----


def _matrix(g, rows, cols, fmt, lo, hi):
    """A stored matrix: codes [rows][cols / 2] and scale bytes lo..hi - 1 [rows][cols / G]."""
    G = 16 if fmt == "nvfp4" else 32
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
    return codes, torch.randint(lo, hi, (rows, cols // G), dtype=torch.uint8, device="cuda", generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda"}

    def normal(*size, std=1.0, dtype=torch.float32):
        return torch.empty(size, dtype=dtype, **dev).normal_(0, std, generator=g)

    def grid(*size, step):
        """Values on a coarse grid: router logits of them are exact in fp32 in any order, so that the choice of experts is the same for everybody."""
        return normal(*size).mul_(16).round_().clamp_(-63, 63).mul_(step)

    op, st = case["op"], {"case": dict(case)}
    if op == "quant":
        rows, cols, fmt = case["rows"], case["cols"], case["fmt"]
        dt = DTYPES[case["dtype"]]
        # rows of unequal size and a few large values, as weights and activations have them
        v = normal(rows, cols) * torch.exp(normal(rows, 1)) * 0.05
        v = torch.where(torch.rand(rows, cols, generator=g, **dev) < 1e-3, 30 * v, v)
        st["x"] = v.to(dt)
        st["out"] = {"values": torch.empty((rows, cols), dtype=dt, **dev), "codes": torch.empty((rows, cols // 2), dtype=torch.uint8, **dev),
                     "scales": torch.empty((rows, cols // (16 if fmt == "nvfp4" else 32)), dtype=torch.uint8, **dev)}
        if fmt == "nvfp4":
            st["out"]["row_exp"] = torch.empty(rows, dtype=torch.int8, **dev)
    elif op in ("product", "product_backward"):
        T, K, N, dt = case["T"], case["K"], case["N"], DTYPES[case["dtype"]]
        st["codes"], st["scales"] = _matrix(g, N, K, case["fmt"], *((0x18, 0x49) if case["fmt"] == "nvfp4" else (115, 124)))
        st["row_exp"] = torch.randint(-8, -4, (N,), dtype=torch.int8, generator=g, **dev) if case["fmt"] == "nvfp4" else None
        if op == "product":
            st["x"] = normal(T, K, dtype=dt)
            st["out"] = {"y": torch.empty((T, N), dtype=dt, **dev)}
        else:
            st["dy"] = normal(T, N, std=0.1, dtype=dt)
            st["base"] = normal(T, K, std=0.1, dtype=dt)
            st["out"] = {"dx": torch.empty((T, K), dtype=dt, **dev)}
    elif op == "layer":
        T, H, I, E, k, fmt = case["T"], case["H"], case["I"], case["E"], case["k"], case["fmt"]
        G = 16 if fmt == "nvfp4" else 32
        n = 3 * H * I
        st["blocks"] = torch.empty((E, n // 2 + n // G), dtype=torch.uint8, **dev)
        st["blocks"][:, :n // 2].random_(0, 256, generator=g)
        lo, hi = (0x18, 0x49) if fmt == "nvfp4" else (121, 130)
        st["blocks"][:, n // 2:].random_(lo, hi, generator=g)
        st["table"] = st["blocks"].data_ptr() + torch.arange(E, dtype=torch.int64, **dev) * st["blocks"].shape[1]
        st["x"], st["Wr"] = grid(T, H, step=1 / 256), grid(E, H, step=1 / 64)
        st["shared"] = None
        if case["shared"]:
            st["shared"] = tuple(normal(*s, std=1.0, dtype=torch.bfloat16) for s in ((I, H), (I, H), (H, I)))
        st["mask"] = None
        if case["masked"]:
            st["mask"] = torch.ones(T, dtype=torch.uint8, **dev)
            st["mask"][torch.randperm(T, generator=g, **dev)[:case["masked"]]] = 0
        st["out"] = {"y": torch.full((T, H), 7.0, **dev), "idx": torch.zeros((T, k), dtype=torch.int32, **dev), "w": torch.zeros((T, k), **dev)}
    else:
        T, H = case["T"], case["H"]
        r, y, x = (DTYPES[case[k]] for k in ("r", "y", "x"))
        st["r"], st["y"] = normal(T, H, std=2.0, dtype=r), normal(T, H, std=30.0, dtype=y)
        st["post"], st["pre"] = 1 + normal(H, std=0.1), 1 + normal(H, std=0.1)
        st["gate"] = {"none": None, "channel": normal(H, std=0.5), "token": torch.sigmoid(normal(T))}[case["gate"]]
        st["mask"] = None
        if case["masked"]:  # slots behind the last sequence
            st["mask"] = (torch.arange(T, **dev) < T - case["masked"]).to(torch.uint8)
        st["out"] = {"r": torch.zeros((T, H), dtype=r, **dev), "x": torch.zeros((T, H), dtype=x, **dev)}
        if case["train"]:
            st["dr_out"], st["dx"] = normal(T, H, std=0.1, dtype=r), normal(T, H, std=0.1, dtype=x)
            st["grad"] = {"dr": torch.empty((T, H), dtype=r, **dev), "dy": torch.empty((T, H), dtype=y, **dev),
                          "dpost": torch.empty(H, **dev), "dpre": torch.empty(H, **dev)}
            if st["gate"] is not None:
                st["grad"]["dgate"] = torch.empty_like(st["gate"])
    return st


def run(state):
    if own:
        return _own(state)
    return {"quant": _quant, "product": _product, "product_backward": _product_backward, "layer": _layer, "norm": _norm}[state["case"]["op"]](state)


# ---- the framework's calls ----


def _workspace(n):
    return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")


def _own(st):
    import block_scaled_fp4_route_amd as m

    c, o = st["case"], st["out"]
    if c["op"] == "quant":
        rows, cols, nv = c["rows"], c["cols"], c["fmt"] == "nvfp4"
        rule = m.MOE_SCALE_NEAREST if nv else m.MOE_SCALE_CEIL if c["ceil"] else m.MOE_SCALE_FLOOR
        m.moe_fp4_quant(st["x"], cols, rows, cols, st["x"].dtype, c["fmt"], rule, o.get("row_exp"), o["codes"], o["scales"], o["values"], cols)
        kind = torch.float8_e4m3fn if nv else torch.float8_e8m0fnu
        return {"values": o["values"], "scales": o["scales"].view(kind), "row_exp": o.get("row_exp")}
    if c["op"] in ("product", "product_backward"):
        T, K, N, back = c["T"], c["K"], c["N"], c["op"] == "product_backward"
        if "ws" not in st:
            st["f"] = m.fp4_desc(K, N, c["fmt"], DTYPES[c["dtype"]])
            st["ws"] = _workspace(m.moe_fp4_workspace_bytes(st["f"], T, back))
        if back:
            m.moe_fp4_backward(st["f"], st["dy"], N, T, st["codes"], st["scales"], st["row_exp"], st["base"], K, o["dx"], K, st["ws"])
        else:
            m.moe_fp4_apply(st["f"], st["x"], K, T, st["codes"], st["scales"], st["row_exp"], c["round"], None, 0, o["y"], N, st["ws"])
        return o
    if c["op"] == "layer":
        if "ws" not in st:
            st["d"] = m.desc(c["H"], c["I"], c["E"], c["k"], c["fmt"])
            st["ws"] = _workspace(m.moe_workspace_bytes(st["d"], c["T"], m.MOE_MODE_DECODE_BATCH))
        m.moe_layer_decode_batch(st["d"], st["x"], c["T"], st["mask"], st["Wr"], st["table"], st["shared"], o["y"], o["idx"], o["w"], st["ws"])
        return o
    T, H = c["T"], c["H"]
    if "n" not in st:
        st["n"] = m.norm_desc(H, st["r"].dtype, st["y"].dtype, o["x"].dtype, c["gate"], RES_SCALE, EPS)
        st["ws"] = _workspace(m.moe_block_norm_workspace_bytes(st["n"], T) if c["train"] else 0)
    m.moe_block_norm(st["n"], st["r"], H, st["y"], H, T, st["mask"], st["post"], st["gate"], st["pre"], o["r"], H, o["x"], H)
    if not c["train"]:
        return o
    q = st["grad"]
    m.moe_block_norm_backward(st["n"], o["r"], H, st["y"], H, T, st["mask"], st["post"], st["gate"], st["pre"], st["dr_out"], H, st["dx"], H,
                              q["dr"], H, q["dy"], H, q["dpost"], q.get("dgate"), q["dpre"], 0, st["ws"])
    return {**o, **q}


# ---- the plain forms ----


def _pow2(e):
    """2^e in fp32 for whole e of -126..127, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _code_values():
    m = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    return torch.cat([m, -m])


def _values(codes, scales, fmt):
    """The stored matrices' values in fp32, [..., cols] from [..., cols / 2] bytes."""
    v, b = _code_values(), torch.arange(256, device="cuda")
    table = torch.stack([v[b % 16], v[b // 16]], dim=1)
    out = torch.index_select(table, 0, codes.reshape(-1).to(torch.int32))
    s = scales.view(torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu).float()
    return (out.view(*scales.shape, -1) * s[..., None]).view(*codes.shape[:-1], -1)


def _round_codes(t, s):
    """The magnitudes that |t| / s rounds to (nearest, ties to the even code, at most 6), without dividing: a border times s is exact."""
    m, one = _code_values(), s[..., None]
    n = (t > 0.25 * one).int() + (t >= 0.75 * one) + (t > 1.25 * one) + (t >= 1.75 * one) + (t > 2.5 * one) + (t >= 3.5 * one) + (t > 5.0 * one)
    return torch.where(one > 0, m[n], torch.zeros((), device="cuda"))


def _mx(x, ceil):
    """x [rows][cols] in fp32 rounded to MXFP4: the values, and the exponents of the blocks."""
    v = x.view(x.shape[0], -1, 32)
    bits = v.abs().amax(2).view(torch.int32)
    e = (bits >> 23) - 129
    if ceil:  # the smallest exponent with the largest value at most 6 times 2^e
        e = e + ((bits & 0x7FFFFF) > 0x400000)
    e = torch.where(bits == 0, -127, e.clamp(-127, 125))
    s = _pow2(e.clamp(min=-126))
    return (torch.copysign(_round_codes(v.abs(), s), v) * s[..., None]).view_as(x), e


def _nv(x):
    """x in fp32 rounded to NVFP4 with a power of two for each row: values, scales and the rows' exponents."""
    bits = x.abs().amax(1).view(torch.int32)
    e = (bits >> 23) - 138 + ((bits & 0x7FFFFF) > 0x280000).int()
    e = torch.where(bits == 0, 0, e.clamp(-100, 116))
    v = (x * _pow2(-e)[:, None]).view(x.shape[0], -1, 16)
    s = (v.abs().amax(2).double() / 6).float().clamp(max=448.0).to(torch.float8_e4m3fn)  # a sixth lies on a border often
    q = torch.copysign(_round_codes(v.abs(), s.float()), v) * s.float()[..., None]
    return q.view_as(x) * _pow2(e)[:, None], s, e


def _quant(st):
    c, x = st["case"], st["x"].float()
    top = torch.finfo(st["x"].dtype).max
    if c["fmt"] == "nvfp4":
        v, s, e = _nv(x)
        return {"values": v.clamp(-top, top).to(st["x"].dtype), "scales": s, "row_exp": e.to(torch.int8)}
    v, e = _mx(x, c["ceil"])
    return {"values": v.clamp(-top, top).to(st["x"].dtype), "scales": (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu), "row_exp": None}


def _weights(st):
    w = _values(st["codes"], st["scales"], st["case"]["fmt"])
    return w if st["row_exp"] is None else w * _pow2(st["row_exp"])[:, None]


def _product(st):
    x = st["x"].float()
    if st["case"]["round"]:
        x = _mx(x, False)[0]
    return {"y": (x @ _weights(st).t()).to(st["x"].dtype)}


def _product_backward(st):
    return {"dx": (st["base"].float() + st["dy"].float() @ _weights(st)).to(st["dy"].dtype)}


def _layer(st):
    c, x = st["case"], st["x"]
    T, H, I, k, fmt = c["T"], c["H"], c["I"], c["k"], c["fmt"]
    G, n = (16 if fmt == "nvfp4" else 32), H * I
    top = torch.sort(x @ st["Wr"].t(), dim=1, descending=True, stable=True)
    idx, l = top.indices[:, :k], top.values[:, :k]
    ex = torch.exp(l - l[:, :1])
    w = ex / ex.sum(1, keepdim=True)
    mine = st["blocks"][idx.reshape(-1)]  # [T k][block bytes]

    def product(i, v):
        """Matrix i of every chosen expert times its row of v."""
        rows, cols = (H, I) if i == 2 else (I, H)
        codes = mine[:, i * n // 2:(i + 1) * n // 2].reshape(T * k, rows, cols // 2)
        at = 3 * n // 2 + i * (n // G)
        scales = mine[:, at:at + n // G].reshape(T * k, rows, cols // G)
        return torch.bmm(_values(codes, scales, fmt), v[:, :, None])[:, :, 0]

    xs = x.repeat_interleave(k, 0)
    a = product(0, xs)
    h = a / (1 + torch.exp(-a)) * product(1, xs)
    y = (product(2, h).view(T, k, H) * w[:, :, None]).sum(1)
    if st["shared"] is not None:
        gate, up, down = (s.float() for s in st["shared"])
        a = x @ gate.t()
        y = y + (a / (1 + torch.exp(-a)) * (x @ up.t())) @ down.t()
    o = st["out"]
    on = torch.ones((T, 1), dtype=torch.bool, device="cuda") if st["mask"] is None else (st["mask"] != 0)[:, None]
    return {"y": torch.where(on, y, o["y"]), "idx": torch.where(on, idx.to(torch.int32), o["idx"]), "w": torch.where(on, w, o["w"])}


def _gates(st, like):
    gate = st["gate"]
    if gate is None:
        return torch.ones((1, 1), dtype=like, device="cuda")
    return gate.to(like)[None, :] if st["case"]["gate"] == "channel" else gate.to(like)[:, None]


def _norm(st):
    c = st["case"]
    f4 = torch.float32
    on = torch.ones((c["T"], 1), dtype=torch.bool, device="cuda") if st["mask"] is None else (st["mask"] != 0)[:, None]
    y = st["y"].float()
    gate = RES_SCALE * _gates(st, f4)
    rs_y = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    unit = y * rs_y
    r = st["r"].float() + gate * (unit * st["post"])
    x = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * st["pre"]
    o = st["out"]
    out = {"r": torch.where(on, r.to(o["r"].dtype), o["r"]), "x": torch.where(on, x.to(o["x"].dtype), o["x"])}
    if not c["train"]:
        return out
    r = out["r"].float()
    rs_r = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    dx = st["dx"].float()
    a = dx * st["pre"]
    d = st["dr_out"].float() + rs_r * (a - r * (rs_r * rs_r * (a * r).mean(1, keepdim=True)))
    d = torch.where(on, d, torch.zeros((), device="cuda"))
    out["dr"], out["dpre"] = d.to(o["r"].dtype), torch.where(on, dx * r * rs_r, 0.0).sum(0)
    u = gate * d
    out["dpost"] = (u * unit).sum(0)
    u = u * st["post"]
    out["dy"] = (rs_y * (u - unit * (u * unit).mean(1, keepdim=True))).to(st["y"].dtype)
    if c["gate"] != "none":
        out["dgate"] = (RES_SCALE * d * unit * st["post"]).sum(0 if c["gate"] == "channel" else 1)
    return out


# ---- what a pass cannot do without ----


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] == "quant":
        n, G = case["rows"] * case["cols"], 16 if case["fmt"] == "nvfp4" else 32
        return {"bytes": n * (2 * size[case["dtype"]] + 0.5) + n / G + (case["rows"] if G == 16 else 0), "flops": 4 * n}
    if case["op"] in ("product", "product_backward"):
        T, K, N, s = case["T"], case["K"], case["N"], size[case["dtype"]]
        matrix = N * K / 2 + N * K / (16 if case["fmt"] == "nvfp4" else 32) + (N if case["fmt"] == "nvfp4" else 0)
        return {"bytes": matrix + s * T * (K + N + (K if case["op"] == "product_backward" else 0)), "flops": 2 * T * K * N}
    if case["op"] == "layer":
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        T -= case["masked"]
        used = E * (1 - (1 - k / E) ** T)  # experts that some token chooses, where the router has no favourites
        block = 3 * H * I / 2 + 3 * H * I / (16 if case["fmt"] == "nvfp4" else 32)
        return {"bytes": used * block + 4 * E * H + 8 * T * H + 8 * T * k + (6 * H * I if case["shared"] else 0),
                "flops": 6 * T * (k + (1 if case["shared"] else 0)) * H * I + 2 * T * E * H}
    n = (case["T"] - case["masked"]) * case["H"]
    r, y, x = (size[case[k]] for k in ("r", "y", "x"))
    if not case["train"]:
        return {"bytes": n * (2 * r + y + x) + 8 * case["H"], "flops": 12 * n}
    return {"bytes": n * (2 * r + y + x) + n * (3 * r + 2 * y + x) + 20 * case["H"], "flops": 40 * n}


# ---- the definitions in 64 bits ----


def _two(e):
    """2^e in fp64 for whole e, from its bits (pow() is an ulp off for some)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _decoded(codes, scales, fmt):
    """codes [rows][cols / 2], scales [rows][cols / G] -> fp64 [rows][cols]."""
    n = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(codes.shape[0], -1).to(torch.int64)
    mag, e = (n & 1).double(), (n >> 1) & 3
    v = torch.where(e == 0, 0.5 * mag, (1 + 0.5 * mag) * _two(e - 1))
    v = torch.where(n >= 8, -v, v)
    b = scales.to(torch.int64)
    if fmt == "nvfp4":
        ex, mant = (b >> 3) & 15, (b & 7).double()
        s = torch.where(ex == 0, mant / 8 * 2.0 ** -6, (1 + mant / 8) * _two(ex - 7))
        s = torch.where(b >= 128, -s, s)
    else:
        s = _two(b - 127)
    return v * s.repeat_interleave(v.shape[1] // s.shape[1], dim=1)


def _nearest(t):
    """|t| to the nearest of the eight magnitudes, ties to the even code."""
    even = torch.tensor([0.0, 1.0, 2.0, 4.0], dtype=torch.float64, device="cuda")
    odd = torch.tensor([0.5, 1.5, 3.0, 6.0], dtype=torch.float64, device="cuda")
    de, we = (t[..., None] - even).abs().min(-1)
    do, wo = (t[..., None] - odd).abs().min(-1)
    return torch.where(de <= do, even[we], odd[wo])


def _rounded_mx(x, ceil):
    v = x.double().view(x.shape[0], -1, 32)
    top = v.abs().amax(2)
    m, p = torch.frexp(top)  # top = m 2^p, m in [0.5, 1)
    e = (p + torch.where(m > 0.75, 1, 0) - 3) if ceil else p - 3
    e = torch.where(top == 0, torch.full_like(e, -127), e.clamp(-127, 125))
    s = _two(e)[..., None]
    return (torch.sign(v) * _nearest(v.abs() / s) * s).view(x.shape), _two(e)


def exact(case, seed):
    st = prepare(case, seed)
    op, f8 = case["op"], torch.float64
    if op == "quant":
        if case["fmt"] == "mxfp4":
            v, s = _rounded_mx(st["x"], case["ceil"])
            return {"values": v, "scales": s, "row_exp": None}
        x = st["x"].double()
        top = x.abs().amax(1)
        e = torch.ceil(torch.log2(top / 2688)).clamp(-100, 116)
        v = (x * _two(-e)[:, None]).view(x.shape[0], -1, 16)
        grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
        want = v.abs().amax(2) / 6
        up = torch.searchsorted(grid, want.contiguous()).clamp(max=126)
        lo = (up - 1).clamp(min=0)
        a, b = want - grid[lo], grid[up] - want
        s = grid[torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, up)]
        q = torch.where(s[..., None] > 0, torch.sign(v) * _nearest(v.abs() / s.clamp(min=2.0 ** -9)[..., None]) * s[..., None], 0.0)
        return {"values": q.view(x.shape) * _two(e)[:, None], "scales": s, "row_exp": None}
    if op in ("product", "product_backward"):
        w = _decoded(st["codes"], st["scales"], case["fmt"])
        if st["row_exp"] is not None:
            w = w * _two(st["row_exp"])[:, None]
        if op == "product":
            x = _rounded_mx(st["x"], False)[0] if case["round"] else st["x"].double()
            return {"y": torch.mm(x, w.t().contiguous())}
        return {"dx": st["base"].double() + torch.mm(st["dy"].double(), w)}
    if op == "layer":
        T, H, I, E, k, fmt = (case[n] for n in ("T", "H", "I", "E", "k", "fmt"))
        G, n = 16 if fmt == "nvfp4" else 32, H * I
        x, o = st["x"].double(), st["out"]
        logits = torch.mm(x, st["Wr"].double().t().contiguous()).cpu()
        y, wts = o["y"].double(), o["w"].double()
        for t in range(T):
            if st["mask"] is not None and not int(st["mask"][t]):
                continue
            best = sorted(range(E), key=lambda e: (-float(logits[t, e]), e))[:k]
            wts[t] = torch.softmax(logits[t, best], 0).cuda()
            y[t] = 0
            for j, e in enumerate(best):
                b, mats = st["blocks"][e], []
                for i, (rows, cols) in enumerate(((I, H), (I, H), (H, I))):
                    at = 3 * n // 2 + i * (n // G)
                    mats.append(_decoded(b[i * n // 2:(i + 1) * n // 2].view(rows, cols // 2), b[at:at + n // G].view(rows, cols // G), fmt))
                h = torch.mv(mats[0], x[t])
                h = h * torch.sigmoid(h) * torch.mv(mats[1], x[t])
                y[t] += wts[t, j] * torch.mv(mats[2], h)
            if st["shared"] is not None:
                gate, up, down = (s.double() for s in st["shared"])
                h = torch.mv(gate, x[t])
                y[t] += torch.mv(down, h * torch.sigmoid(h) * torch.mv(up, x[t]))
        return {"y": y, "idx": None, "w": wts}
    T, H, o = case["T"], case["H"], st["out"]
    rows = torch.arange(T, device="cuda") if st["mask"] is None else torch.nonzero(st["mask"])[:, 0]
    y, post, pre = st["y"][rows].double(), st["post"].double(), st["pre"].double()
    gate = torch.ones((1, 1), dtype=f8, device="cuda")
    if case["gate"] == "channel":
        gate = st["gate"].double()[None, :]
    elif case["gate"] == "token":
        gate = st["gate"][rows].double()[:, None]
    len_y = ((y * y).sum(1, keepdim=True) / H + EPS).sqrt()
    p = y / len_y * post
    r = st["r"][rows].double() + RES_SCALE * gate * p
    out = {"r": o["r"].double(), "x": o["x"].double()}
    out["r"][rows] = r
    out["x"][rows] = r / ((r * r).sum(1, keepdim=True) / H + EPS).sqrt() * pre
    if not case["train"]:
        return out
    r = r.to(o["r"].dtype).double()  # the backward pass starts from the stored sum
    len_r = ((r * r).sum(1, keepdim=True) / H + EPS).sqrt()
    n, dx = r / len_r, st["dx"][rows].double()
    d = st["dr_out"][rows].double() + (dx * pre - n * (dx * pre * n).sum(1, keepdim=True) / H) / len_r
    dn = RES_SCALE * gate * d
    g = dn * post
    ny = y / len_y
    out["dr"], out["dy"] = torch.zeros((T, H), dtype=f8, device="cuda"), torch.zeros((T, H), dtype=f8, device="cuda")
    out["dr"][rows] = d
    out["dy"][rows] = (g - ny * (g * ny).sum(1, keepdim=True) / H) / len_y
    out["dpost"], out["dpre"] = (dn * ny).sum(0), (dx * n).sum(0)
    if case["gate"] == "channel":
        out["dgate"] = (RES_SCALE * d * p).sum(0)
    elif case["gate"] == "token":
        out["dgate"] = torch.zeros(T, dtype=f8, device="cuda")
        out["dgate"][rows] = (RES_SCALE * d * p).sum(1)
    return out
