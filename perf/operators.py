"""Measured cases of the decode-step operators around the 4-bit experts: the
residual addition with RMSNorm and a Q8_1 output, SwiGLU with a Q8_1 output, the
routing of tokens to experts, and the products of Q8_1 activations with 4-bit
weights that carry group scales, for one matrix and for the experts a router
chose.

`run` computes a case in its plain form (elementary torch operations) or, where
`own` is set, through the package's entry points. `exact` computes the same from
the definitions in 64 bits.

Definitions used below
  Q8_1 block of 32 values v: d = max|v| / 127, q = rint(v / d) (by the product
  with 1 / d), 36 bytes [fp16 d][fp16 d * sum(q)][int8 q[32]].
  4-bit weights with group scales: w[m, k] = s[m, k // G] * (c[m, k] - z[m, k // G]),
  c the 4-bit codes (two to a byte, the even k in the low half), z = 8 where no
  zero points are given.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # One token enters a layer of width 4096 in the library's fp32: the call's latency.
        {"name": "norm decode", "op": "norm", "N": 1, "K": 4096, "dtype": "fp32", "residual": True, "y": True, "pad": 0},
        # A prompt of 4099 tokens, bf16, with the normed rows for the router and the Q8_1 rows for the experts.
        {"name": "norm prompt", "op": "norm", "N": 4099, "K": 4096, "dtype": "bf16", "residual": True, "y": True, "pad": 0},
        # The eight experts' gate and up rows of one token, between the two expert products.
        {"name": "swiglu decode", "op": "swiglu", "N": 8, "K": 768, "dtype": "fp32"},
        # A dense layer's gate and up rows for a prompt: the two halves of one bf16 buffer.
        {"name": "swiglu prompt", "op": "swiglu", "N": 2048, "K": 14336, "dtype": "bf16"},
        # One token over 128 experts, top 8: the call's latency.
        {"name": "route decode", "op": "route", "T": 1, "E": 128, "top_k": 8, "score": "softmax", "bias": False,
         "n_groups": 1, "topk_groups": 1, "group_top": 1, "renorm": True, "scale": 1.0, "dtype": "fp32", "masked": 0},
        # 1024 tokens over 128 experts, top 8, five experts out of service.
        {"name": "route batch", "op": "route", "T": 1024, "E": 128, "top_k": 8, "score": "softmax", "bias": False,
         "n_groups": 1, "topk_groups": 1, "group_top": 1, "renorm": True, "scale": 1.0, "dtype": "fp32", "masked": 5},
        # A long prompt over 384 experts in 12 groups of which 4 are kept, sigmoid scores with a balance bias.
        {"name": "route groups", "op": "route", "T": 8192, "E": 384, "top_k": 6, "score": "sigmoid", "bias": True,
         "n_groups": 12, "topk_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5, "dtype": "bf16", "masked": 0},
        # An attention projection for one token.
        {"name": "g4 4096x4096", "op": "g4", "N": 1, "M": 4096, "K": 4096, "G": 128, "scales": "fp16", "zeros": False},
        # A feed-forward matrix for a batch of 16 sequences, small groups with zero points.
        {"name": "g4 14336x4096 n16", "op": "g4", "N": 16, "M": 14336, "K": 4096, "G": 32, "scales": "bf16", "zeros": True},
        # The output projection over a vocabulary of 152064 for one token.
        {"name": "g4 152064x3584", "op": "g4", "N": 1, "M": 152064, "K": 3584, "G": 128, "scales": "fp16", "zeros": False},
        # Gate and up of the eight experts (768 wide) of one token: eight matrices of 128 are read.
        {"name": "moe up t1", "op": "moe", "T": 1, "E": 128, "top_k": 8, "M": 1536, "K": 2048, "G": 128,
         "scales": "fp16", "zeros": False, "per_slot": False},
        # The down product for 64 sequences: nearly every expert is read, with a row for each slot.
        {"name": "moe down t64", "op": "moe", "T": 64, "E": 128, "top_k": 8, "M": 2048, "K": 768, "G": 32,
         "scales": "bf16", "zeros": True, "per_slot": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _blocks_wide(rng, lo, hi):
    """A width of whole 32-element blocks, odd counts among them."""
    n = _log(rng, lo, hi)
    return 32 * (n if n != 96 else 97)


def draw(rng):
    op = rng.choice(["norm", "swiglu", "route", "g4", "moe"])
    if op == "norm":
        K = _blocks_wide(rng, 4, 448)
        N = _log(rng, 1, max(1, min(8192, 4099 * 4096 // K)))
        return {"op": op, "N": N, "K": K, "dtype": rng.choice(["fp32", "fp16", "bf16"]) if N * K <= 1 << 23 else "bf16",
                "residual": rng.random() < 0.8, "y": rng.random() < 0.5, "pad": rng.choice([0, 0, 64, 1])}
    if op == "swiglu":
        K = _blocks_wide(rng, 4, 448)
        N = _log(rng, 1, max(1, min(8192, 2048 * 14336 // K)))
        return {"op": op, "N": N, "K": K, "dtype": rng.choice(["fp32", "fp16", "bf16"]) if N * K <= 1 << 23 else "bf16"}
    if op == "route":
        n_groups = rng.choice([1, 1, 2, 4, 6, 8, 16])
        E = n_groups * rng.randint(max(2, 8 // n_groups), 512 // n_groups)
        topk_groups = rng.randint(1, n_groups)
        top_k = rng.randint(1, min(12, topk_groups * (E // n_groups)))
        dtype = rng.choice(["fp32", "fp16", "bf16"])
        most = 8192 * 384 * 2 // ((4 if dtype == "fp32" else 2) * (E + 4 * top_k))
        return {"op": op, "T": _log(rng, 1, min(8192, most)), "E": E, "top_k": top_k, "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "n_groups": n_groups, "topk_groups": topk_groups, "group_top": rng.choice([1, 2]),
                "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]), "dtype": dtype,
                "masked": rng.choice([0, 0, 1, E // 3])}
    G = rng.choice([32, 64, 128, 256, 1 << 20])
    more = {"G": G, "scales": rng.choice(["fp16", "bf16"]), "zeros": rng.random() < 0.5}
    if op == "g4":
        N = _log(rng, 1, 16)
        K = _blocks_wide(rng, 8, 592)
        most = 14336 * 4096 * 16 // N if N > 1 else 152064 * 3584
        return {"op": op, "N": N, "M": _log(rng, 16, min(152064, most // K)), "K": K, **more}
    T, E = _log(rng, 1, 64), _log(rng, 8, 160)
    top_k = rng.randint(1, 8)
    K = _blocks_wide(rng, 8, 128)
    most = 64 * 8 * 2048 * 768 // (T * top_k * K)
    all_of = 128 * 2048 * 768 // (E * K)
    return {"op": op, "T": T, "E": E, "top_k": top_k, "M": _log(rng, 16, max(17, min(4096, most, all_of))), "K": K,
            "per_slot": rng.random() < 0.5, **more}


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, N, K):
    """Rows of about unit size in which a few channels are large, as a model's residual stream has them."""
    x = _randn(gen, N, K)
    big = torch.rand(K, generator=gen, device="cuda") < 0.01
    return torch.where(big, 8.0 * x, x)


def _blocks(x):
    """fp32 [N, K] -> Q8_1 blocks, uint8 [N, K / 32, 36]."""
    v = x.reshape(x.shape[0], -1, 32)
    d, q = _codes(v)
    d = d.to(torch.float16)
    s = (d.float() * q.sum(-1, keepdim=True)).to(torch.float16)
    return torch.cat([d.view(torch.uint8), s.view(torch.uint8), q.to(torch.int8).view(torch.uint8)], -1).contiguous()


def _weights(gen, rows, K, case):
    groups = -(-K // case["G"])
    W = torch.randint(0, 256, (rows, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s = (0.02 * torch.exp(0.25 * _randn(gen, rows, groups))).to(DTYPES[case["scales"]])
    z = torch.randint(5, 11, (rows, groups), generator=gen, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    return {"W": W, "scales": s, "zeros": z}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "norm":
        N, K, t = case["N"], case["K"], DTYPES[case["dtype"]]
        st["X"] = _activations(gen, N, K + case["pad"]).to(t)[:, :K]
        st["R"] = (2.0 * _activations(gen, N, K)).to(t) if case["residual"] else None
        st["gamma"] = 1.0 + 0.2 * _randn(gen, K)
    elif op == "swiglu":
        gu = _randn(gen, case["N"], 2 * case["K"]).to(DTYPES[case["dtype"]])
        st["gate"], st["up"] = gu[:, :case["K"]], gu[:, case["K"]:]
    elif op == "route":
        x = (1.5 * _randn(gen, case["T"], case["E"])).to(DTYPES[case["dtype"]])
        if case["masked"]:  # experts out of service, the same for all tokens
            x[:, torch.randperm(case["E"], generator=gen, device="cuda")[:case["masked"]]] = float("-inf")
        st["logits"] = x
        # A balance bias as its update makes it: a whole number of small steps.
        st["bias"] = 1e-3 * torch.round(20 * _randn(gen, case["E"])) if case["bias"] else None
    elif op == "g4":
        st.update(_weights(gen, case["M"], case["K"], case))
        st["Xq"] = _blocks(_activations(gen, case["N"], case["K"]))
    else:
        T, E, top_k = case["T"], case["E"], case["top_k"]
        st.update(_weights(gen, E * case["M"], case["K"], case))
        st["Xq"] = _blocks(_activations(gen, T * top_k if case["per_slot"] else T, case["K"]))
        st["ids"] = torch.topk(_randn(gen, T, E), top_k, dim=1).indices.to(torch.int32).contiguous()
    return st


# ---- plain form ---------------------------------------------------------------

def _codes(v):
    """The scales (fp32) and codes (whole numbers in fp32) of Q8_1 blocks v [..., 32]."""
    d = v.abs().amax(-1, keepdim=True) / 127.0
    inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    return d, torch.clamp(torch.round(v * inv), -128, 127)


def _q8_values(v, N, K):
    """What the Q8_1 blocks of fp32 rows v stand for, and their block sums, as `_of_blocks` gives them."""
    d, q = _codes(v.reshape(N, K // 32, 32))
    d = d.to(torch.float16)
    return q.to(torch.float16) * d, (d.float() * q.sum(-1, keepdim=True)).to(torch.float16)


def _of_blocks(Xq):
    """Q8_1 blocks as the values that they stand for (fp16, the type of their scales) and their block sums."""
    h = Xq.view(torch.float16)
    return Xq.view(torch.int8).narrow(-1, 4, 32) * h.narrow(-1, 0, 1), h.narrow(-1, 1, 1)


def _plain_norm(st):
    case = st["case"]
    h = st["X"].float()
    out = {}
    if st["R"] is not None:
        h = h + st["R"].float()
        out["H"] = h.to(st["X"].dtype)
    r = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    y = h * r * st["gamma"]
    if case["y"]:
        out["Y"] = y.to(st["X"].dtype)
    out["Xq"], out["sums"] = _q8_values(y, case["N"], case["K"])
    return out


def _plain_swiglu(st):
    g, u = st["gate"].float(), st["up"].float()
    v, s = _q8_values(g / (1.0 + torch.exp(-g)) * u, st["case"]["N"], st["case"]["K"])
    return {"Xq": v, "sums": s}


def _plain_route(st):
    # In 64 bits: with a bias the order goes by sums whose neighbours can be closer than 32 bits tell apart.
    case = st["case"]
    x = st["logits"].double()
    T, E = x.shape
    low = torch.full_like(x, float("-inf"))
    off = x == float("-inf")
    if case["score"] == "softmax":
        e = torch.exp(x - x.amax(-1, keepdim=True))
        s = e / e.sum(-1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    key = torch.where(off, low, s if st["bias"] is None else s + st["bias"].double())
    order = torch.where(off, low, x) if st["bias"] is None else key  # without a bias the logits have the scores' order, exactly
    if case["topk_groups"] < case["n_groups"]:
        by = key.reshape(T, case["n_groups"], -1)
        best = torch.sort(by, dim=-1, descending=True).values[..., :case["group_top"]]
        got = torch.where(best == float("-inf"), torch.zeros_like(best), best).sum(-1)
        got = torch.where(best[..., 0] == float("-inf"), torch.full_like(got, float("-inf")), got)
        rank = torch.sort(got, dim=-1, descending=True, stable=True).indices.argsort(-1)
        order = torch.where((rank < case["topk_groups"]).repeat_interleave(E // case["n_groups"], 1), order, low)
    val, idx = torch.sort(order, dim=-1, descending=True, stable=True)
    idx = idx[:, :case["top_k"]]
    w = torch.where(val[:, :case["top_k"]] == float("-inf"), torch.zeros_like(val[:, :case["top_k"]]), s.gather(1, idx))
    if case["renorm"]:
        t = w.sum(-1, keepdim=True)
        w = torch.where(t > 0, w / t, torch.zeros_like(w))
    return {"ids": idx.to(torch.int32), "probs": (w * case["scale"]).float()}


def _plain_x(Xq):
    return (Xq[..., 4:].view(torch.int8).float() * Xq[..., 0:2].view(torch.float16).float()).reshape(Xq.shape[0], -1)


def _plain_w(st, rows, K):
    G = min(st["case"]["G"], 32 * (-(-K // 32)))
    c = torch.stack([st["W"] & 15, st["W"] >> 4], -1).reshape(rows, K).float()
    s = st["scales"].float().repeat_interleave(G, 1)[:, :K]
    z = 8.0 if st["zeros"] is None else st["zeros"].float().repeat_interleave(G, 1)[:, :K]
    return s * (c - z)


def _plain_g4(st):
    return _plain_x(st["Xq"]) @ _plain_w(st, st["case"]["M"], st["case"]["K"]).T


def _plain_moe(st):
    case = st["case"]
    E, M, K, T, top_k = case["E"], case["M"], case["K"], case["T"], case["top_k"]
    w = _plain_w(st, E * M, K).reshape(E, M, K)[st["ids"].reshape(-1).long()]
    x = _plain_x(st["Xq"])
    x = x if case["per_slot"] else x.repeat_interleave(top_k, 0)
    return torch.bmm(w, x[:, :, None]).reshape(T, top_k, M)


def _own(st):
    import quantized_weight_matmul_q4_gb300 as kq

    case, op = st["case"], st["case"]["op"]
    if op == "norm":
        H, Y, Xq = kq.kq_add_rmsnorm_q8_1(st["X"], st["R"], st["gamma"], EPS, Y=case["y"])
        v, s = _of_blocks(Xq)
        out = {"Xq": v, "sums": s}
        if H is not None:
            out["H"] = H
        if Y is not None:
            out["Y"] = Y
        return out
    if op == "swiglu":
        v, s = _of_blocks(kq.kq_swiglu_q8_1(st["gate"], st["up"]))
        return {"Xq": v, "sums": s}
    if op == "route":
        ids, probs = kq.kq_moe_route(st["logits"], case["top_k"], score=case["score"], bias=st["bias"],
                                     n_groups=case["n_groups"], topk_groups=case["topk_groups"], group_top=case["group_top"],
                                     renormalise=case["renorm"], scale=case["scale"])
        return {"ids": ids, "probs": probs}
    if op == "g4":
        return kq.kq_matvec_g4(st["W"], st["scales"], st["Xq"], case["M"], case["K"], case["G"], zeros=st["zeros"])
    return kq.kq_moe_matvec_g4(st["W"], st["scales"], case["E"], st["ids"], st["Xq"], case["M"], case["K"], case["G"],
                               zeros=st["zeros"])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "swiglu": _plain_swiglu, "route": _plain_route, "g4": _plain_g4,
            "moe": _plain_moe}[state["case"]["op"]](state)


# ---- from the definitions, in 64 bits -------------------------------------------

def _exact_blocks(v):
    """Values and block sums of the Q8_1 blocks of v (float64 [N, K])."""
    b = v.unflatten(-1, (-1, 32))
    top = torch.maximum(b.max(-1).values, -b.min(-1).values).unsqueeze(-1)
    d = top / 127
    q = torch.where(top > 0, b / d, torch.zeros_like(b)).round()
    d = d.half().double()
    return q * d, (d * q.sum(-1, keepdim=True))


def _exact_route(case, st):
    x = st["logits"].cpu().double()
    T, E = x.shape
    ok = torch.isfinite(x)
    if case["score"] == "softmax":
        s = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    else:
        s = torch.sigmoid(x)
    key = s + (st["bias"].cpu().double() if case["bias"] else 0.0)
    rank = key if case["bias"] else x.clone()
    per = E // case["n_groups"]
    may = ok.clone()
    if case["topk_groups"] < case["n_groups"]:
        sums = torch.full((T, case["n_groups"]), -math.inf, dtype=torch.float64)
        for g in range(case["n_groups"]):
            k, o = key[:, g * per:(g + 1) * per].clone(), ok[:, g * per:(g + 1) * per].clone()
            total, some = torch.zeros(T, dtype=torch.float64), torch.zeros(T, dtype=torch.bool)
            for _ in range(min(per, case["group_top"])):
                best = torch.where(o, k, torch.full_like(k, -math.inf)).max(1)
                has = o.any(1)
                total, some = total + torch.where(has, best.values, torch.zeros_like(total)), some | has
                o[torch.arange(T), best.indices] = False
            sums[:, g] = torch.where(some, total, torch.full_like(total, -math.inf))
        keep = torch.zeros(T, case["n_groups"], dtype=torch.bool)
        for _ in range(case["topk_groups"]):
            left = sums.masked_fill(keep, -math.inf)
            top = left.max(1, keepdim=True).values
            first = ((left == top) & ~keep).int().argmax(1)
            keep[torch.arange(T), first] = True
        may &= keep[:, torch.arange(E) // per]
    ids, w = [], []
    taken = torch.zeros(T, E, dtype=torch.bool)
    for _ in range(case["top_k"]):
        free = may & ~taken
        any_ = free.any(1)
        r = rank.masked_fill(~free, -math.inf)
        pick = torch.where(any_, ((r == r.max(1, keepdim=True).values) & free).int().argmax(1), (~taken).int().argmax(1))
        taken[torch.arange(T), pick] = True
        ids.append(pick)
        w.append(torch.where(any_, s[torch.arange(T), pick], torch.zeros(T, dtype=torch.float64)))
    w = torch.stack(w, 1)
    if case["renorm"]:
        t = w.sum(1, keepdim=True)
        w = torch.where(t > 0, w / t, torch.zeros_like(w))
    return {"ids": torch.stack(ids, 1).int(), "probs": w * case["scale"]}


def _exact_rows(st, at, rows, K, G):
    """Weights of rows [at, at + rows) in float64."""
    W = st["W"][at:at + rows]
    c = torch.empty(rows, K, dtype=torch.float64, device="cuda")
    c[:, 0::2] = (W % 16).double()
    c[:, 1::2] = torch.div(W, 16, rounding_mode="floor").double()
    g = torch.arange(K, device="cuda") // G
    c -= 8 if st["zeros"] is None else st["zeros"][at:at + rows].double()[:, g]
    return c * st["scales"][at:at + rows].double()[:, g]


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "norm":
        h = st["X"].double()
        out = {}
        if case["residual"]:
            h = out["H"] = h + st["R"].double()
        y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["K"] + EPS) * st["gamma"].double()
        if case["y"]:
            out["Y"] = y
        out["Xq"], out["sums"] = _exact_blocks(y)
        return out
    if op == "swiglu":
        g = st["gate"].double()
        v, s = _exact_blocks(g * torch.sigmoid(g) * st["up"].double())
        return {"Xq": v, "sums": s}
    if op == "route":
        return _exact_route(case, st)
    M, K, G = case["M"], case["K"], case["G"]
    x = (st["Xq"][..., 4:].view(torch.int8).double() * st["Xq"][..., 0:2].view(torch.float16).double()).flatten(1)
    step = max(1, (1 << 27) // K)
    if op == "g4":
        return torch.cat([x @ _exact_rows(st, a, min(step, M - a), K, G).T for a in range(0, M, step)], 1)
    ids = st["ids"].long()
    y = torch.empty(*ids.shape, M, dtype=torch.float64, device="cuda")
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        y[t, j] = x[t * ids.shape[1] + j if case["per_slot"] else t] @ _exact_rows(st, e * M, M, K, G).T
    return y


def work(case):
    op = case["op"]
    if op in ("norm", "swiglu"):
        N, K, size = case["N"], case["K"], 4 if case["dtype"] == "fp32" else 2
        if op == "swiglu":
            return {"bytes": N * K * (2 * size + 36 / 32), "flops": 12 * N * K}
        rows = 1 + (2 if case["residual"] else 0) + (1 if case["y"] else 0)
        return {"bytes": N * K * (rows * size + 36 / 32) + 4 * K, "flops": 10 * N * K}
    if op == "route":
        T, E, size = case["T"], case["E"], 4 if case["dtype"] == "fp32" else 2
        return {"bytes": T * (E * size + 8 * case["top_k"]) + (4 * E if case["bias"] else 0), "flops": T * E * (8 + case["top_k"])}
    M, K = case["M"], case["K"]
    groups = -(-K // case["G"])
    matrix = M * (K / 2 + groups * (3 if case["zeros"] else 2))
    if op == "g4":
        return {"bytes": matrix + case["N"] * (K // 32 * 36 + 4 * M), "flops": 2 * case["N"] * M * K}
    pairs = case["T"] * case["top_k"]
    read = case["E"] * (1 - (1 - min(1.0, case["top_k"] / case["E"])) ** case["T"])  # experts that any token chose
    return {"bytes": read * matrix + (pairs if case["per_slot"] else case["T"]) * (K // 32 * 36) + pairs * (4 * M + 4),
            "flops": 2 * pairs * M * K}
