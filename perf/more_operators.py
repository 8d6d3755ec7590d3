"""Measured cases of the operators of a decode step's attention and of the choice of
its tokens: the norm and the position rotation of the heads of queries and keys,
the paged cache that holds keys and values in 4 bits (written, read back, and
attended to), and the sampling of the next tokens.

`run` computes a case in its plain form (elementary torch operations) or, where
`own` is set, through the package's entry points. `exact` computes the same from
the definitions in 64 bits.

Definitions used below
  Rotation: cos_sin[p] holds the cosines of position p's rot / 2 angles, then their
  sines. The first rot elements of a head are turned by pairs (a, b) ->
  (a cos - b sin, b cos + a sin): elements i and i + rot / 2 ("half") or 2i and
  2i + 1 ("pairs").
  4-bit blocks of 32 values v of a head: m = fp16(min v), s = fp16((max v - min v) * (1 / 15)),
  c = clamp(rint((v - m) / s), 0, 15) (0 where s is 0); the block stands for m + s * c.
  Cache: bytes [pages][heads][page / 16][20 * D]; each 20 * D bytes hold 16 tokens of
  one head: key codes [16][D / 2], key parameters [16][s of the D / 32 blocks, then their
  m, fp16], value codes and value parameters alike. With G = D / 32 blocks, element r of block
  g is in byte 4G * (r / 8) + 4g + (r % 8) / 2 of a token's key codes and in byte
  2G * (r / 4) + 2g + (r % 4) / 2 of its value codes, in the low half where r is even.
  Sampling: with the tokens in descending order of their logits (ties to the lower index)
  and weights w = exp((l - max l) / T), the tokens kept are the shortest of three prefixes:
  the first top_k; the shortest with at least top_p of the weight of those; the ones
  with w >= min_p. The token chosen is the first, by index, at which the sum of the kept
  weights passes u times their total. T = 0: the first token with the largest logit. A row of
  logits that are all -inf gives token 0 with probability 0.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # One token's 32 query and 8 key heads after the projections' fp32 rows: the call's latency.
        {"name": "rope decode", "op": "rope", "N": 1, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "pairing": "half",
         "norm": True, "dtype": "fp32", "out": "bf16", "table": 40960},
        # A prompt of 4099 tokens: heads inside packed query, key and value rows.
        {"name": "rope prompt", "op": "rope", "N": 4099, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "pairing": "half",
         "norm": True, "dtype": "bf16", "out": "bf16", "table": 40960},
        # One new token of each of 64 sequences at places up to 32768, fp32 rows as the products give them.
        {"name": "append decode", "op": "append", "N": 64, "seqs": 64, "H": 8, "D": 128, "P": 16, "rot": 128,
         "pairing": "half", "dtype": "fp32", "table": 32768},
        # 8191 tokens of five prompts packed together.
        {"name": "append prompts", "op": "append", "N": 8191, "seqs": 5, "H": 8, "D": 128, "P": 64, "rot": 128,
         "pairing": "half", "dtype": "bf16", "table": 32768},
        # The first tokens of one conversation: the call's latency.
        {"name": "attn short", "op": "attn", "B": 1, "L": 37, "ql": 1, "Hq": 32, "Hk": 8, "D": 128, "P": 16, "window": 0,
         "dtype": "bf16", "xq": False, "empty": False},
        # One conversation of 131072 tokens.
        {"name": "attn long", "op": "attn", "B": 1, "L": 131072, "ql": 1, "Hq": 32, "Hk": 8, "D": 128, "P": 64, "window": 0,
         "dtype": "bf16", "xq": False, "empty": False},
        # 64 sequences of 100 to 8192 tokens; the output goes on as Q8_1 rows to the 4-bit product.
        {"name": "attn batch", "op": "attn", "B": 64, "L": 8192, "ql": 1, "Hq": 28, "Hk": 4, "D": 128, "P": 16, "window": 0,
         "dtype": "fp16", "xq": True, "empty": False},
        # Up to five drafted tokens of each of 16 sequences checked at once, in a sliding window, fp32 rows.
        {"name": "attn drafts", "op": "attn", "B": 16, "L": 16384, "ql": 5, "Hq": 16, "Hk": 4, "D": 64, "P": 32,
         "window": 4096, "dtype": "fp32", "xq": False, "empty": True},
        # A wide head with one key head for all queries.
        {"name": "attn wide", "op": "attn", "B": 8, "L": 6001, "ql": 1, "Hq": 8, "Hk": 1, "D": 256, "P": 128, "window": 0,
         "dtype": "bf16", "xq": False, "empty": False},
        # The next token of one conversation: all of the usual limits.
        {"name": "sample one", "op": "sample", "N": 1, "V": 152064, "k": True, "p": True, "m": True, "spread": 2.5,
         "masked": 0.0, "dtype": "fp32"},
        # 64 sequences, a nucleus alone, bf16 logits with their many ties.
        {"name": "sample nucleus", "op": "sample", "N": 64, "V": 152064, "k": False, "p": True, "m": False, "spread": 2.5,
         "masked": 0.0, "dtype": "bf16"},
        # 200 sequences of a small vocabulary, most of it ruled out by a grammar.
        {"name": "sample masked", "op": "sample", "N": 200, "V": 32003, "k": True, "p": False, "m": True, "spread": 2.0,
         "masked": 0.9, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "sample"])
    dtype = rng.choice(["fp32", "fp16", "bf16"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 256])
        Hk = rng.choice([0, 1, 2, 4, 8])
        Hq = max(1, Hk) * rng.randint(1, 8)
        N = _log(rng, 1, min(32768, 4099 * 40 * 128 * 4 // ((Hq + Hk) * D * (8 if dtype == "fp32" else 4))))
        return {"op": op, "N": N, "Hq": Hq, "Hk": Hk, "D": D, "rot": rng.choice([D, D, 16 * (D // 32)]),
                "pairing": rng.choice(["half", "pairs"]), "norm": rng.random() < 0.6, "dtype": dtype,
                "out": dtype if dtype != "fp32" else rng.choice(["fp32", "bf16"]), "table": _log(rng, 64, 131072)}
    if op == "append":
        D, H, P = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 5, 8]), rng.choice([16, 32, 64, 128])
        N = _log(rng, 1, min(16384, 8191 * 8 * 128 // (H * D * (2 if dtype == "fp32" else 1))))
        return {"op": op, "N": N, "seqs": rng.choice([N, rng.randint(1, N), min(N, 7)]), "H": H, "D": D, "P": P,
                "rot": rng.choice([0, D, D, D // 2]), "pairing": rng.choice(["half", "pairs"]), "dtype": dtype,
                "table": _log(rng, 20000, 100000)}
    if op == "attn":
        D, Hk, P = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
        Hq = Hk * rng.choice([1, 3, 4, 5, 7, 8, 12])
        B = _log(rng, 1, 96)
        ql = rng.choice([1, 1, 1, 1, 2, 4, 7])
        L = _log(rng, 1, 131072 * 8 * 128 // (B * Hk * D * ql * max(1, Hq // Hk // 4)))
        return {"op": op, "B": B, "L": max(ql, min(L, 131072)), "ql": ql, "Hq": Hq, "Hk": Hk, "D": D, "P": P,
                "window": rng.choice([0, 0, 0, 100, 4096]), "dtype": dtype, "xq": rng.random() < 0.3,
                "empty": B > 1 and rng.random() < 0.3}
    V = _log(rng, 500, 262144)
    k, p = rng.random() < 0.5, rng.random() < 0.6
    return {"op": op, "N": _log(rng, 1, min(512, 64 * 152064 // V // (2 if dtype == "fp32" else 1))), "V": V, "k": k, "p": p,
            "m": rng.random() < 0.4, "spread": rng.choice([1.0, 2.5, 4.0]), "masked": rng.choice([0.0, 0.0, 0.5, 0.99]),
            "dtype": dtype}


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _ints(gen, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=gen, device="cuda")


def _table(n, rot):
    """Cosines and sines of `n` positions' angles, fp32 [n, rot]."""
    f = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float().contiguous()


def _heads(gen, N, H, D):
    """Head rows in which a few channels are large, as a model's keys have them."""
    x = _randn(gen, N, H, D)
    return x * torch.where(torch.rand(H, D, generator=gen, device="cuda") < 0.03, 6.0, 1.0)


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, spread over their logarithm; the largest comes first."""
    return [max(lo, min(hi, int(round(hi * (lo / hi) ** ((i * 0.6180339887) % 1.0))))) for i in range(n)]


def _lengths(case):
    """(cached tokens, new tokens) of each sequence of an attention case."""
    new = [1 + (case["ql"] - 1 - i) % case["ql"] for i in range(case["B"])]
    cached = [max(n, c) for n, c in zip(new, _spread(case["B"], max(1, case["L"] // 80), case["L"]))]
    if case["empty"]:
        cached[-1] = 0
    return cached, new


def _codes(gen, *shape):
    """Bytes of two 4-bit codes each, bell-shaped over 0 to 15 as the blocks of about normal values have them."""
    lut = torch.clamp(torch.round(7.5 + 3.3 * _randn(gen, 1 << 16, 2)), 0, 15).to(torch.uint8)
    return (lut[:, 0] | (lut[:, 1] << 4))[_ints(gen, 0, 1 << 16, *shape)]


def _cache(gen, pages, H, P, D):
    """A cache whose keys and values are about normal, as prompts of a model leave it."""
    c = torch.empty(pages, H, P // 16, 20 * D, dtype=torch.uint8, device="cuda")
    G = D // 32
    for at, size in ((0, 0.25), (10 * D, 0.15)):
        c[..., at:at + 8 * D] = _codes(gen, pages, H, P // 16, 8 * D)
        s = (size * torch.exp(0.3 * _randn(gen, pages, H, P // 16, 16, G))).half()
        m = (-7.5 * s.float() + 0.3 * _randn(gen, pages, H, P // 16, 16, G)).half()
        c[..., at + 8 * D:at + 10 * D] = torch.cat([s, m], -1).flatten(3).view(torch.uint8)
    return c


def _tables(gen, lengths, P):
    """(pages, block table int32 [sequences, most pages]): pages in random places, page 0 belonging to nobody."""
    need = [-(-n // P) for n in lengths]
    at = (torch.randperm(sum(need), generator=gen, device="cuda") + 1).to(torch.int32)
    table = torch.zeros(len(need), max(1, max(need)), dtype=torch.int32, device="cuda")
    for i, n in enumerate(need):
        table[i, :n] = at[sum(need[:i]):sum(need[:i]) + n]
    return sum(need) + 1, table


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    op, t = case["op"], DTYPES[case["dtype"]]
    i32 = {"dtype": torch.int32, "device": "cuda"}
    if op == "rope":
        N, Hq, Hk, D = case["N"], case["Hq"], case["Hk"], case["D"]
        rows = _heads(gen, N, Hq + 2 * Hk, D).to(t)  # queries, keys and values of one projection
        st["Q"], st["K"] = rows[:, :Hq], rows[:, Hq:Hq + Hk] if Hk else None
        st["q_gamma"] = 1.0 + 0.2 * _randn(gen, D) if case["norm"] else None
        st["k_gamma"] = 1.0 + 0.2 * _randn(gen, D) if case["norm"] and Hk else None
        st["cos_sin"] = _table(case["table"], case["rot"])
        st["positions"] = _ints(gen, 0, case["table"], N).to(torch.int32)
    elif op == "append":
        N, n_seqs, H, D, P = case["N"], case["seqs"], case["H"], case["D"], case["P"]
        rows = _heads(gen, N, 2 * H, D).to(t)
        st["K"], st["V"] = rows[:, :H], rows[:, H:]
        new = [N // n_seqs + (i < N % n_seqs) for i in range(n_seqs)]
        seq = torch.repeat_interleave(torch.arange(n_seqs, device="cuda"), torch.tensor(new, device="cuda"), output_size=N)
        first = torch.cumsum(torch.tensor([0] + new[:-1], device="cuda"), 0)
        start = _ints(gen, 0, case["table"] - max(new) + 1, n_seqs)  # tokens that were there before
        pos = start[seq] + torch.arange(N, device="cuda") - first[seq]
        page = torch.unique(seq * 8192 + pos // P)                   # pages that are written, one by one
        table = torch.zeros(n_seqs, -(-case["table"] // P), **i32)
        table[page // 8192, page % 8192] = (torch.randperm(page.numel(), generator=gen, device="cuda") + 1).to(torch.int32)
        st["table"], st["positions"], st["seq_ids"] = table, pos.to(torch.int32), seq.to(torch.int32)
        st["cache"] = torch.zeros(page.numel() + 1, H, P // 16, 20 * D, dtype=torch.uint8, device="cuda")
        st["cos_sin"] = _table(case["table"], case["rot"]) if case["rot"] else None
    elif op == "attn":
        cached, new = _lengths(case)
        pages, st["table"] = _tables(gen, cached, case["P"])
        st["cache"] = _cache(gen, pages, case["Hk"], case["P"], case["D"])
        N = sum(new)
        st["Q"] = (2.0 * _randn(gen, N, case["Hq"], case["D"])).to(t)
        st["kv_len"] = torch.tensor(cached, **i32)
        start = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], **i32)
        st["q_start"] = start if case["ql"] > 1 else None
        # Each row's sequence, its place among its sequence's new rows, and how many tokens it sees.
        seq = torch.repeat_interleave(torch.arange(case["B"], device="cuda"), torch.tensor(new, device="cuda"), output_size=N)
        at = torch.arange(N, device="cuda") - start[seq]
        n = torch.tensor(new, device="cuda")
        st["seq"], st["at"] = seq, at
        st["row"] = torch.clamp(start[:-1, None] + torch.arange(max(new), device="cuda"), max=N - 1).long()
        st["sees"] = torch.tensor(cached, device="cuda")[:, None] - n[:, None] + 1 + torch.arange(max(new), device="cuda")
    else:
        N, V = case["N"], case["V"]
        x = case["spread"] * _randn(gen, N, V)
        x += 3.0 * (torch.rand(N, V, generator=gen, device="cuda") < 2e-4)  # the words that fit
        if case["masked"]:
            x[torch.rand(N, V, generator=gen, device="cuda") < case["masked"]] = float("-inf")
        st["logits"] = x.to(t)
        st["u"] = torch.rand(N, generator=gen, device="cuda")
        T = 0.6 + 0.6 * torch.rand(N, generator=gen, device="cuda")
        T[5::16] = 0.0  # some sequences want the likeliest token
        st["temperature"] = T
        st["top_k"] = _ints(gen, 1, min(V, 1000) + 1, N).to(torch.int32) if case["k"] else None
        st["top_p"] = 0.5 + 0.49 * torch.rand(N, generator=gen, device="cuda") if case["p"] else None
        st["min_p"] = 0.1 * torch.rand(N, generator=gen, device="cuda") if case["m"] else None
    return st


# ---- plain form ---------------------------------------------------------------

def _turned(x, cs, rot, pairing):
    """Heads x [N, H, D] (fp32) turned by rows cs [N, rot] of the table."""
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if pairing == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), x[..., rot:]], -1)


def _plain_rope(st):
    case = st["case"]
    cs = st["cos_sin"][st["positions"].long()]

    def one(x, gamma):
        x = x.float()
        if gamma is not None:
            x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * gamma
        return _turned(x, cs, case["rot"], case["pairing"]).to(DTYPES[case["out"]])

    out = {"Q": one(st["Q"], st["q_gamma"])}
    if st["K"] is not None:
        out["K"] = one(st["K"], st["k_gamma"])
    return out


def _in_blocks(x):
    """What the 4-bit blocks of heads x [N, H, D] (fp32) stand for."""
    v = x.unflatten(-1, (-1, 32))
    low, high = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    m = low.half().float()
    s = ((high - low) * (1.0 / 15.0)).half().float()
    c = torch.where(s > 0, torch.clamp(torch.round((v - m) / s), 0, 15), torch.zeros_like(v))
    return (m + s * c).flatten(-2)


def _plain_append(st):
    case = st["case"]
    K, V = st["K"].float(), st["V"].float()
    if case["rot"]:
        K = _turned(K, st["cos_sin"][st["positions"].long()], case["rot"], case["pairing"])
    t = _row_type(case)
    return {"K": _in_blocks(K).to(t), "V": _in_blocks(V).to(t)}


def _row_type(case):
    """The type of rows that are read back from the cache: that of the rows that went in, fp16 for fp32."""
    return torch.float16 if case["dtype"] == "fp32" else DTYPES[case["dtype"]]


def _plain_read(st):
    """Keys and values of all sequences, fp32 [B, H, places, D] each."""
    D, G = st["case"]["D"], st["case"]["D"] // 32
    c = st["cache"][st["table"].long()]                   # [B, pages, H, page / 16, 20 D]
    c = c.permute(0, 2, 1, 3, 4).flatten(2, 3)            # [B, H, granules, 20 D]
    got = []
    for at, shape, order in ((0, (4, G, 4), 8), (10 * D, (8, G, 2), 4)):
        b = c[..., at:at + 8 * D].unflatten(-1, (16, *shape))
        q = torch.stack([b & 15, b >> 4], -1).flatten(-2).transpose(-2, -3).reshape(*b.shape[:4], G, 32)
        p = c[..., at + 8 * D:at + 10 * D].contiguous().view(torch.float16).unflatten(-1, (16, 2, G)).float()
        got.append((p[..., 1, :, None] + p[..., 0, :, None] * q).flatten(2, 3).flatten(-2))
    return got


def _q8(v):
    """What the Q8_1 blocks of fp32 rows v [N, K] stand for (fp16, the type of their scales), and their block sums."""
    b = v.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / 127.0
    inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    q = torch.clamp(torch.round(b * inv), -128, 127)
    d = d.to(torch.float16)
    return q.to(torch.float16) * d, (d.float() * q.sum(-1, keepdim=True)).to(torch.float16)


def _plain_attn(st):
    case = st["case"]
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    K, V = _plain_read(st)
    B, _, L, _ = K.shape
    q = st["Q"].float()[st["row"]]                                            # [B, new, Hq, D]
    n = q.shape[1]
    q = q.reshape(B, n, Hk, Hq // Hk, D).transpose(1, 2).flatten(2, 3)        # [B, Hk, new * group, D]
    s = torch.matmul(q, K.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    at = torch.arange(L, device="cuda")
    sees = st["sees"][:, :, None]
    may = at < sees
    if case["window"]:
        may = may & (at >= sees - case["window"])
    may = may.repeat_interleave(Hq // Hk, 1)[:, None]                         # [B, 1, new * group, L]
    s = torch.where(may, s, torch.full_like(s, float("-inf")))
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    z = e.sum(-1, keepdim=True)
    v = torch.where(at[None, :, None] < st["kv_len"][:, None, None], torch.ones((), device="cuda"),
                    torch.zeros((), device="cuda"))[:, None] * V              # places behind a sequence's end
    o = torch.matmul(e, v) / torch.where(z > 0, z, torch.ones_like(z))
    o = o.unflatten(2, (n, Hq // Hk)).transpose(1, 2).flatten(2, 3)           # [B, new, Hq, D]
    o = o[st["seq"], st["at"]]
    out = {"O": o.to(st["Q"].dtype)}
    if case["xq"]:
        out["Xq"], out["sums"] = _q8(o.flatten(1))
    return out


def _plain_sample(st):
    # In 64 bits: sums over a whole vocabulary are compared with one another.
    x = st["logits"].double()
    N, V = x.shape
    T = st["temperature"].double()[:, None]
    top = x.amax(-1, keepdim=True)
    some = top > float("-inf")
    w = torch.exp((x - torch.where(some, top, torch.zeros_like(top))) / torch.where(T > 0, T, torch.ones_like(T)))
    first = torch.arange(V, device="cuda") == torch.argmax((x == top).to(torch.int32), -1, keepdim=True)
    w = torch.where(T > 0, w, (first & some).double())
    val, order = torch.sort(x, dim=-1, descending=True, stable=True)
    ws = w.gather(1, order)
    if st["top_k"] is not None:
        k = st["top_k"].long()[:, None]
        ws = torch.where((torch.arange(V, device="cuda") < k) | (k <= 0), ws, torch.zeros_like(ws))
    keep = ws > 0
    if st["top_p"] is not None:
        before = torch.cumsum(ws, -1) - ws
        p = st["top_p"].double()[:, None]
        keep = keep & ((before < p * ws.sum(-1, keepdim=True)) | (p >= 1))
    if st["min_p"] is not None:
        keep = keep & (ws >= st["min_p"].double()[:, None])
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, torch.zeros_like(ws)))
    c = torch.cumsum(w, -1)
    total = c[:, -1:]
    ids = torch.where(some, (c <= st["u"].double()[:, None] * total).sum(-1, keepdim=True).clamp(max=V - 1), 0)
    return {"ids": ids[:, 0].to(torch.int32), "probs": (w.gather(1, ids) / torch.where(some, total, 1.0))[:, 0].float()}


def _own(st):
    import quantized_weight_matmul_q4_gb300 as kq

    case, op = st["case"], st["case"]["op"]
    if op == "rope":
        Q, K = kq.kq_qk_norm_rope(st["Q"], st["K"], st["cos_sin"], st["positions"], q_gamma=st["q_gamma"],
                                  k_gamma=st["k_gamma"], eps=EPS, pairing=case["pairing"], out_dtype=DTYPES[case["out"]])
        return {"Q": Q} if K is None else {"Q": Q, "K": K}
    if op == "append":
        kq.kq_kv_append_q4(st["K"], st["V"], st["cache"], st["table"], st["positions"], seq_ids=st["seq_ids"],
                           cos_sin=st["cos_sin"], pairing=case["pairing"])
        K, V = kq.kq_kv_gather_q4(st["cache"], st["table"], st["positions"], seq_ids=st["seq_ids"], dtype=_row_type(case))
        return {"K": K, "V": V}
    if op == "attn":
        O, Xq = kq.kq_attn_q4(st["Q"], st["cache"], st["table"], st["kv_len"], q_start=st["q_start"],
                              window=case["window"], Xq=case["xq"])
        if Xq is None:
            return {"O": O}
        h = Xq.view(torch.float16)
        return {"O": O, "Xq": Xq.view(torch.int8).narrow(-1, 4, 32) * h.narrow(-1, 0, 1), "sums": h.narrow(-1, 1, 1)}
    ids, probs = kq.kq_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                              top_p=st["top_p"], min_p=st["min_p"])
    return {"ids": ids, "probs": probs}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "sample": _plain_sample}[
        state["case"]["op"]](state)


# ---- from the definitions, in 64 bits -------------------------------------------

def _exact_turn(x, st, case):
    """Each pair as a complex number times cos + i sin."""
    rot, h = case["rot"], case["rot"] // 2
    cs = st["cos_sin"].index_select(0, st["positions"].long()).double()
    unit = torch.complex(cs[:, :h], cs[:, h:]).unsqueeze(1)
    i = torch.arange(h, device="cuda")
    a, b = (i, i + h) if case["pairing"] == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(x[..., a], x[..., b]) * unit
    x = x.clone()
    x[..., a], x[..., b] = z.real, z.imag
    return x


def _exact_blocks4(x):
    N, H, D = x.shape
    b = x.reshape(N, H, D // 32, 32)
    low = b.min(-1, keepdim=True).values
    m, s = low.half().double(), ((b.max(-1, keepdim=True).values - low) / 15).half().double()
    c = torch.nan_to_num((b - m) / s, nan=0.0).round().clip(0, 15)
    return (m + c * s).reshape(N, H, D)


def _exact_attn(case, st):
    D, G, P, Hk = case["D"], case["D"] // 32, case["P"], case["Hk"]
    group = case["Hq"] // Hk
    cached, new = _lengths(case)
    r = torch.arange(D, device="cuda") % 32
    g = torch.arange(D, device="cuda") // 32
    places = ((0, 4 * G * (r // 8) + 4 * g + r % 8 // 2), (10 * D, 2 * G * (r // 4) + 2 * g + r % 4 // 2))
    O = torch.zeros(sum(new), case["Hq"], D, dtype=torch.float64, device="cuda")
    n0 = 0
    for b, (n, have) in enumerate(zip(new, cached)):
        t = torch.arange(have, device="cuda")
        page = st["table"][b].long()[t // P]
        for h in range(Hk if have else 0):
            got = []
            for at, byte in places:
                rows = st["cache"][page, h, t % P // 16]                                   # [have, 20 D]
                codes = rows.gather(1, at + (t % 16)[:, None] * (D // 2) + byte)
                codes = torch.where(r % 2 == 0, codes % 16, torch.div(codes, 16, rounding_mode="floor")).double()
                par = rows[:, at + 8 * D:at + 10 * D].contiguous().view(torch.float16).double()
                s = par.gather(1, (t % 16)[:, None] * 2 * G + g)
                got.append(par.gather(1, (t % 16)[:, None] * 2 * G + G + g) + s * codes)
            for i in range(n):
                end = have - n + 1 + i
                begin = max(0, end - case["window"]) if case["window"] else 0
                if end > begin:
                    q = st["Q"][n0 + i, h * group:(h + 1) * group].double()
                    p = torch.softmax(q @ got[0][begin:end].T / math.sqrt(D), 1)
                    O[n0 + i, h * group:(h + 1) * group] = p @ got[1][begin:end]
        n0 += n
    out = {"O": O}
    if case["xq"]:
        b = O.reshape(O.shape[0], -1, 32)
        top = b.abs().max(-1, keepdim=True).values
        q = torch.where(top > 0, b * 127 / top, torch.zeros_like(b)).round()
        d = (top / 127).half().double()
        out["Xq"], out["sums"] = q * d, d * q.sum(-1, keepdim=True)
    return out


def _exact_sample(case, st):
    ids, probs = [], []
    x = st["logits"].double().cpu()
    of = {k: st[k].tolist() if st[k] is not None else None for k in ("u", "temperature", "top_k", "top_p", "min_p")}
    for n in range(case["N"]):
        l, T = x[n], of["temperature"][n]
        idx = torch.argsort(l, descending=True, stable=True)
        idx = idx[:int((l > -math.inf).sum())]
        if T == 0 or not len(idx):
            ids.append(int(idx[0]) if len(idx) else 0)
            probs.append(1.0 if len(idx) else 0.0)
            continue
        if of["top_k"] is not None:
            idx = idx[:of["top_k"][n]]
        w = torch.exp((l[idx] - l[idx[0]]) / T)
        count = len(idx)
        if of["top_p"] is not None:
            count = min(count, 1 + int((torch.cumsum(w, 0) < of["top_p"][n] * w.sum()).sum()))
        if of["min_p"] is not None:
            count = min(count, int((w >= of["min_p"][n]).sum()))
        by, at = torch.sort(idx[:count])
        w = w[:count][at]
        c = torch.cumsum(w, 0)
        pick = min(count - 1, int((c <= of["u"][n] * c[-1]).sum()))
        ids.append(int(by[pick]))
        probs.append(float(w[pick] / c[-1]))
    return {"ids": torch.tensor(ids, dtype=torch.int32), "probs": torch.tensor(probs, dtype=torch.float64)}


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "rope":
        out = {}
        for name, gamma in (("Q", st["q_gamma"]), ("K", st["k_gamma"])):
            if st[name] is not None:
                x = st[name].double()
                if gamma is not None:
                    x = x * torch.rsqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / case["D"] + EPS) * gamma.double()
                out[name] = _exact_turn(x, st, case)
        return out
    if op == "append":
        K = st["K"].double()
        return {"K": _exact_blocks4(_exact_turn(K, st, case) if case["rot"] else K), "V": _exact_blocks4(st["V"].double())}
    return _exact_attn(case, st) if op == "attn" else _exact_sample(case, st)


def work(case):
    op, size = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op == "rope":
        values = case["N"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": values * (size + (4 if case["out"] == "fp32" else 2)) + 4 * case["N"] * (case["rot"] + 1),
                "flops": 8 * values}
    if op == "append":
        # Written into the cache, and read back from there as rows.
        values = 2 * case["N"] * case["H"] * case["D"]
        return {"bytes": values * (size + 5 / 8 + 5 / 8 + 2) + 4 * case["N"] * (case["rot"] + 4), "flops": 12 * values}
    if op == "attn":
        cached, new = _lengths(case)
        w = case["window"] or 1 << 40
        seen = sum(min(c, w + n - 1) for c, n in zip(cached, new))
        rows = sum(new) * case["Hq"] * case["D"]
        out = rows * (size + (36 / 32 if case["xq"] else 0))
        return {"bytes": seen * case["Hk"] * case["D"] * 5 / 4 + rows * size + out + 4 * seen / case["P"],
                "flops": 4 * case["Hq"] * case["D"] * sum(n * min(c, w) for c, n in zip(cached, new))}
    return {"bytes": case["N"] * (case["V"] * size + 28), "flops": 8 * case["N"] * case["V"]}
