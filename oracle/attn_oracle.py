"""Plain definitions of the attention-side operators of a decode step: head norms with the position
rotation, the blocks and the layout of the 4-bit paged cache, attention over it, and
sampling.

numpy only, no code shared with the CUDA path. Values are fp64 except where a definition is
one of fp32 steps (the rotation of cached keys and their blocks), which is evaluated in
exactly those steps.
"""
from __future__ import annotations

import numpy as np

F = np.float32


def rope_pairs(rot, pairing):
    """Indices (first, second) of the elements that are turned together."""
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if pairing == "half" else (2 * i, 2 * i + 1)


def norm_rope(x, gamma, eps, cs, pairing):
    """(y, B) for heads x [N, H, D] and table rows cs [N, rot] or None: the normed and turned heads in fp64,
    and |a cos| + |b sin| of every element (|y| where nothing is turned)."""
    y = np.asarray(x, np.float64)
    if gamma is not None:
        with np.errstate(divide="ignore", invalid="ignore"):
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    B = np.abs(y)
    if cs is not None:
        rot = cs.shape[1]
        a, b = rope_pairs(rot, pairing)
        c, s = (np.asarray(cs, np.float64)[:, None, k * (rot // 2):(k + 1) * (rot // 2)] for k in (0, 1))
        out, B = y.copy(), B.copy()
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        B[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
        B[..., b] = np.abs(y[..., b] * c) + np.abs(y[..., a] * s)
        y = out
    return y, B


def turn_fp32(x, cs, pairing):
    """The rotation of cached keys: x fp32 [N, H, D], each product and each sum rounded to fp32."""
    out = np.array(x, F)
    if cs is None:
        return out
    rot = cs.shape[1]
    a, b = rope_pairs(rot, pairing)
    c, s = (np.asarray(cs, F)[:, None, k * (rot // 2):(k + 1) * (rot // 2)] for k in (0, 1))
    out[..., a] = (x[..., a] * c).astype(F) - (x[..., b] * s).astype(F)
    out[..., b] = (x[..., b] * c).astype(F) + (x[..., a] * s).astype(F)
    return out


def blocks4(v):
    """(s fp16, m fp16, codes uint8) of fp32 values v [..., 32]."""
    v = np.asarray(v, F)
    with np.errstate(all="ignore"):
        lo, hi = v.min(-1, keepdims=True), v.max(-1, keepdims=True)
        m = lo.astype(np.float16)
        s = ((hi - lo).astype(F) * F(1.0 / 15.0)).astype(F).astype(np.float16)
        bad = ~(np.isfinite(m) & np.isfinite(s))
        t = ((v - m.astype(F)).astype(F) / s.astype(F)).astype(F)
        c = np.where(s > 0, np.clip(np.rint(t), 0, 15), 0)
    c = np.where(bad, 0, np.nan_to_num(c)).astype(np.uint8)
    return np.where(bad, np.float16(np.nan), s)[..., 0], np.where(bad, np.float16(0), m)[..., 0], c


def code_bytes(D, values):
    """(byte, in the high half) of each element of a token's key codes, or its value codes."""
    G, e = D // 32, np.arange(D)
    g, r = e // 32, e % 32
    byte = 2 * G * (r // 4) + 2 * g + (r % 4) // 2 if values else 4 * G * (r // 8) + 4 * g + (r % 8) // 2
    return byte, r % 2


def append(cache, table, page_size, K, V, positions, seq_ids):
    """Writes fp32 heads K, V [N, H, D] (turned already) into a cache uint8 [pages, H, page / 16, 20 D], in place."""
    N, H, D = K.shape
    G = D // 32
    for n in range(N):
        p = int(positions[n])
        if p < 0:
            continue
        page, off = int(table[seq_ids[n], p // page_size]), p % page_size
        for values, x in ((0, K), (1, V)):
            s, m, c = blocks4(x[n].reshape(H, G, 32))
            byte, high = code_bytes(D, values)
            row = np.zeros((H, D // 2), np.uint8)
            for h in range(H):
                np.bitwise_or.at(row[h], byte, c[h].reshape(D) << (4 * high).astype(np.uint8))
            at, t = 10 * D * values, off % 16
            gr = cache[page, :, off // 16]
            gr[:, at + t * (D // 2):at + (t + 1) * (D // 2)] = row
            par = np.concatenate([s, m], 1).astype(np.float16).view(np.uint8)
            gr[:, at + 8 * D + t * 4 * G:at + 8 * D + (t + 1) * 4 * G] = par


def read(cache, table_row, page_size, places):
    """(s, m, codes) of the keys and of the values at `places` of one sequence: fp64 [T, H, G], [T, H, G], [T, H, G, 32]."""
    _, H, _, size = cache.shape
    D = size // 20
    G = D // 32
    got = []
    places = np.asarray(places, np.int64)
    gr = cache[np.asarray(table_row)[places // page_size], :, places % page_size // 16]   # [T, H, 20 D]
    for values in (0, 1):
        byte, high = code_bytes(D, values)
        at = 10 * D * values
        idx = at + (places % 16 * (D // 2))[:, None] + byte
        b = np.take_along_axis(gr, np.broadcast_to(idx[:, None], (len(places), H, D)), 2)
        c = np.where(high, b >> 4, b & 15).astype(np.float64).reshape(len(places), H, G, 32)
        idx = at + 8 * D + (places % 16 * 4 * G)[:, None] + np.arange(4 * G)
        par = np.take_along_axis(gr, np.broadcast_to(idx[:, None], (len(places), H, 4 * G)), 2)
        par = np.ascontiguousarray(par).view(np.float16).astype(np.float64)
        got.append((par[..., :G], par[..., G:], c))
    return got


def attention(Q, cache, table, page_size, kv_len, q_start=None, scale=None, window=0):
    """(o, E, S) for queries Q [N, Hq, D]: the output in fp64; E [2, N, Hq, D] = Sum_t p_t (|s_t| |c_t - 8| + |m_t + 8 s_t|)
    and Sum_t p_t (|s_t| c_t + |m_t|) per element (what rounding errors of the weights scale with where the codes are taken from
    their middle, and those of sums of codes as they are); S [N, Hq] = the largest over t of scale * Sum (|s| c + |m|) |q| (what those of
    the scores scale with). Rows of no sequence are NaN."""
    Q = np.asarray(Q, np.float64)
    N, Hq, D = Q.shape
    H = cache.shape[1]
    group = Hq // H
    scale = D ** -0.5 if scale is None else scale
    o, E, S = np.full((N, Hq, D), np.nan), np.zeros((2, N, Hq, D)), np.zeros((N, Hq))
    for b in range(len(kv_len)):
        n0, n1 = (b, b + 1) if q_start is None else (int(q_start[b]), int(q_start[b + 1]))
        if n1 <= n0:
            continue
        L = max(0, int(kv_len[b]))
        (ks, km, kc), (vs, vm, vc) = read(cache, table[b], page_size, np.arange(L))
        flat = lambda s, m, c: (m[..., None] + s[..., None] * c).reshape(L, H, D)  # noqa: E731
        k, v = flat(ks, km, kc), flat(vs, vm, vc)
        ka, va = flat(np.abs(ks), np.abs(km), kc), flat(np.abs(vs), np.abs(vm), vc)
        vd = flat(np.abs(vs), np.abs(vm + 8 * vs), np.abs(vc - 8))
        for n in range(n0, n1):
            end = L - (n1 - n0) + 1 + (n - n0)
            begin = max(0, end - window) if window else 0
            if end <= begin:
                o[n] = 0
                continue
            for i in range(Hq):
                h = i // group
                x = scale * (k[begin:end, h] @ Q[n, i])
                S[n, i] = np.max(abs(scale) * (ka[begin:end, h] @ np.abs(Q[n, i])))
                p = np.exp(x - x.max())
                p /= p.sum()
                o[n, i] = p @ v[begin:end, h]
                E[0, n, i], E[1, n, i] = p @ vd[begin:end, h], p @ va[begin:end, h]
    return o, E, S


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(ids, probs fp64) of rows of logits."""
    L = np.asarray(logits, np.float64)
    ids, probs = [], []
    for n, l in enumerate(L):
        l = np.minimum(np.where(np.isnan(l), -np.inf, l), float(np.finfo(F).max))
        order = sorted((i for i in range(len(l)) if l[i] > -np.inf), key=lambda i: (-l[i], i))
        T = 1.0 if temperature is None else float(temperature[n])
        if not order or not T > 0:
            ids.append(order[0] if order else 0)
            probs.append(1.0 if order else 0.0)
            continue
        k = 0 if top_k is None else int(top_k[n])
        if k > 0:
            order = order[:k]
        w = np.exp((l[order] - l[order[0]]) / T)
        keep = len(order)
        p = 1.0 if top_p is None else float(top_p[n])
        if p < 1:
            c = np.cumsum(w)
            keep = next((i + 1 for i in range(len(c)) if c[i] >= p * c[-1]), keep)
        m = 0.0 if min_p is None else min(1.0, float(min_p[n]))
        if m > 0:
            keep = min(keep, int((w >= m).sum()))
        kept = sorted(order[:keep])
        at = {i: x for i, x in zip(order, w)}
        w = np.array([at[i] for i in kept])
        c = np.cumsum(w)
        j = int(np.argmax(c > min(float(u[n]) * c[-1], np.nextafter(c[-1], 0))))
        ids.append(kept[j])
        probs.append(w[j] / c[-1])
    return np.array(ids), np.array(probs)
