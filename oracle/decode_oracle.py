"""Plain fp64 definitions of the operators of a decode step around 4-bit experts:
residual RMSNorm and SwiGLU with their Q8_1 blocks, the routing of tokens to
experts, and the products of Q8_1 rows with group-scaled 4-bit weights.

numpy only, no code shared with the CUDA path. Everything is a direct
evaluation of the definition: loops over tokens, slots and groups.
"""
from __future__ import annotations

import numpy as np


def add_rmsnorm(X, R, gamma, eps):
    """h = x + r and y = h / sqrt(mean h^2 + eps) * gamma, fp64 [N, K]."""
    h = np.asarray(X, np.float64)
    if R is not None:
        h = h + np.asarray(R, np.float64)
    ms = np.mean(h * h, axis=1, keepdims=True)
    return h, h / np.sqrt(ms + eps) * np.asarray(gamma, np.float64)


def swiglu(gate, up):
    g, u = np.asarray(gate, np.float64), np.asarray(up, np.float64)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def unpack_q8_1(Xq):
    """(d_h, s_h as fp64, codes int64 [..., 32]) of Q8_1 blocks uint8 [..., 36]."""
    b = np.ascontiguousarray(Xq)
    h = b[..., 0:4].copy().view(np.float16).astype(np.float64)
    return h[..., 0], h[..., 1], b[..., 4:].view(np.int8).astype(np.int64)


def route(logits, top_k, score="softmax", bias=None, n_groups=1, topk_groups=1, group_top=2, renormalise=True,
          scale=1.0):
    """(ids [T, top_k], probs fp64 [T, top_k]); ties to the lowest index."""
    L = np.asarray(logits, np.float64)
    T, E = L.shape
    per = E // n_groups
    ids = np.zeros((T, top_k), np.int64)
    probs = np.zeros((T, top_k))
    for t in range(T):
        l = np.minimum(np.where(np.isnan(L[t]), -np.inf, L[t]), float(np.finfo(np.float32).max))
        ok = l != -np.inf
        s = np.zeros(E)
        if ok.any():
            if score == "softmax":
                s[ok] = np.exp(l[ok] - l[ok].max())
                s /= s.sum()
            else:
                with np.errstate(over="ignore"):
                    s[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
        key = s if bias is None else s + np.asarray(bias, np.float64)
        ok &= ~(np.isnan(key) | (key == -np.inf))
        order_by = l if bias is None else key
        may = ok.copy()
        if topk_groups < n_groups:
            best = []
            for g in range(n_groups):
                v = sorted((key[e] for e in range(g * per, (g + 1) * per) if ok[e]), reverse=True)[:group_top]
                best.append(sum(v) if v else -np.inf)
            keep = sorted((g for g in range(n_groups) if best[g] != -np.inf), key=lambda g: (-best[g], g))[:topk_groups]
            may &= np.isin(np.arange(E) // per, keep)
        chosen = sorted(np.flatnonzero(may), key=lambda e: (-order_by[e], e))[:top_k]
        w = [s[e] for e in chosen] + [0.0] * (top_k - len(chosen))
        chosen += [e for e in range(E) if e not in set(chosen)][:top_k - len(chosen)]
        w = np.array(w)
        if renormalise:
            w = w / w.sum() if w.sum() > 0 else np.zeros(top_k)
        ids[t], probs[t] = chosen, w * scale
    return ids, probs


def g4_codes(W):
    """4-bit codes int64 [M, K] of bytes uint8 [M, K/2]: the even k in the low half."""
    c = np.empty((W.shape[0], 2 * W.shape[1]), np.int64)
    c[:, 0::2] = W & 15
    c[:, 1::2] = W >> 4
    return c


def g4_matmul(W, scales, zeros, group, Xq):
    """(Y, B): Y[n, m] = Sum_k s (c - z) d q in fp64, and B the sum over the 32-element
    blocks of the blocks' absolute contributions (what fp32 rounding errors scale with)."""
    c = g4_codes(W)
    M, K = c.shape
    g = np.arange(K) // group
    z = 8 if zeros is None else zeros.astype(np.int64)[:, g]
    cz = (c - z).reshape(M, K // 32, 32)
    s = np.asarray(scales, np.float64)[:, np.arange(K // 32) * 32 // group]
    d, _, q = unpack_q8_1(Xq)
    dots = np.einsum("mbk,nbk->nmb", cz.astype(np.float64), q.astype(np.float64))   # exact: integers below 2^53
    terms = dots * s[None] * d[:, None, :]
    return terms.sum(-1), np.abs(terms).sum(-1)


def moe_g4(W, scales, zeros, group, E, ids, Xq, M):
    """kq_moe_matvec_g4's (Y, B); rows of Xq per token or per (token, slot)."""
    T, top_k = ids.shape
    per_slot = Xq.shape[0] != T
    Y = np.zeros((T, top_k, M))
    B = np.zeros((T, top_k, M))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t) == 0:
            continue
        rows = slice(e * M, (e + 1) * M)
        Y[t, j], B[t, j] = g4_matmul(W[rows], scales[rows], None if zeros is None else zeros[rows], group,
                                     Xq[t * top_k + j if per_slot else t])
    return Y, B
