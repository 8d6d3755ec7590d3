"""Inputs shared by the tests of the attention-side operators of a decode step."""
import numpy as np

HALF = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}   # half a step, relative
U32 = 2.0 ** -24


def torch_dtype(name):
    import torch
    return {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}[name]


def f64(t):
    return t.detach().cpu().double().numpy()


def table(n, rot, base=10000.0):
    """Cosines and sines of n positions, fp32 [n, rot]."""
    a = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def heads(rng, N, H, D, dtype, pad=0):
    """A view [N, H, D] of rows H * D + pad elements apart, some channels of it large."""
    import torch
    x = rng.standard_normal((N, H * D + pad)) * np.where(rng.random(H * D + pad) < 0.05, 6.0, 1.0)
    t = torch.from_numpy(x.astype(np.float32)).cuda().to(torch_dtype(dtype))
    return t[:, :H * D].unflatten(1, (H, D))


def random_cache(rng, pages, H, page_size, D, garbage=True):
    """A cache uint8 [pages, H, page / 16, 20 D] of bell-shaped codes, its parameters of mixed signs of m."""
    G = D // 32
    c = rng.integers(0, 256, (pages, H, page_size // 16, 20 * D), dtype=np.uint8)
    for at, size in ((0, 0.2), (10 * D, 0.1)):
        s = (size * np.exp(0.5 * rng.standard_normal((pages, H, page_size // 16, 16, G)))).astype(np.float16)
        m = (-7.5 * s.astype(np.float64) + 0.3 * rng.standard_normal(s.shape)).astype(np.float16)
        par = np.concatenate([s, m], -1).reshape(pages, H, page_size // 16, 32 * G)
        c[..., at + 8 * D:at + 10 * D] = np.ascontiguousarray(par).view(np.uint8)
    return c


def page_table(rng, lengths, page_size, spare=3, extra_columns=0):
    """(pages, table int32 [sequences, most + extra]): distinct random pages; entries that no length reaches are out of range."""
    need = [-(-max(0, n) // page_size) for n in lengths]
    pages = sum(need) + spare
    perm = rng.permutation(pages)
    t = np.full((len(need), max(1, max(need)) + extra_columns), -7, np.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = perm[at:at + n]
        at += n
    return pages, t
