"""kq_attn_q4 where scores, weights or parameters are far from the usual ones."""
import numpy as np
import pytest

from _attnutil import f64
from oracle import attn_oracle as ao
from test_gpu_attn import _case, _run

pytestmark = pytest.mark.gpu


def constant_blocks(cache, values, m):
    """Sets the parameters of keys or values (s = 0): block values m [pages, H, page / 16, 16] in every block of a place."""
    D = cache.shape[-1] // 20
    G, at = D // 32, 10 * D * values + 8 * D
    par = np.zeros((*m.shape, 2, G), np.float16)
    par[..., 1, :] = m[..., None]
    cache[..., at:at + 2 * D] = np.ascontiguousarray(par).view(np.uint8).reshape(*cache.shape[:3], 2 * D)


def rising_keys(case, P):
    """Keys (all elements of a place alike) that rise with the place in its sequence, all above 0: 1, 1 1/64, ..."""
    cache, t, _, lens, _ = case
    m = np.ones(cache.shape[:3] + (16,))
    for b, n in enumerate(lens):
        for p in range(n):
            m[t[b, p // P], :, p % P // 16, p % 16] = 1 + p / 64
    constant_blocks(cache, False, m)


@pytest.mark.parametrize("dtype,q,scale", [("fp32", 1e29, None), ("fp32", 1e32, None), ("fp32", 3e35, None), ("bf16", 1e32, None),
                                           ("bf16", 2.0, 9e29), ("fp16", 1000.0, 1e29), ("fp32", -1e20, -1e15)])
@pytest.mark.parametrize("D,group,P,lens", [(128, 4, 16, [1, 17, 200]), (64, 3, 32, [700, 2]), (256, 8, 16, [90, 33])])
def test_scores_far_below_zero(dtype, q, scale, D, group, P, lens):
    """All scores beyond -1e30: the place whose score is the largest has all of the weight."""
    import torch
    case = _case(D + group, D, 1, group, P, lens, dtype=dtype)
    rising_keys(case, P)
    Q = torch.full_like(case[2], -q)
    want = np.concatenate([(v[1][..., None] + v[0][..., None] * v[2]).reshape(1, 1, D)
                           for b in range(len(lens)) for v in ao.read(case[0], case[1][b], P, [0])[1:]])
    for Xq in (False, True):
        O, _ = _run(case[0], case[1], Q, *case[3:], scale=scale, Xq=Xq)
        # Half a step of bf16, and 2^-10 of |s| |c - 8| + |m + 8 s| < 4 for weights of 16 bits.
        assert np.all(np.abs(f64(O) - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -8), np.abs(f64(O) - want).max()


def test_scores_beyond_fp32():
    """Above its range, or all below it: NaN. Rows beside them, and rows that see no place, are not touched by it."""
    import torch
    lens, new = [40, 1, 3], [2, 1, 5]
    case = _case(1, 128, 2, 4, 16, lens, new, dtype="fp32")
    rising_keys(case, 16)
    Q = case[2].clone()
    want, _ = _run(*case, scale=1e20)
    Q[:, 3], Q[:, 6] = -3e35, 3e35
    for Xq in (False, True):
        O, _ = _run(case[0], case[1], Q, *case[3:], scale=1e20, Xq=Xq)
        sees = torch.tensor([1, 1, 1, 0, 0, 1, 1, 1], dtype=torch.bool, device="cuda")
        assert bool(torch.isnan(O[sees][:, [3, 6]]).all()) and not O[~sees].any()
        rest = [0, 1, 2, 4, 5, 7]
        assert torch.allclose(O[:, rest], want[:, rest], rtol=2.0 ** -16, atol=2.0 ** -16)      # (one place's values)
    # Of many places, in parts of several warps and CTAs.
    case = _case(2, 64, 1, 2, 64, [9000], dtype="fp32")
    rising_keys(case, 64)
    for size, nan in ((-3e35, True), (-1e15, False)):
        O, _ = _run(case[0], case[1], torch.full_like(case[2], size), *case[3:], scale=1e20)
        assert bool(torch.isnan(O).all()) == nan and (nan or bool(torch.isfinite(O).all()))
