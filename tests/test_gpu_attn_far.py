"""kq_attn_q4 where scores, weights or parameters are far from the usual ones, and in tables whose older pages are gone."""
import numpy as np
import pytest

import quantized_weight_matmul_q4_gb300 as kq
from _attnutil import HALF, f64, random_cache, torch_dtype
from oracle import attn_oracle as ao
from test_gpu_attn import SCORE, _bound, _case, _dev, _run

pytestmark = pytest.mark.gpu


def bound(o, E, S, dtype, places, fine):
    """Largest error of an output. 16-bit rows: weights rounded to fp16 (half a step, 2^-11) in the sum and in the total, their products
    with s or m + 8 s once more: 3 * 2^-11, and 2^-19 for the exponential; of Sum p (s c + |m|) 2^-16 that the tensor cores' sums of 8 s p
    and s c p cut off (twice 17 addends a granule, a step of 2^-22 at most each); else, and the rounding to the row's type, as there."""
    if fine or dtype == "fp32":
        b = _bound(o, E, S, dtype, places, True)
    else:
        b = (3 * 2.0 ** -11 + 2.0 ** -19 + np.expm1(2 * SCORE * S[..., None]) + (places / 16 + 1) * 2.0 ** -22) * E[0] + 2.0 ** -16 * E[1] + 1e-30
    return b + HALF[dtype] * (np.abs(o) + b) + (2.0 ** -25 if dtype == "fp16" else 0)


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


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("Xq", [False, True])
def test_many_light_places_beside_a_large_block(dtype, Xq):
    """A few heavy places and some 10^5 with 2^-19 of their weight, in runs of thousands of places, and a block of a very large s that
    no row gives weight to. Values are constant in a block: o is the share of the light places in the total."""
    import torch
    D, P, L, B = 64, 65536, 131072, 512
    rng = np.random.default_rng(3)
    cache = random_cache(rng, 2, 1, P, D)
    place = np.arange(L).reshape(2, 1, P // 16, 16)
    k = np.where(place % 32768 == 77, 0.0, np.log(0.9) - 19 * np.log(2))
    k[place % 4096 == 5] = -100.0
    v = np.where(place % 32768 == 77, -1.0, 1.0)
    v[place % 4096 == 5] = 0.0
    constant_blocks(cache, False, k)
    constant_blocks(cache, True, v)
    s = cache[..., 18 * D:].view(np.float16).reshape(2, 1, P // 16, 16, 2, 2)
    s[place % 4096 == 5, 0] = 60000.0
    Q = torch.ones(B, 1, D, device="cuda", dtype=torch_dtype(dtype))
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").expand(B, 2).contiguous()
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    O, _ = kq.kq_attn_q4(Q, _dev(cache), table, lens, scale=1 / D, Xq=Xq)
    o, E, S = ao.attention(f64(Q[:1]), cache, np.array([[0, 1]]), P, [L], scale=1 / D)
    assert abs(o[0, 0, 0]) < 0.95
    assert np.all(np.abs(f64(O) - o) <= bound(o, E, S, dtype, L, Xq))


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("Xq", [False, True])
@pytest.mark.parametrize("least,most,floor", [(2.0 ** -24, 2.0 ** -14, 2.0 ** -23), (2.0 ** -16, 2.0 ** -6, 2.0 ** -23), (1.0, 30.0, 2.0 ** -20)])
def test_values_of_every_size(dtype, Xq, least, most, floor):
    """Values next to fp16's least numbers, and ones whose s is 2 and more: m + 8 s to within an absolute error of `floor`, and the products
    of weights with s to (1 + s) S 2^-35 of the largest weight, |c - 8| times that, for each of the places."""
    D, P, lens = 128, 16, [200, 37, 1]
    cache, t, Q, n, start = _case(int(1 / least) % 1000, D, 2, 4, P, lens, dtype=dtype)
    rng = np.random.default_rng(5)
    s = (least * (most / least) ** rng.random((*cache.shape[:3], 16, D // 32))).astype(np.float16)
    m = (-15 * s.astype(np.float64) * rng.random(s.shape)).astype(np.float16)
    cache[..., 18 * D:] = np.ascontiguousarray(np.concatenate([s, m], -1).reshape(*cache.shape[:3], -1)).view(np.uint8)
    O, _ = _run(cache, t, Q, n, start, Xq=Xq)
    o, E, S = ao.attention(f64(Q), cache, t, P, lens)
    top = max(1.0, 2.0 ** np.ceil(np.log2(most)))
    tol = bound(o, E, S, dtype, max(lens), Xq) + (1 + HALF[dtype]) * (floor + max(lens) * 8 * (1 + top) * top * 2.0 ** -35)
    assert np.all(np.abs(f64(O) - o) <= tol), (np.abs(f64(O) - o) / tol).max()


@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("dtype,new", [("bf16", None), ("fp32", [1, 3, 2])])
def test_pages_older_than_the_window_may_be_gone(P, dtype, new):
    """A window that begins in the second half of 32 places, whose first half's page is no longer in the table."""
    lens, window = [63, 130, 97], 14
    case = _case(P, 128, 2, 4, P, lens, new, dtype=dtype)
    want, _ = _run(*case, window=window)
    t = case[1].copy()
    for b, n in enumerate(lens):
        first = n - (new[b] if new else 1) + 1 - window
        t[b, :first // P] = -1
    got, _ = _run(case[0], t, *case[2:], window=window)
    assert np.array_equal(f64(got), f64(want))
    assert kq.kq_get_device_error() == 0
    # One that is seen is recorded.
    t[1, (lens[1] - 1) // P] = -1
    _run(case[0], t, *case[2:], window=window)
    assert kq.kq_get_device_error() == kq.KQ_DEVERR_PAGE


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,H,group,P", [(64, 8, 16, 256), (128, 3, 16, 32), (256, 8, 7, 16)])
def test_rows_of_one_place_whose_parts_cancel(dtype, D, H, group, P):
    """Scores of a hundred and more give one place all of the weight; where its value is next to 0, s c and m are many times that, and
    what is cut off of their sums is all the error there is."""
    lens = [16] * 24 + [309, 100, 15, 1, 2, 371]
    for seed in range(6):
        case = _case(seed, D, H, group, P, lens, dtype=dtype, size=3.0)
        O, _ = _run(*case)
        o, E, S = ao.attention(f64(case[2]), case[0], case[1], P, lens)
        err, tol = np.abs(f64(O) - o), bound(o, E, S, dtype, max(lens), False)
        assert np.all(err <= tol), (err / tol).max()
