"""kq_attn_q4 on the GPU against its fp64 definition."""
import numpy as np
import pytest

import quantized_weight_matmul_q4_gb300 as kq
from _attnutil import HALF, U32, f64, page_table, random_cache, torch_dtype
from _decodeutil import assert_q8_blocks  # noqa: F401  (the Q8_1 layout)
from oracle import attn_oracle as ao
from oracle import decode_oracle as deo

pytestmark = pytest.mark.gpu

# Relative error of a weight p (but for that of its score): exponential 2 ulp and a few products, below 2^-20; rounded to fp16
# for the tensor cores where rows are fp16 or bf16 (half a step, 2^-12) in the values' sum and in the total (their quotient: 2^-11),
# the product with s once more, and m + 8 s: 2^-10 in all. Split into two halves in fp32 rows, and where Q8_1 rows are asked
# for: 2^-23 each time.
WEIGHT = {"fp32": 2.0 ** -19, "fp16": 2.0 ** -10 + 2.0 ** -19, "bf16": 2.0 ** -10 + 2.0 ** -19}
# Error of a score, relative to scale * Sum (|s| c + |m|) |q|: exact products, sums in fp32 of at most
# 256 terms whose additions may each cut off a step (2^-23), most of them within 16 by a tree: 2^-18.
SCORE = 2.0 ** -18


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bound(o, E, S, dtype, places, fine=False):
    """Largest error of an unrounded output: that of the weights; scores off by d change them by 2 d at most; the sums of
    a granule of 16 places are products with the codes as they are (two or four additions that may cut off a step), and are added up
    (n granules, one or two additions each)."""
    d, n = SCORE * S[..., None], places / 16 + 1
    w = WEIGHT["fp32" if fine else dtype]
    return (w + np.expm1(2 * d) + n * 2.0 ** -22) * E[0] + 2.0 ** -21 * E[1] + 1e-30


def _check(got, o, E, S, dtype, what, places=4096, fine=False):
    tol = _bound(o, E, S, dtype, places, fine)
    tol = tol + HALF[dtype] * (np.abs(o) + tol) + (2.0 ** -25 if dtype == "fp16" else 0)
    err = np.abs(got - o)
    assert np.all(err <= tol), f"{what}: {np.nanmax(err / tol)} times the bound"


def _check_q8(Xq, o, tol, what):
    """Q8_1 blocks of values within tol of o (both [N, K])."""
    N, K = o.shape
    d_h, s_h, q = deo.unpack_q8_1(Xq)
    b, t = o.reshape(N, -1, 32), tol.reshape(N, -1, 32)
    d, dt = np.abs(b).max(-1) / 127, t.max(-1) / 127
    assert np.all(np.abs(d_h - d) <= dt + (d + dt) * (2.0 ** -11 + 4 * U32) + 2.0 ** -25), what
    with np.errstate(divide="ignore", invalid="ignore"):
        live = d > 1e-30
        at = np.where(live[..., None], b / d[..., None], 0)
        slack = np.where(live[..., None], t / d[..., None] + np.abs(at) * (dt / np.maximum(d - dt, 1e-30))[..., None], 0) + 127 * 4 * U32
    assert np.all(np.abs(q - at)[live] <= 0.5 + slack[live]), what
    want = (d_h.astype(np.float32) * q.sum(-1).astype(np.float32)).astype(np.float16).astype(np.float64)
    assert np.array_equal(s_h, want), what


def _case(seed, D, H, group, P, lens, new=None, dtype="bf16", size=1.0, **kw):
    rng = np.random.default_rng(seed)
    pages, t = page_table(rng, lens, P)
    cache = random_cache(rng, pages, H, P, D)
    n = new if new is not None else [1] * len(lens)
    Q = (size * rng.standard_normal((sum(n), H * group, D))).astype(np.float32)
    Q = _dev(Q).to(torch_dtype(dtype))
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32) if new is not None else None
    return cache, t, Q, np.array(lens, np.int32), start


def _run(cache, t, Q, lens, start, **kw):
    return kq.kq_attn_q4(Q, _dev(cache), _dev(t), _dev(lens), q_start=_dev(start) if start is not None else None, **kw)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("D,H,group,P,lens", [
    (128, 2, 4, 16, [1]), (128, 1, 1, 16, [15, 16, 17, 2]), (64, 3, 5, 32, [33, 1, 100]), (256, 1, 8, 16, [40, 300]),
    (128, 2, 7, 64, [64, 65, 63, 1000]), (64, 1, 12, 16, [257, 5]), (256, 2, 16, 128, [129, 128]), (128, 4, 8, 16, [3001]),
    (64, 8, 1, 16, [500, 31, 77, 1, 16]), (128, 1, 20, 32, [70]), (64, 2, 32, 16, [333, 48])])
def test_one_new_row_each(dtype, D, H, group, P, lens):
    case = _case(D + group + len(lens), D, H, group, P, lens, dtype=dtype)
    O, Xq = _run(*case, Xq=True)
    o, E, S = ao.attention(f64(case[2]), case[0], case[1], P, lens)
    _check(f64(O), o, E, S, dtype, "O", max(lens), True)
    plain, _ = _run(*case)
    _check(f64(plain), o, E, S, dtype, "O without Xq", max(lens))
    tol = _bound(o, E, S, dtype, max(lens), True)
    _check_q8(Xq.cpu().numpy(), o.reshape(len(lens), -1), tol.reshape(len(lens), -1), "Xq")
    assert kq.kq_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("window", [0, 1, 20, 64])
@pytest.mark.parametrize("D,H,group,P,lens,new", [
    (128, 2, 4, 16, [50, 7, 130], [3, 7, 1]), (64, 1, 3, 32, [33, 40], [5, 9]), (256, 1, 1, 16, [90], [17]),
    (128, 1, 8, 64, [200, 64, 65], [6, 0, 2]), (64, 2, 7, 16, [48, 100], [48, 1])])
def test_several_new_rows(dtype, window, D, H, group, P, lens, new):
    case = _case(D + group + window, D, H, group, P, lens, new, dtype=dtype)
    O, _ = _run(*case, window=window)
    o, E, S = ao.attention(f64(case[2]), case[0], case[1], P, lens, q_start=case[4], window=window)
    _check(f64(O), o, E, S, dtype, "O")


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("D,H,group,P,lens,new,window", [
    (128, 2, 4, 16, [250, 70, 3], [40, 33, 3], 0), (64, 1, 65, 32, [333], [1], 0), (128, 1, 16, 64, [65, 0, 900], [9, 0, 7], 50),
    (128, 1, 33, 16, [2000, 2001], [2, 3], 0), (64, 3, 5, 16, [90, 17, 64, 1], [60, 17, 1, 1], 30), (128, 8, 8, 128, [700], [9], 0)])
def test_many_pairs_of_row_and_head(dtype, D, H, group, P, lens, new, window):
    """More than 64 (row, query head) pairs of a key head: tiles of 16; with one sequence whose tiles several CTAs share."""
    case = _case(D + group, D, H, group, P, lens, new, dtype=dtype)
    o, E, S = ao.attention(f64(case[2]), case[0], case[1], P, lens, q_start=case[4], window=window)
    O, Xq = _run(*case, window=window, Xq=True)
    _check(f64(O), o, E, S, dtype, "O", max(lens), True)
    tol = _bound(o, E, S, dtype, max(lens), True)
    _check_q8(Xq.cpu().numpy(), o.reshape(sum(new), -1), tol.reshape(sum(new), -1), "Xq")
    _check(f64(_run(*case, window=window)[0]), o, E, S, dtype, "O without Xq", max(lens))


def test_rows_that_see_nothing():
    """Sequences without places, with fewer places than new rows, and of negative length: zeros in both outputs."""
    lens, new = [0, 2, 5, -3, 40], [2, 4, 1, 1, 2]
    case = _case(1, 128, 2, 4, 16, lens, new)
    O, Xq = _run(*case, Xq=True)
    o, E, S = ao.attention(f64(case[2]), case[0], case[1], 16, lens, q_start=case[4])
    _check(f64(O), o, E, S, "bf16", "O")
    empty = [0, 1, 2, 3, 7]
    assert not f64(O)[empty].any() and not Xq.cpu().numpy()[empty].any()
    case = _case(2, 64, 1, 4, 16, [0, 0])
    assert not f64(_run(*case)[0]).any()


def test_rows_of_no_sequence_are_left_as_they_were():
    import torch
    case = list(_case(3, 128, 2, 4, 16, [30, 20], [2, 3]))
    Q = torch.cat([case[2], torch.full_like(case[2][:4], float("nan"))])
    O = torch.full_like(Q, 7.0)
    Xq = torch.full((9, 8 * 128 // 32, 36), 9, dtype=torch.uint8, device="cuda")
    _run(case[0], case[1], Q, case[3], case[4], O=O, Xq=Xq)
    want, wq = _run(*case, Xq=True)
    assert torch.equal(O[:5], want) and bool((O[5:] == 7).all())
    assert torch.equal(Xq[:5], wq) and bool((Xq[5:] == 9).all())


def test_places_behind_the_end_are_not_used():
    """Codes and parameters of places that no token was written to: NaN and infinities everywhere."""
    lens = [5, 17, 32, 63]
    case = _case(4, 128, 2, 4, 32, lens)
    want, _ = _run(*case)
    cache, D = case[0].copy(), 128
    bad = np.full(8, np.nan, np.float16)
    bad[1::3] = np.inf
    for page in range(cache.shape[0]):
        for g in range(2):
            for r in range(16):
                used = any(p * 32 + g * 16 + r < n and case[1][b, p] == page for b, n in enumerate(lens)
                           for p in range(case[1].shape[1]))
                if not used:
                    for at in (8 * D, 18 * D):
                        cache[page, :, g, at + 16 * r:at + 16 * (r + 1)] = bad.view(np.uint8)
    got, _ = _run(cache, *case[1:])
    assert np.array_equal(f64(got), f64(want))
    # And a window's older places, whose pages may be gone from the table.
    t = case[1].copy()
    t[3, 0] = -5
    got, _ = _run(case[0], t, *case[2:], window=20)
    want, _ = _run(*case, window=20)
    assert np.array_equal(f64(got), f64(want)) and kq.kq_get_device_error() == 0


def test_values_that_are_not_numbers_reach_the_rows_that_see_them():
    """A token with an infinity among its values, later than some rows' places: those rows do not see it."""
    import torch
    D, H, P, n, L = 128, 1, 16, 4, 30
    case = _case(5, D, H, 4, P, [L], [n])
    K, V = torch.randn(1, H, D, device="cuda"), torch.randn(1, H, D, device="cuda")
    at = torch.tensor([L - 2], dtype=torch.int32, device="cuda")
    for keys in (False, True):
        x = (K if keys else V).clone()
        x[0, 0, 33] = float("inf")
        cache = _dev(case[0])
        kq.kq_kv_append_q4(x if keys else K, V if keys else x, cache, _dev(case[1]), at)
        O = f64(kq.kq_attn_q4(case[2], cache, _dev(case[1]), _dev(case[3]), q_start=_dev(case[4]))[0])
        assert np.isfinite(O[:2]).all()
        if keys:
            assert np.isnan(O[2:]).all()
        else:
            assert np.isnan(O[2:, :, 32:64]).all() and np.isfinite(O[2:, :, :32]).all() and np.isfinite(O[2:, :, 64:]).all()


def test_queries_that_are_not_numbers_stay_in_their_rows():
    import torch
    case = list(_case(6, 64, 2, 4, 16, [40, 50], [3, 2]))
    want, _ = _run(*case)
    Q = case[2].clone()
    Q[1, 5, 7], Q[3, 0, 0] = float("nan"), float("inf")
    got, _ = _run(case[0], case[1], Q, case[3], case[4])
    bad = torch.zeros_like(want, dtype=torch.bool)
    bad[1, 5], bad[3, 0] = True, True
    assert torch.equal(got[~bad], want[~bad])
    assert torch.isnan(got[1, 5]).all() and not torch.isfinite(got[3, 0]).any()


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-3, 30.0, 1e4])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_queries_of_any_size(dtype, size):
    """From equal weights for all tokens to one token alone."""
    case = _case(7, 128, 2, 4, 16, [200, 31], dtype=dtype, size=size)
    O, _ = _run(*case)
    o, E, S = ao.attention(f64(case[2]), case[0], case[1], 16, [200, 31])
    if size >= 30:                     # scores of hundreds: where their error passes a unit, nothing is claimed
        ok = SCORE * S[..., None] < 0.1
    else:
        ok = np.ones_like(S[..., None], bool)
    tol = _bound(o, E, np.where(ok[..., 0], S, 0), dtype, 200)
    tol = tol + HALF[dtype] * (np.abs(o) + tol)
    assert np.all((np.abs(f64(O) - o) <= tol) | ~ok)


def test_values_of_very_different_sizes():
    """Parameters over fp16's whole range, in one sequence and between tokens of a tile."""
    rng = np.random.default_rng(8)
    cache, t, Q, lens, _ = _case(9, 64, 1, 4, 16, [100, 40])
    D, G = 64, 2
    s = (10.0 ** rng.uniform(-7, 4.5, (*cache.shape[:3], 16, G))).astype(np.float16)
    m = (-8 * s.astype(np.float64) * rng.uniform(0, 1, s.shape)).clip(-65504, 65504).astype(np.float16)
    cache[..., 18 * D:] = np.ascontiguousarray(np.concatenate([s, m], -1).reshape(*cache.shape[:3], -1)).view(np.uint8)
    for dtype in ("fp32", "bf16"):
        q = Q.to(torch_dtype(dtype))
        o, E, S = ao.attention(f64(q), cache, t, 16, lens)
        # Scales far below the largest seen so far are rounded relative to that one: 2^-38 of it.
        far = 2.0 ** -38 * 65504 * 16
        got, _ = kq.kq_attn_q4(q, _dev(cache), _dev(t), _dev(lens))
        tol = _bound(o, E, S, dtype, 100) + far
        assert np.all(np.abs(f64(got) - o) <= tol + HALF[dtype] * (np.abs(o) + tol))


def test_scale_and_strides_and_shared_query_rows():
    import torch
    case = _case(10, 128, 2, 4, 16, [90, 33], dtype="fp16")
    wide = torch.zeros(2, 12, 128, dtype=torch.float16, device="cuda")
    wide[:, 2:10] = case[2]
    out = torch.full((2, 11, 128), 3.0, dtype=torch.float16, device="cuda")
    O, _ = _run(case[0], case[1], wide[:, 2:10], *case[3:], scale=0.3, O=out[:, :8])
    o, E, S = ao.attention(f64(case[2]), case[0], case[1], 16, [90, 33], scale=0.3)
    _check(f64(O), o, E, S, "fp16", "O")
    assert bool((out[:, 8:] == 3).all())
    one, _ = _run(case[0], case[1], case[2][:1].expand(2, 8, 128), *case[3:])
    two, _ = _run(case[0], case[1], case[2][:1].repeat(2, 1, 1), *case[3:])
    assert torch.equal(one, two)
    neg, _ = _run(*case, scale=-0.1)
    o, E, S = ao.attention(f64(case[2]), case[0], case[1], 16, [90, 33], scale=-0.1)
    _check(f64(neg), o, E, S, "fp16", "negative scale")


def test_pages_out_of_range_count_as_unseen():
    case = _case(11, 128, 1, 4, 16, [64, 20])
    t = case[1].copy()
    t[0, 1] = case[0].shape[0]
    O, _ = _run(case[0], t, *case[2:])
    assert kq.kq_get_device_error() == kq.KQ_DEVERR_PAGE
    (ks, km, kc), (vs, vm, vc) = ao.read(case[0], case[1][0], 16, [i for i in range(64) if not 16 <= i < 32])
    k, v = ((m[..., None] + s[..., None] * c).reshape(48, 128) for s, m, c in ((ks, km, kc), (vs, vm, vc)))
    for i in range(4):
        x = k @ f64(case[2])[0, i] * 128 ** -0.5
        p = np.exp(x - x.max())
        assert np.allclose(f64(O)[0, i], p @ v / p.sum(), atol=0.02)
    # A length beyond the table's pages.
    lens = case[3].copy()
    lens[1] = 16 * t.shape[1] + 1
    _run(case[0], case[1], case[2], lens, None)
    assert kq.kq_get_device_error() == kq.KQ_DEVERR_PAGE


def test_same_results_every_time_and_from_a_graph():
    import torch
    cache, t, Q, lens, _ = _case(12, 128, 4, 6, 64, [4097, 100, 1, 2500])
    args = (Q, _dev(cache), _dev(t), _dev(lens))
    want, wq = kq.kq_attn_q4(*args, Xq=True)
    ws = torch.full((kq.kq_attn_q4_workspace_bytes(24, 4, 128, 4, 4),), 0xFF, dtype=torch.uint8, device="cuda")
    O, Xq = torch.empty_like(want), torch.empty_like(wq)
    for _ in range(5):
        kq.kq_attn_q4(*args, O=O, Xq=Xq, ws=ws)
        assert torch.equal(O, want) and torch.equal(Xq, wq)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            kq.kq_attn_q4(*args, O=O, Xq=Xq, ws=ws)
    for k in range(4):                                     # other lengths of the same buffers
        n = torch.tensor([4097 - 1000 * k, 100 + k, k, 2500], dtype=torch.int32, device="cuda")
        args[3].copy_(n)
        O.zero_(), g.replay()
        torch.cuda.synchronize()
        want, wq = kq.kq_attn_q4(Q, args[1], args[2], n, Xq=True)
        assert torch.equal(O, want) and torch.equal(Xq, wq)


def test_two_streams_at_once():
    import torch
    a, b = _case(13, 128, 2, 4, 16, [3000, 900]), _case(14, 64, 8, 1, 32, [5000])
    streams = [torch.cuda.Stream() for _ in range(2)]
    want = [_run(*c)[0] for c in (a, b)]
    dev = [(c[2], _dev(c[0]), _dev(c[1]), _dev(c[3])) for c in (a, b)]
    torch.cuda.synchronize()
    got = [[kq.kq_attn_q4(*d, stream=s)[0] for s, d in zip(streams, dev)] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for pair in got for x, w in zip(pair, want))


def test_long_sequence():
    """A sequence in parts of every CTA; many places that count alike, whose codes' sums are far larger than the output."""
    D, H, P, L = 64, 1, 64, 70001
    cache, t, Q, lens, _ = _case(16, D, H, 2, P, [L], dtype="fp32")
    o, E, S = ao.attention(f64(Q), cache, t, P, [L])
    for dtype in ("fp32", "fp16"):
        q = Q.to(torch_dtype(dtype))
        if dtype == "fp16":
            o, E, S = ao.attention(f64(q), cache, t, P, [L])
        O, Xq = kq.kq_attn_q4(q, _dev(cache), _dev(t), _dev(lens), Xq=True)
        _check(f64(O), o, E, S, dtype, "O", L, True)
        tol = _bound(o, E, S, dtype, L, True)
        _check_q8(Xq.cpu().numpy(), o.reshape(1, -1), tol.reshape(1, -1), "Xq")
        O, _ = kq.kq_attn_q4(q, _dev(cache), _dev(t), _dev(lens))
        _check(f64(O), o, E, S, dtype, "O", L)
        # In norm, far below the bound of each element: the roundings are independent of one another.
        assert np.linalg.norm(f64(O) - o) <= (4e-6 if dtype == "fp32" else 2.0 ** -11) * np.linalg.norm(o)


def test_pages_past_32_bits():
    import torch
    D, H, P = 256, 8, 64
    rng = np.random.default_rng(17)
    pages = (5 << 30) // (H * P * 20 * D // 16)
    small = random_cache(rng, 3, H, P, D)
    cache = torch.empty(kq.kv_cache_q4_shape(pages, H, P, D), dtype=torch.uint8, device="cuda")
    at = [pages - 1, 3, pages * 7 // 8]
    for i, p in enumerate(at):
        cache[p] = _dev(small[i])
    Q = torch.randn(1, 2 * H, D, device="cuda", dtype=torch.bfloat16)
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    O, _ = kq.kq_attn_q4(Q, cache, torch.tensor([at], dtype=torch.int32, device="cuda"), lens)
    o, E, S = ao.attention(f64(Q), small, np.array([[0, 1, 2]]), P, [150])
    _check(f64(O), o, E, S, "bf16", "O")


def test_many_sequences():
    """More sequences than a CTA has threads, most of them short, some empty."""
    rng = np.random.default_rng(18)
    lens = [int(n) for n in rng.choice([0, 1, 2, 7, 16, 33, 90], 700)]
    case = _case(19, 64, 2, 3, 16, lens)
    O, _ = _run(*case)
    o, E, S = ao.attention(f64(case[2]), case[0], case[1], 16, lens)
    _check(f64(O), o, E, S, "bf16", "O")


def test_places_next_to_the_last_of_32_bits():
    """Sequences of up to 2^31 - 1 places, all in one page that the table repeats, of which a window is seen."""
    import torch
    D, H, P = 64, 1, 65536
    rng = np.random.default_rng(20)
    page = random_cache(rng, 1, H, P, D)
    lens = [2 ** 31 - 1, 2 ** 31 - 20, 2 ** 31 - 32]
    Q = torch.randn(3, 4, D, device="cuda", dtype=torch.bfloat16)
    O, _ = kq.kq_attn_q4(Q, _dev(page), torch.zeros(3, 2 ** 31 // P, dtype=torch.int32, device="cuda"),
                         torch.tensor(lens, dtype=torch.int32, device="cuda"), window=100)
    # The same places in a short sequence: 2^31 is a multiple of the page, so that these are its last ones.
    o, E, S = ao.attention(f64(Q), page, np.zeros((3, 1), np.int32), P, [n % P for n in lens], window=100)
    _check(f64(O), o, E, S, "bf16", "O")
