"""The 4-bit paged cache on the GPU: written byte for byte as the fp32 definition has it, and read back."""
import numpy as np
import pytest

import quantized_weight_matmul_q4_gb300 as kq
from _attnutil import f64, heads, page_table, random_cache, table, torch_dtype
from oracle import attn_oracle as ao

pytestmark = pytest.mark.gpu


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _f32(t):
    return t.float().cpu().numpy()


def _rows(want, dtype):
    """fp32 values rounded once to dtype, as fp64."""
    import torch
    return torch.from_numpy(want).to(torch_dtype(dtype)).double().numpy()


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("D,H,P,rot,pairing,pad", [(64, 3, 16, 64, "half", 0), (128, 8, 64, 128, "half", 0),
                                                   (256, 1, 32, 128, "pairs", 0), (128, 2, 16, 32, "pairs", 8),
                                                   (64, 5, 256, 0, "half", 1), (256, 4, 16, 256, "half", 0)])
def test_append_and_gather(dtype, D, H, P, rot, pairing, pad):
    rng = np.random.default_rng(D + H + P)
    lens, had = [P + 7, 1, 0, 3 * P], [5, 0, 4, 16]       # tokens now, and before
    seq = np.repeat(np.arange(4), lens)
    pos = np.concatenate([h + np.arange(n) for h, n in zip(had, lens)]).astype(np.int32)
    order = rng.permutation(len(seq))                     # tokens of a batch in any order
    seq, pos = seq[order].astype(np.int32), pos[order]
    pages, t = page_table(rng, [a + b for a, b in zip(lens, had)], P, extra_columns=1)
    cache = random_cache(rng, pages, H, P, D)
    N = len(seq)
    K, V = heads(rng, N, H, D, dtype, pad), heads(rng, N, H, D, dtype, 3 * pad)
    cs = table(500, rot) if rot else None
    got = kq.kq_kv_append_q4(K, V, _dev(cache), _dev(t), _dev(pos), seq_ids=_dev(seq),
                             cos_sin=_dev(cs) if rot else None, pairing=pairing)
    ao.append(cache, t, P, ao.turn_fp32(_f32(K), cs[pos] if rot else None, pairing), _f32(V), pos, seq)
    assert np.array_equal(got.cpu().numpy(), cache)       # every byte, those of no token as they were
    for out in ("fp32", "fp16", "bf16"):
        rows = kq.kq_kv_gather_q4(got, _dev(t), _dev(pos), seq_ids=_dev(seq), dtype=torch_dtype(out))
        for i in range(4):
            for x, (s, m, c) in zip(rows, ao.read(cache, t[i], P, pos[seq == i])):
                # s * c is exact in fp32, the sum is rounded once.
                want = ((s[..., None] * c).astype(np.float32) + m[..., None].astype(np.float32)).reshape(-1, H, D)
                assert np.array_equal(f64(x)[seq == i], _rows(want, out)), (out, i)
    assert kq.kq_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_tokens(dtype):
    """Enough tokens that a group of lanes takes four heads, with an odd number of heads."""
    rng = np.random.default_rng(11)
    N, H, D, P = 6000, 5, 128, 64
    pages, t = page_table(rng, [N], P)
    cache = np.zeros(kq.kv_cache_q4_shape(pages, H, P, D), np.uint8)
    K, V = heads(rng, N, H, D, dtype), heads(rng, N, H, D, dtype)
    pos, seq, cs = np.arange(N, dtype=np.int32), np.zeros(N, np.int32), table(N, D)
    got = kq.kq_kv_append_q4(K, V, _dev(cache), _dev(t), _dev(pos), seq_ids=_dev(seq), cos_sin=_dev(cs))
    k, v = kq.kq_kv_gather_q4(got, _dev(t), _dev(pos), seq_ids=_dev(seq), dtype=torch_dtype("fp32"))
    for x, y in ((ao.turn_fp32(_f32(K), cs, "half"), k), (_f32(V), v)):
        s, m, c = ao.blocks4(x.reshape(N, H, 4, 32))
        want = ((s.astype(np.float32)[..., None] * c).astype(np.float32) + m.astype(np.float32)[..., None]).reshape(N, H, D)
        assert np.array_equal(_f32(y), want)


def test_blocks_at_their_limits():
    """Constant blocks, least and largest values, quotients at a half, infinities and NaN."""
    import torch
    rng = np.random.default_rng(12)
    D, H, P = 128, 1, 16
    x = np.zeros((16, 1, 4, 32), np.float32)
    x[0] = 1.5
    x[1, 0, :, 3] = [np.inf, -np.inf, np.nan, 65504]
    x[2] = rng.standard_normal((4, 32)) * 1e-7
    x[3] = rng.standard_normal((4, 32)) * 1e-40
    x[4] = rng.uniform(-65504, 65504, (4, 32))
    x[5, 0, :, 0] = [65520, -65520, 1e6, -1e30]
    x[6] = np.arange(128).reshape(4, 32) % 31                     # quotients of whole numbers by 2
    x[7] = (np.arange(128).reshape(4, 32) % 31) / 2 - 3
    x[8, 0, :, 31] = [2.0 ** -24, 7 * 2.0 ** -24, 2.0 ** -22, 2.0 ** -14]
    x[9] = 3e38 * np.sign(rng.standard_normal((4, 32)))
    x[10] = -np.arange(128).reshape(4, 32)
    x[11] = np.where(rng.random((4, 32)) < 0.5, 0.0, 15 * 1.25)
    x[12:] = rng.standard_normal((4, 1, 4, 32)) * 10.0 ** rng.uniform(-6, 4, (4, 1, 4, 1))
    x = x.reshape(16, 1, D)
    pos, seq, t = np.arange(16, dtype=np.int32), np.zeros(16, np.int32), np.zeros((1, 1), np.int32)
    cache = np.full(kq.kv_cache_q4_shape(1, H, P, D), 0xAB, np.uint8)
    got = kq.kq_kv_append_q4(_dev(x), _dev(x), _dev(cache), _dev(t), _dev(pos), seq_ids=_dev(seq)).cpu().numpy()
    ao.append(cache, t, P, x, x, pos, seq)
    # A NaN's bits are not compared, all else is.
    for at in (0, 10 * D):
        assert np.array_equal(got[..., at:at + 8 * D], cache[..., at:at + 8 * D])
        a, b = (np.ascontiguousarray(c[..., at + 8 * D:at + 10 * D]).view(np.float16) for c in (got, cache))
        assert np.array_equal(a, b, equal_nan=True)
    k, _ = kq.kq_kv_gather_q4(_dev(got), _dev(t), _dev(pos), seq_ids=_dev(seq), dtype=torch.float32)
    assert np.isnan(_f32(k)[1].reshape(4, 32)).all(1).tolist() == [True, True, True, False]


def test_quotients_next_to_a_half():
    """Blocks with s a power of two, whose values lie on and one step beside the halves between codes."""
    rng = np.random.default_rng(13)
    N, D, P = 256, 64, 16
    half = (np.arange(30) % 15 + 0.5).astype(np.float32)
    x = np.zeros((N, 2, 32), np.float32)
    x[:, :, 1] = 15.0
    x[:, :, 2:] = half
    x[1::3, :, 2:] = np.nextafter(half, np.float32(99))
    x[2::3, :, 2:] = np.nextafter(half, np.float32(-99))
    # (15 - 0) * fl(1 / 15) is 1 to fp16, so s is 1 times the power of two.
    x = (x * np.float32(2.0) ** rng.integers(-8, 9, (N, 1, 1))).reshape(N, 1, D).astype(np.float32)
    pages, t = page_table(rng, [N], P)
    pos, seq = np.arange(N, dtype=np.int32), np.zeros(N, np.int32)
    cache = np.zeros(kq.kv_cache_q4_shape(pages, 1, P, D), np.uint8)
    got = kq.kq_kv_append_q4(_dev(x), _dev(-x), _dev(cache), _dev(t), _dev(pos), seq_ids=_dev(seq)).cpu().numpy()
    ao.append(cache, t, P, x, -x, pos, seq)
    assert np.array_equal(got, cache)


def test_tokens_that_have_no_place():
    import torch
    rng = np.random.default_rng(14)
    D, H, P, N = 64, 2, 16, 8
    cache = np.full(kq.kv_cache_q4_shape(4, H, P, D), 3, np.uint8)
    t = np.array([[2, 4], [-1, 0]], np.int32)              # page 4 is not in the cache, page -1 nowhere
    pos = np.array([5, 16, 0, 16, 32, -1, 7, 12], np.int32)
    seq = np.array([0, 0, 1, 1, 0, 0, 2, -1], np.int32)
    K = heads(rng, N, H, D, "fp16")
    got = kq.kq_kv_append_q4(K, K, _dev(cache), _dev(t), _dev(pos), seq_ids=_dev(seq))
    assert kq.kq_get_device_error() == kq.KQ_DEVERR_PAGE
    want = cache.copy()
    keep = [0, 3]                                          # the places that there are
    ao.append(want, t, P, _f32(K)[keep], _f32(K)[keep], pos[keep], seq[keep])
    assert np.array_equal(got.cpu().numpy(), want)
    k = torch.full((N, H, D), 7.0, device="cuda")
    v = k.clone()
    kq.kq_kv_gather_q4(got, _dev(t), _dev(pos), seq_ids=_dev(seq), K=k, V=v)
    assert kq.kq_get_device_error() == kq.KQ_DEVERR_PAGE
    assert [bool((k[n] == 7).all()) for n in range(N)] == [n not in keep for n in range(N)]
    # A padded batch: tokens without a place are no error.
    pos2 = np.array([5, -1, -1, 16, -5, -1, -1, -1], np.int32)
    got = kq.kq_kv_append_q4(K, K, _dev(cache), _dev(t), _dev(pos2), seq_ids=_dev(seq))
    assert kq.kq_get_device_error() == 0 and np.array_equal(got.cpu().numpy(), want)
    # A position that the table of cosines does not have: neither key nor value is written.
    got = kq.kq_kv_append_q4(K, K, _dev(cache), _dev(t), _dev(pos2), seq_ids=_dev(seq), cos_sin=_dev(table(16, 64)))
    assert kq.kq_get_device_error() == kq.KQ_DEVERR_POSITION
    want = cache.copy()
    ao.append(want, t, P, ao.turn_fp32(_f32(K)[:1], table(16, 64)[5:6], "half"), _f32(K)[:1], pos[:1], seq[:1])
    assert np.array_equal(got.cpu().numpy(), want)


def test_one_token_each_without_seq_ids():
    rng = np.random.default_rng(15)
    D, H, P, B = 128, 2, 32, 9
    lens = [int(n) for n in rng.integers(1, 100, B)]
    pages, t = page_table(rng, lens, P)
    cache = random_cache(rng, pages, H, P, D)
    pos = np.array(lens, np.int32) - 1
    K, V = heads(rng, B, H, D, "bf16"), heads(rng, B, H, D, "bf16")
    got = kq.kq_kv_append_q4(K, V, _dev(cache), _dev(t), _dev(pos))
    ao.append(cache, t, P, _f32(K), _f32(V), pos, np.arange(B))
    assert np.array_equal(got.cpu().numpy(), cache)


def test_offsets_past_32_bits():
    """Places whose bytes lie beyond the first 4 GiB of a cache."""
    import torch
    D, H, P = 256, 8, 64
    pages = (5 << 30) // (H * P * 20 * D // 16)
    cache = torch.empty(kq.kv_cache_q4_shape(pages, H, P, D), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(16)
    K, V = heads(rng, 3, H, D, "bf16"), heads(rng, 3, H, D, "bf16")
    t = torch.tensor([[pages - 1], [0], [pages * 7 // 8]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([63, 1, 17], dtype=torch.int32, device="cuda")
    kq.kq_kv_append_q4(K, V, cache, t, pos)
    k, v = kq.kq_kv_gather_q4(cache, t, pos, dtype=torch.float32)
    for x, y in ((K, k), (V, v)):
        s, m, c = ao.blocks4(_f32(x).reshape(3, H, 8, 32))
        want = ((s.astype(np.float32)[..., None] * c).astype(np.float32) + m.astype(np.float32)[..., None]).reshape(3, H, D)
        assert np.array_equal(_f32(y), want)
    small = cache[pages - 1:].cpu().numpy()
    assert np.array_equal(_f32(k)[0], sum_blocks(ao.read(small, np.zeros(4, np.int64), P, [63])[0], H, D))


def sum_blocks(smc, H, D):
    s, m, c = smc
    return ((s[..., None] * c).astype(np.float32) + m[..., None].astype(np.float32)).reshape(H, D)
