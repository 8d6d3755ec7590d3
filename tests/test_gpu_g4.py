"""kq_matvec_g4 and kq_moe_matvec_g4 on the GPU against the fp64 oracle."""
import numpy as np
import pytest

from oracle import decode_oracle as deo
import quantized_weight_matmul_q4_gb300 as kq
from _decodeutil import assert_g4, g4_weights, q8_rows
from _kqutil import to_dev

pytestmark = pytest.mark.gpu


def _dev_weights(W, s, z, scales):
    import torch
    t = torch.float16 if scales == "fp16" else torch.bfloat16
    sd = torch.from_numpy(s).cuda().to(t)
    return to_dev(W, torch), sd, sd.cpu().double().numpy(), None if z is None else to_dev(z, torch)


CASES = [
    # N, M, K, group, zeros, scales
    (1, 1, 32, 32, False, "fp16"),
    (1, 17, 64, 32, True, "bf16"),
    (1, 4096, 4096, 128, False, "fp16"),
    (1, 1000, 11008, 64, True, "fp16"),
    (1, 130, 14336, 1 << 20, True, "bf16"),     # one scale per row
    (1, 333, 1056, 128, True, "fp16"),          # the last group is short
    (1, 70, 18944, 32, True, "bf16"),
    (2, 257, 2048, 128, True, "bf16"),
    (3, 100, 4128, 256, False, "fp16"),
    (4, 515, 768, 64, False, "bf16"),
    (5, 64, 3584, 512, True, "fp16"),
    (7, 200, 4096, 32, True, "bf16"),
    (8, 129, 11008, 128, False, "fp16"),
    (9, 31, 992, 32, True, "fp16"),
    (16, 300, 2080, 64, True, "bf16"),
    (17, 48, 4096, 128, True, "fp16"),
    (37, 150, 768, 128, False, "bf16"),
    (130, 65, 512, 32, True, "fp16"),
]


@pytest.mark.parametrize("N,M,K,group,zeros,scales", CASES)
def test_matvec_g4(N, M, K, group, zeros, scales):
    import torch
    rng = np.random.default_rng(N + M + K)
    W, s, z = g4_weights(rng, M, K, group, zeros)
    Xq = q8_rows(rng, N, K)
    Wd, sd, sr, zd = _dev_weights(W, s, z, scales)
    Y = torch.full((N * M + 64,), 7.5, device="cuda")
    out = kq.kq_matvec_g4(Wd, sd, to_dev(Xq, torch), M, K, group, zeros=zd, Y=Y[:N * M].view(N, M))
    assert bool((Y[N * M:] == 7.5).all())        # nothing past the output
    ref, B = deo.g4_matmul(W, sr, z, group, Xq)
    assert_g4(out.cpu().numpy(), ref, B, K, f"{N}x{M}x{K}")
    again = kq.kq_matvec_g4(Wd, sd, to_dev(Xq, torch), M, K, group, zeros=zd)
    assert torch.equal(out, again)
    assert kq.kq_get_device_error() == 0


def test_zero_points_beyond_four_bits():
    import torch
    rng = np.random.default_rng(1)
    W, s, _ = g4_weights(rng, 90, 512, 64, False)
    z = rng.integers(0, 256, s.shape, dtype=np.uint8)
    for N in (1, 6, 12):
        Xq = q8_rows(rng, N, 512)
        Xq[0, 0, 4:] = 0x80                      # codes of -128
        Wd, sd, sr, zd = _dev_weights(W, s, z, "fp16")
        got = kq.kq_matvec_g4(Wd, sd, to_dev(Xq, torch), 90, 512, 64, zeros=zd)
        ref, B = deo.g4_matmul(W, sr, z, 64, Xq)
        assert_g4(got.cpu().numpy(), ref, B, 512, "wide zero points")


def test_each_code_and_position():
    """One-hot activations read back every weight exactly: s (c - z) of each k."""
    import torch
    K, M = 256, 16
    rng = np.random.default_rng(2)
    W, s, z = g4_weights(rng, M, K, 64, True)
    Wd, sd, sr, zd = _dev_weights(W, s, z, "fp16")
    Xq = np.zeros((K, K // 32, 36), np.uint8)
    one = np.float16(1.0).view(np.uint16)
    for k in range(K):
        Xq[k, k // 32, 0:2] = np.array([one]).view(np.uint8)
        Xq[k, k // 32, 4 + k % 32] = 1
    want = (sr[:, np.arange(K) // 64] * (deo.g4_codes(W) - z.astype(int)[:, np.arange(K) // 64])).T
    for n in (1, 5, 8, 16, K):
        got = torch.cat([kq.kq_matvec_g4(Wd, sd, to_dev(Xq[i:i + n], torch), M, K, 64, zeros=zd) for i in range(0, K, n)])
        assert np.array_equal(got.cpu().double().numpy(), want), n


# Many weight rows: 32 activation rows to a CTA (which fill the GPU), two rows on the tensor cores;
# and a split K whose clusters of eight need every second SM.
@pytest.mark.parametrize("N,M,K,group,zeros,scales", [
    (33, 45_000, 96, 32, True, "bf16"),
    (64, 44_001, 160, 64, False, "fp16"),
    (40, 44_001, 160, 128, True, "fp16"),
    (70, 30_001, 352, 256, False, "bf16"),
    (2, 70_001, 96, 32, True, "fp16"),
    (2, 61_000, 128, 128, False, "bf16"),
    (5, 2_001, 2048, 128, False, "fp16"),
    (16, 2_048, 2080, 32, True, "bf16"),
    (1, 40, 59_072, 64, True, "bf16"),       # an activation row too long for the weight stream
    (2, 33, 29_600, 128, False, "fp16"),
])
def test_many_weight_rows(N, M, K, group, zeros, scales):
    test_matvec_g4(N, M, K, group, zeros, scales)


@pytest.mark.parametrize("group", [32, 64, 128, 1 << 20])
@pytest.mark.parametrize("zeros", [False, True])
def test_integers_are_exact(group, zeros):
    """Unit scales: every output is a sum of integers below 2^24, and is exact."""
    import torch
    rng = np.random.default_rng(group % 97 + zeros)
    M, K = 70, 416
    W, s, z = g4_weights(rng, M, K, group, zeros)
    W[0], W[1] = 0xff, 0x00
    if zeros:
        z[0], z[1] = 0, 255
    Wd, sd, sr, zd = _dev_weights(W, np.ones_like(s), z, "bf16")
    for N in (1, 2, 3, 8, 9, 16, 33):
        Xq = q8_rows(rng, N, K)
        Xq[..., 0:2] = np.array([np.float16(1.0)]).view(np.uint8)
        Xq[0, :, 4:] = 0x80
        got = kq.kq_matvec_g4(Wd, sd, to_dev(Xq, torch), M, K, group, zeros=zd).cpu().double().numpy()
        ref, _ = deo.g4_matmul(W, sr, z, group, Xq)
        assert np.array_equal(got, ref), N


@pytest.mark.parametrize("N", [1, 9])
def test_offsets_beyond_32_bits(N):
    """A matrix of 5.2 GB (its last rows' offsets are past 2^32 bytes)."""
    import torch
    M, K, group = 320_000, 32_768, 256
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    W = torch.randint(0, 256, (M, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s = (0.02 * torch.rand(M, K // group, generator=gen, device="cuda") + 0.01).half()
    z = torch.randint(0, 16, (M, K // group), generator=gen, device="cuda", dtype=torch.uint8)
    Xq = q8_rows(np.random.default_rng(N), N, K)
    Y = kq.kq_matvec_g4(W, s, to_dev(Xq, torch), M, K, group, zeros=z).cpu().numpy()
    rows = [0, 1, 131_071, 262_143, 262_144, M - 130, M - 2, M - 1]
    ref, B = deo.g4_matmul(W[rows].cpu().numpy(), s[rows].cpu().double().numpy(), z[rows].cpu().numpy(), group, Xq)
    assert_g4(Y[:, rows], ref, B, K, "5.2 GB")


def test_more_activation_rows_than_one_launch_takes():
    import torch
    N, M, K = 65535 * 32 + 70, 3, 32
    rng = np.random.default_rng(5)
    W, s, z = g4_weights(rng, M, K, 32, True)
    Wd, sd, sr, zd = _dev_weights(W, s, z, "fp16")
    Xq = torch.from_numpy(q8_rows(rng, 4096, K)).cuda().repeat(N // 4096 + 1, 1, 1)[:N].contiguous()
    Y = kq.kq_matvec_g4(Wd, sd, Xq, M, K, 32, zeros=zd)
    at = torch.tensor([0, 31, 4095, 65535 * 32 - 1, 65535 * 32, N - 1], device="cuda")
    ref, B = deo.g4_matmul(W, sr, z, 32, Xq[at].cpu().numpy())
    assert_g4(Y[at].cpu().numpy(), ref, B, K, "many rows")
    assert torch.equal(Y[4096:8192], Y[:4096])


def test_non_finite_scales_reach_the_output():
    import torch
    rng = np.random.default_rng(6)
    for N in (1, 9):
        W, s, z = g4_weights(rng, 20, 256, 64, True)
        s[3, 1] = np.inf
        Xq = q8_rows(rng, N, 256)
        Xq[0, 2, 0:2] = np.array([np.float16(np.nan)]).view(np.uint8)
        Wd, sd, sr, zd = _dev_weights(W, s, z, "fp16")
        got = kq.kq_matvec_g4(Wd, sd, to_dev(Xq, torch), 20, 256, 64, zeros=zd).cpu().numpy()
        assert np.all(np.isnan(got[0]))
        if N > 1:
            assert not np.isfinite(got[1:, 3]).any()
            assert np.isfinite(np.delete(got[1:], 3, 1)).all()


MOE = [
    # T, E, top_k, M, K, group, zeros, scales, per_slot
    (1, 8, 2, 96, 256, 32, True, "fp16", False),
    (1, 128, 8, 1536, 2048, 128, False, "fp16", False),
    (1, 16, 8, 2048, 768, 64, True, "bf16", True),
    (3, 4, 4, 50, 544, 128, True, "fp16", True),
    (16, 32, 4, 130, 1024, 32, True, "bf16", False),
    (40, 3, 2, 100, 768, 128, False, "bf16", True),     # many rows to every expert
    (64, 96, 8, 64, 512, 64, True, "fp16", True),
    (9, 1, 1, 33, 64, 32, True, "fp16", False),
    (200, 6, 3, 40, 288, 32, True, "fp16", False),
    (700, 512, 8, 17, 64, 64, False, "fp16", False),
    (600, 1, 1, 33, 96, 32, True, "bf16", False),       # more rows to one expert than are collected at once
    (1100, 3, 1, 20, 128, 64, False, "fp16", True),
]


@pytest.mark.parametrize("T,E,top_k,M,K,group,zeros,scales,per_slot", MOE)
def test_moe_matvec_g4(T, E, top_k, M, K, group, zeros, scales, per_slot):
    import torch
    rng = np.random.default_rng(T + E + M)
    W, s, z = g4_weights(rng, E * M, K, group, zeros)
    Xq = q8_rows(rng, T * top_k if per_slot else T, K)
    ids = np.argsort(rng.standard_normal((T, E)), 1)[:, :top_k].astype(np.int32)
    Wd, sd, sr, zd = _dev_weights(W, s, z, scales)
    Y = torch.full((T * top_k * M + 64,), 7.5, device="cuda")
    got = kq.kq_moe_matvec_g4(Wd, sd, E, to_dev(ids, torch), to_dev(Xq, torch), M, K, group, zeros=zd,
                              Y=Y[:T * top_k * M].view(T, top_k, M))
    assert bool((Y[T * top_k * M:] == 7.5).all())
    ref, B = deo.moe_g4(W, sr, z, group, E, ids, Xq, M)
    assert_g4(got.cpu().numpy(), ref, B, K, f"T={T} E={E}")
    again = kq.kq_moe_matvec_g4(Wd, sd, E, to_dev(ids, torch), to_dev(Xq, torch), M, K, group, zeros=zd)
    assert torch.equal(got, again)
    assert kq.kq_get_device_error() == 0


@pytest.mark.parametrize("T,E,top_k,M,K,group,zeros,scales,per_slot", [
    (10, 128, 8, 130, 768, 32, True, "bf16", True),
    (14, 32, 2, 70, 2048, 128, False, "fp16", False),
    (13, 40, 3, 129, 416, 64, True, "fp16", False),
    (15, 128, 8, 130, 768, 32, True, "bf16", True),
    (30, 256, 8, 40, 768, 64, True, "fp16", True),      # more pairs than a round of CTAs divides by
    (1, 6, 4, 40, 59_072, 128, True, "fp16", False),
    (2, 8, 3, 70, 1056, 32, True, "bf16", True),
    (6, 8, 2, 257, 768, 128, False, "fp16", False),
])
def test_about_one_row_per_expert(T, E, top_k, M, K, group, zeros, scales, per_slot):
    """Experts without rows beside experts with one or two; rows too long for the weight stream."""
    test_moe_matvec_g4(T, E, top_k, M, K, group, zeros, scales, per_slot)


def test_invalid_ids_where_few_experts_have_rows():
    import torch
    T, E, top_k, M, K = 12, 40, 3, 150, 352
    rng = np.random.default_rng(5)
    W, s, z = g4_weights(rng, E * M, K, 32, True)
    Xq = q8_rows(rng, T, K)
    ids = rng.integers(1, E, (T, top_k)).astype(np.int32)    # expert 0, which writes the zeros, has no rows
    Wd, sd, sr, zd = _dev_weights(W, s, z, "bf16")
    ref, B = deo.moe_g4(W, sr, z, 32, E, ids, Xq, M)
    bad = ids.copy()
    bad[0, 1], bad[5, 0], bad[11, 2] = -1, E, 2_000_000_000
    kq.kq_get_device_error()
    got = kq.kq_moe_matvec_g4(Wd, sd, E, to_dev(bad, torch), to_dev(Xq, torch), M, K, 32, zeros=zd).cpu().numpy()
    assert kq.kq_get_device_error() == kq.KQ_DEVERR_EXPERT_ID
    for t, j in ((0, 1), (5, 0), (11, 2)):
        assert not got[t, j].any()
        got[t, j] = ref[t, j]
    assert_g4(got, ref, B, K, "invalid ids")


@pytest.mark.parametrize("group,zeros,scales", [(32, True, "bf16"), (64, False, "fp16"), (128, True, "fp16"), (128, False, "bf16")])
def test_many_rows_per_expert(group, zeros, scales):
    """Some 40 rows to an expert, 32 at a time."""
    test_moe_matvec_g4(161, 8, 2, 8_400, 160, group, zeros, scales, False)


@pytest.mark.parametrize("T", [1, 30])
def test_repeated_and_invalid_expert_ids(T):
    import torch
    E, top_k, M, K = 5, 3, 70, 320
    rng = np.random.default_rng(T)
    W, s, z = g4_weights(rng, E * M, K, 64, True)
    Xq = q8_rows(rng, T, K)
    ids = rng.integers(0, E, (T, top_k)).astype(np.int32)    # repeats within a token
    ids[0] = [4, 4, 4]
    Wd, sd, sr, zd = _dev_weights(W, s, z, "fp16")
    call = lambda i: kq.kq_moe_matvec_g4(Wd, sd, E, to_dev(i, torch), to_dev(Xq, torch), M, K, 64, zeros=zd).cpu().numpy()  # noqa: E731
    ref, B = deo.moe_g4(W, sr, z, 64, E, ids, Xq, M)
    kq.kq_get_device_error()
    assert_g4(call(ids), ref, B, K, "repeats")
    assert kq.kq_get_device_error() == kq.KQ_DEVERR_NONE
    bad = ids.copy()
    bad[0, 1], bad[T - 1, 2] = -1, E
    got = call(bad)
    assert kq.kq_get_device_error() == kq.KQ_DEVERR_EXPERT_ID
    ok = bad == ids
    assert np.all(got[~ok] == 0)
    assert_g4(got[ok], ref[ok], B[ok], K, "valid slots")


def test_on_another_stream_and_in_a_graph():
    import torch
    rng = np.random.default_rng(11)
    M, K, N = 512, 1024, 3
    W, s, z = g4_weights(rng, M, K, 128, True)
    Wd, sd, _, zd = _dev_weights(W, s, z, "bf16")
    xq = to_dev(q8_rows(rng, N, K), torch)
    want = kq.kq_matvec_g4(Wd, sd, xq, M, K, 128, zeros=zd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kq.kq_matvec_g4(Wd, sd, xq, M, K, 128, zeros=zd, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    Y = torch.zeros(N, M, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kq.kq_matvec_g4(Wd, sd, xq, M, K, 128, zeros=zd, Y=Y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)
