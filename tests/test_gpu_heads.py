"""kq_qk_norm_rope on the GPU against its fp64 definition."""
import numpy as np
import pytest

import quantized_weight_matmul_q4_gb300 as kq
from _attnutil import HALF, U32, f64, heads, table, torch_dtype
from oracle import attn_oracle as ao

pytestmark = pytest.mark.gpu


def _check(got, x, gamma, eps, cs, pairing, out, what):
    # A sum of at most 256 squares by 8 and then 5 additions, halved by the root; the root, two
    # divisions, two products, and the rotation's product and sum: below 16 half steps. Then one rounding.
    y, B = ao.norm_rope(x, gamma, eps, cs, pairing)
    tol = 16 * U32 * B + HALF[out] * (np.abs(y) + 16 * U32 * B) + (2.0 ** -25 if out == "fp16" else 1e-38)
    err = np.abs(got - y)
    assert np.all(err <= tol), f"{what}: {np.nanmax(err / tol)}"


def _dev(a):
    import torch
    return torch.from_numpy(a).cuda()


@pytest.mark.parametrize("pairing", ["half", "pairs"])
@pytest.mark.parametrize("dtype,out", [("fp32", "fp32"), ("fp32", "bf16"), ("fp32", "fp16"), ("fp16", "fp16"), ("bf16", "bf16")])
@pytest.mark.parametrize("N,Hq,Hk,D,rot,pad,norm", [
    (1, 32, 8, 128, 128, 0, True), (3, 4, 1, 64, 32, 8, False), (7, 5, 0, 80, 80, 1, True), (2, 3, 3, 256, 128, 0, True),
    (5, 1, 1, 16, 16, 0, True), (4, 7, 1, 96, 48, 3, False), (9, 2, 1, 240, 240, 0, True), (3000, 5, 2, 128, 64, 0, True)])
def test_norm_rope(dtype, out, pairing, N, Hq, Hk, D, rot, pad, norm):
    rng = np.random.default_rng(N + D + rot)
    Q, K = heads(rng, N, Hq, D, dtype, pad), heads(rng, N, Hk, D, dtype, 2 * pad) if Hk else None
    cs, pos = table(500, rot), rng.integers(0, 500, N).astype(np.int32)
    gq, gk = ((1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if norm else None for _ in range(2))
    Qo, Ko = kq.kq_qk_norm_rope(Q, K, _dev(cs), _dev(pos), q_gamma=_dev(gq) if norm else None,
                                k_gamma=_dev(gk) if norm and Hk else None, eps=1e-6, pairing=pairing,
                                out_dtype=torch_dtype(out))
    assert Qo.dtype == torch_dtype(out) and (Ko is None) == (Hk == 0)
    _check(f64(Qo), f64(Q), gq, 1e-6, cs[pos], pairing, out, "queries")
    if Hk:
        _check(f64(Ko), f64(K), gk, 1e-6, cs[pos], pairing, out, "keys")
    assert kq.kq_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_in_place_inside_packed_rows(dtype):
    """Queries and keys of packed query, key and value rows, turned where they are."""
    import torch
    rng = np.random.default_rng(4)
    rows = heads(rng, 33, 12, 128, dtype)
    before = rows.clone()
    cs, pos, g = table(64, 128), np.arange(33, dtype=np.int32), np.ones(128, np.float32)
    want = kq.kq_qk_norm_rope(rows[:, :8], rows[:, 8:10], _dev(cs), _dev(pos), q_gamma=_dev(g), k_gamma=_dev(g))
    got = kq.kq_qk_norm_rope(rows[:, :8], rows[:, 8:10], _dev(cs), _dev(pos), q_gamma=_dev(g), k_gamma=_dev(g),
                             Qo=rows[:, :8], Ko=rows[:, 8:10])
    assert got[0].data_ptr() == rows.data_ptr()
    assert torch.equal(rows[:, :8], want[0]) and torch.equal(rows[:, 8:10], want[1])
    assert torch.equal(rows[:, 10:], before[:, 10:])


def test_norm_alone_rotation_alone_and_positions_by_row():
    import torch
    rng = np.random.default_rng(6)
    Q = heads(rng, 5, 3, 64, "fp32")
    g = (1 + 0.3 * rng.standard_normal(64)).astype(np.float32)
    y, none = kq.kq_qk_norm_rope(Q, None, q_gamma=_dev(g), eps=1e-5)
    assert none is None
    _check(f64(y), f64(Q), g, 1e-5, None, "half", "fp32", "norm alone")
    cs = table(5, 64)
    y, _ = kq.kq_qk_norm_rope(Q, None, _dev(cs))
    _check(f64(y), f64(Q), None, 0, cs, "half", "fp32", "rotation alone")
    assert torch.equal(kq.kq_qk_norm_rope(Q, None)[0], Q)
    one = Q[:1].expand(5, 3, 64)                      # one row read for all
    y, _ = kq.kq_qk_norm_rope(one, None, _dev(cs))
    _check(f64(y), f64(one), None, 0, cs, "half", "fp32", "one row")


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e18, 1e25, 3e38])
def test_heads_of_any_finite_size(scale):
    """Squares that leave fp32's range, beside heads of ordinary size in the same call."""
    import torch
    rng = np.random.default_rng(7)
    x = rng.uniform(-1, 1, (6, 4, 128)) * np.where(np.arange(6) % 2, 1.0, scale)[:, None, None]
    Q = _dev(x.astype(np.float32))
    y, _ = kq.kq_qk_norm_rope(Q, None, q_gamma=torch.ones(128, device="cuda"), eps=0.0)
    _check(f64(y), f64(Q), np.ones(128), 0.0, None, "half", "fp32", "sizes")


def test_infinities_and_nan_stay_in_their_heads():
    import torch
    rng = np.random.default_rng(8)
    Q = heads(rng, 4, 3, 128, "bf16").clone()
    Q[1, 1, 5], Q[2, 0, 127] = float("nan"), float("inf")
    g, cs = torch.ones(128, device="cuda"), _dev(table(4, 128))
    y, _ = kq.kq_qk_norm_rope(Q, None, cs, q_gamma=g)
    bad = ~torch.isfinite(y).all(-1)
    assert bad[1, 1] and bad[2, 0] and int(bad.sum()) == 2


def test_rows_without_a_position_are_left_as_they_were():
    import torch
    rng = np.random.default_rng(9)
    Q, K = heads(rng, 6, 2, 64, "fp16"), heads(rng, 6, 1, 64, "fp16")
    cs = _dev(table(10, 64))
    pos = torch.tensor([3, -1, 9, 10, -(1 << 31), 0], dtype=torch.int32, device="cuda")
    Qo, Ko = torch.full_like(Q.contiguous(), 7), torch.full_like(K.contiguous(), 7)
    kq.kq_qk_norm_rope(Q, K, cs, pos, Qo=Qo, Ko=Ko)
    assert kq.kq_get_device_error() == kq.KQ_DEVERR_POSITION        # 10 is not in the table
    assert kq.kq_get_device_error() == 0
    for n, there in enumerate([1, 0, 1, 0, 0, 1]):
        assert bool((Qo[n] == 7).all()) != bool(there) and bool((Ko[n] == 7).all()) != bool(there)
    want, _ = kq.kq_qk_norm_rope(Q, None, cs, torch.clamp(pos, 0, 9))
    assert torch.equal(Qo[[0, 2, 5]], want[[0, 2, 5]])


def test_another_stream():
    import torch
    rng = np.random.default_rng(10)
    Q, cs = heads(rng, 50, 4, 128, "fp32"), _dev(table(50, 128))
    want, _ = kq.kq_qk_norm_rope(Q, None, cs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, _ = kq.kq_qk_norm_rope(Q, None, cs, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
