"""kq_moe_route's weights over the whole range of logits: chosen experts far below the
token's largest score, and scores below fp32's range. Against the fp64 definition."""
import numpy as np
import pytest

from oracle import decode_oracle as deo
import quantized_weight_matmul_q4_gb300 as kq

pytestmark = pytest.mark.gpu

# For chosen logits within 60 of the largest chosen one: the rounding of their distance
# (60 * 2^-24), expf, the sum and the quotient, as for ordinary rows.
REL = 120 * 2.0 ** -24


def _check(L, top_k, bias=None, dtype="fp32", **kw):
    import torch
    t = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    x = torch.from_numpy(np.asarray(L, np.float32)).cuda().to(t)
    b = None if bias is None else np.asarray(bias, np.float32)
    ids, probs = kq.kq_moe_route(x, top_k, bias=None if b is None else torch.from_numpy(b).cuda(), **kw)
    want_ids, want = deo.route(x.cpu().double().numpy(), top_k, bias=b, **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    p = probs.cpu().double().numpy()
    assert np.all(np.abs(p - want) <= REL * np.abs(want) + 1e-37), (p[0], want[0])
    return p


@pytest.mark.parametrize("E", [24, 200])
@pytest.mark.parametrize("top_k", [1, 4])
@pytest.mark.parametrize("below", [60, 88, 92, 95, 103, 104, 150, 600])
def test_softmax_weights_below_an_expert_out_of_service(E, top_k, below):
    """A bias of -inf keeps the dominant expert out; it keeps its share of the softmax sum."""
    rng = np.random.default_rng(below)
    L = 1.5 * rng.standard_normal((5, E))
    L[:, 7] = below
    L[1, 8:] = -np.inf                     # seven experts left
    L[2, [0, 1, 2] + list(range(8, E))] = -np.inf
    L[3, :6] = -np.inf
    L[3, 9:] = -np.inf                     # two: fewer than four slots
    bias = np.zeros(E)
    bias[7] = -np.inf
    p = _check(L, top_k, bias=bias, scale=2.5)
    assert np.all(np.isfinite(p)) and np.allclose(p.sum(1), 2.5, rtol=1e-5)
    p = _check(L, top_k, bias=bias, n_groups=4, topk_groups=2)
    assert np.all(np.isfinite(p))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("at", [-60.0, -87.0, -88.5, -89.0, -95.0, -104.0, -120.0, -500.0])
def test_sigmoid_weights_of_very_negative_logits(dtype, biased, at):
    rng = np.random.default_rng(int(-at))
    E = 96
    L = at + 1.5 * rng.standard_normal((6, E))
    L[1] = at                              # equal: weights of 1 / top_k
    L[2, :40] = -np.inf
    L[3, 5] = at + 30
    L[4, 5] = 3.0                          # one ordinary expert among them
    L[5, 5:] = -np.inf                     # fewer experts than slots
    bias = 1e-3 * np.round(20 * rng.standard_normal(E)) if biased else None
    p = _check(L, 6, bias=bias, dtype=dtype, score="sigmoid", scale=2.5)
    assert np.allclose(p.sum(1), 2.5, rtol=1e-5)
    if not biased:
        assert np.allclose(p[1], 2.5 / 6, rtol=1e-6)
    _check(L, 6, bias=bias, dtype=dtype, score="sigmoid", n_groups=8, topk_groups=3)


def test_scores_below_fp64s_range_are_zero():
    L = np.full((3, 32), -2000.0)
    L[1, 3] = -700.0
    L[2] = -1e38
    p = _check(L, 4, score="sigmoid")
    assert np.all(p[[0, 2]] == 0) and p[1, 0] == 1
    L = np.zeros((1, 32))
    L[0, 9] = 2000.0
    bias = np.zeros(32)
    bias[9] = -np.inf
    assert np.all(_check(L, 4, bias=bias) == 0)


def test_more_slots_than_lanes():
    rng = np.random.default_rng(1)
    L = -100 + 5 * rng.standard_normal((3, 120))
    p = _check(L, 50, score="sigmoid", scale=2.0)
    assert np.allclose(p.sum(1), 2.0, rtol=1e-5)
    L[:, 4] = 0.0
    bias = np.zeros(120)
    bias[4] = -np.inf
    p = _check(L, 50, bias=bias)
    assert np.allclose(p.sum(1), 1.0, rtol=1e-5)
