"""kq_moe_route on the GPU against its fp64 definition: the same experts in the
same order, ties to the lowest index, and weights within fp32's error."""
import numpy as np
import pytest

from oracle import decode_oracle as deo
import quantized_weight_matmul_q4_gb300 as kq

pytestmark = pytest.mark.gpu

# Relative error of a weight for logits within 60 of the largest: the rounding of
# l - max (60 * 2^-24), expf, a sum of up to 512 terms in 21 steps, the top-k sum
# and five single operations: under 120 * 2^-24.
REL = 120 * 2.0 ** -24


def _check(logits, top_k, dtype="fp32", **kw):
    import torch
    t = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
    x = logits if isinstance(logits, torch.Tensor) else torch.from_numpy(np.asarray(logits, np.float32)).cuda().to(t)
    dev = dict(kw)
    if kw.get("bias") is not None:
        dev["bias"] = torch.from_numpy(np.asarray(kw["bias"], np.float32)).cuda()
    ids, probs = kq.kq_moe_route(x, top_k, **dev)
    want_ids, want = deo.route(x.cpu().double().numpy(), top_k, **kw)
    got = ids.cpu().numpy()
    assert np.array_equal(got, want_ids), np.argwhere(got != want_ids)[:3]
    p = probs.cpu().double().numpy()
    assert np.all(np.abs(p - want) <= REL * np.abs(want) + 1e-37)
    return got, p


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,top_k", [(1, 128, 8), (5, 1, 1), (33, 7, 7), (130, 60, 4), (9, 160, 6), (70, 512, 10),
                                       (3, 512, 512), (2, 33, 32)])
def test_random(dtype, score, biased, T, E, top_k):
    rng = np.random.default_rng(T + E)
    bias = 1e-3 * np.round(20 * rng.standard_normal(E)) if biased else None
    _check(1.5 * rng.standard_normal((T, E)), top_k, dtype, score=score, bias=bias, renormalise=T % 2 == 1, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("E,n_groups,topk_groups,top_k", [(96, 4, 2, 4), (384, 12, 4, 6), (64, 64, 5, 5), (40, 8, 1, 3),
                                                          (512, 16, 15, 12), (6, 3, 2, 4), (48, 2, 2, 5)])
def test_groups(score, biased, group_top, E, n_groups, topk_groups, top_k):
    rng = np.random.default_rng(E + n_groups)
    bias = 0.05 * rng.standard_normal(E) if biased else None
    _check(1.5 * rng.standard_normal((57, E)), top_k, score=score, bias=bias, n_groups=n_groups, topk_groups=topk_groups,
           group_top=group_top)


def test_ties_go_to_the_lowest_index():
    L = np.zeros((4, 64))
    L[1] = np.arange(64) % 3
    L[2, 10:20] = 5.0
    L[3] = -0.0
    L[3, ::2] = 0.0
    for kw in ({}, {"bias": np.zeros(64)}, {"score": "sigmoid", "bias": np.repeat([0.25, 0.0], 32)},
               {"n_groups": 8, "topk_groups": 3}, {"n_groups": 8, "topk_groups": 3, "bias": np.zeros(64)}):
        _check(L, 12, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_keys_closer_than_fp32_tells_apart(score):
    """Biases that bring the keys of many experts within 1e-8 of one another: fp32 keys
    tie or turn around there, and the order has to be that of 64 bits."""
    rng = np.random.default_rng(3)
    E = 128
    l = (1.5 * rng.standard_normal(E)).astype(np.float32)
    _, s = deo.route(l[None], E, score=score, renormalise=False)
    ids, _ = deo.route(l[None], E, score=score, renormalise=False)
    sc = np.empty(E)
    sc[ids[0]] = s[0]
    bias = (0.7 - sc).astype(np.float32)               # keys 0.7 up to the bias's rounding (3e-8)
    key = sc + bias.astype(np.float64)
    assert np.unique(key).size == E and np.ptp(key) < 1.2e-7
    assert np.unique((sc.astype(np.float32) + bias)).size < 16    # what fp32 would see
    L = np.tile(l, (40, 1))
    _check(L, 16, score=score, bias=bias)
    _check(L, 8, score=score, bias=bias, n_groups=8, topk_groups=3)


def test_masked_experts_and_rows():
    rng = np.random.default_rng(4)
    L = rng.standard_normal((8, 40))
    L[0] = -np.inf                          # nothing available
    L[1, 3:] = -np.inf                      # fewer than top_k
    L[2] = np.nan
    L[3, 5] = np.nan
    L[4, 7] = np.inf
    L[5] = np.finfo(np.float32).min         # the type's lowest value is an ordinary logit
    L[6, ::2] = -np.inf
    L[7, 39] = np.finfo(np.float32).min
    bias = 0.1 * rng.standard_normal(40)
    bias[1] = -np.inf
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for kw in ({}, {"n_groups": 8, "topk_groups": 2}, {"n_groups": 8, "topk_groups": 2, "group_top": 1}):
                ids, p = _check(L, 6, score=score, bias=b, **kw)
                assert np.all(np.sort(ids, 1)[:, 1:] != np.sort(ids, 1)[:, :-1])    # distinct
                assert np.all(p[0] == 0) and np.all(np.isfinite(p))


def test_infinite_bias_forces_an_expert():
    rng = np.random.default_rng(5)
    bias = np.zeros(32)
    bias[[9, 4]] = np.inf
    ids, _ = _check(rng.standard_normal((6, 32)), 4, bias=bias)
    assert np.all(ids[:, :2] == [4, 9])


def test_strided_and_broadcast_rows():
    import torch
    x = torch.randn(50, 131, device="cuda")
    _check(x[:, 1:130].contiguous()[:, :128], 8)
    _check(x[:1, :128].expand(9, 128), 8)
    _check(x[::2, :127], 5)


def test_deterministic():
    import torch
    x = torch.randn(3000, 256, device="cuda")
    b = 0.01 * torch.randn(256, device="cuda")
    a = kq.kq_moe_route(x, 8, score="sigmoid", bias=b, n_groups=8, topk_groups=4)
    c = kq.kq_moe_route(x, 8, score="sigmoid", bias=b, n_groups=8, topk_groups=4)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
