"""kq_moe_route's group limits where the sum of a group's two largest keys passes fp32's range.
Against the fp64 definition."""
import numpy as np
import pytest

from oracle import decode_oracle as deo
import quantized_weight_matmul_q4_gb300 as kq

pytestmark = pytest.mark.gpu


def _check(L, top_k, bias, **kw):
    import torch
    L, b = np.asarray(L, np.float32), np.asarray(bias, np.float32)
    ids, probs = kq.kq_moe_route(torch.from_numpy(L).cuda(), top_k, bias=torch.from_numpy(b).cuda(), **kw)
    want_ids, want = deo.route(L, top_k, bias=b, **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    # Logits within 60 of one another: the router's bound for ordinary rows.
    assert np.all(np.abs(probs.cpu().double().numpy() - want) <= 120 * 2.0 ** -24 * want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("sign", [1, -1])
def test_group_scores_beyond_fp32(score, sign):
    rng = np.random.default_rng(3)
    E, n_groups = 40, 8
    L = rng.standard_normal((4, E))
    bias = np.float64(sign) * (2e38 + 1.3e38 * rng.random(E))
    _check(L, 5, bias, score=score, n_groups=n_groups, topk_groups=3, group_top=2)
    bias[10:15] = 0.1 * rng.standard_normal(5)         # one group of ordinary biases
    _check(L, 5, bias, score=score, n_groups=n_groups, topk_groups=3, group_top=2)
    _check(L, 5, bias, score=score, n_groups=n_groups, topk_groups=3, group_top=1)
