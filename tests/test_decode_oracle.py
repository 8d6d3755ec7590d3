"""Pins of the decode-step oracle (CPU): hand-computed values and identities."""
import numpy as np
import pytest

from oracle import decode_oracle as deo
from _decodeutil import g4_weights, q8_rows


def test_add_rmsnorm_closed_form():
    h, y = deo.add_rmsnorm([[1.0, 2.0]], [[2.0, 2.0]], [1.0, 10.0], 0.0)
    assert np.allclose(h, [[3, 4]]) and np.allclose(y, [[3 / np.sqrt(12.5), 40 / np.sqrt(12.5)]])


def test_swiglu_closed_form():
    v = deo.swiglu([[0.0, np.log(3.0), -1000.0]], [[5.0, 2.0, 1.0]])
    assert np.allclose(v, [[0.0, 2 * np.log(3.0) * 0.75, 0.0]])


def test_route_by_hand():
    ids, p = deo.route([[0.0, np.log(2.0), np.log(2.0), -np.inf]], 2, renormalise=False)
    assert ids.tolist() == [[1, 2]] and np.allclose(p, [[0.4, 0.4]])
    ids, p = deo.route([[0.0, np.log(2.0), np.log(2.0), -np.inf]], 4, scale=2.0)
    assert ids.tolist() == [[1, 2, 0, 3]] and np.allclose(p, [[0.8, 0.8, 0.4, 0.0]])
    # the bias moves the choice, not the weight
    ids, p = deo.route([[0.0, 0.0, 0.0, 0.0]], 1, bias=[0, 0, 1, 0], renormalise=False)
    assert ids.tolist() == [[2]] and np.allclose(p, [[0.25]])
    # group 1 wins by its best two though group 0 has the best one
    L = [[3.0, 0.0, 2.5, 2.5]]
    assert deo.route(L, 1, score="sigmoid", n_groups=2, topk_groups=1, group_top=2)[0].tolist() == [[2]]
    assert deo.route(L, 1, score="sigmoid", n_groups=2, topk_groups=1, group_top=1)[0].tolist() == [[0]]


def test_route_empty_row():
    ids, p = deo.route(np.full((1, 5), -np.inf), 3)
    assert ids.tolist() == [[0, 1, 2]] and np.all(p == 0)


@pytest.mark.parametrize("zeros", [False, True])
def test_g4_against_dequantised_product(zeros):
    rng = np.random.default_rng(1)
    W, s, z = g4_weights(rng, 6, 160, 64, zeros)
    Xq = q8_rows(rng, 3, 160)
    d, _, q = deo.unpack_q8_1(Xq)
    x = (d[..., None] * q).reshape(3, 160)
    w = np.empty((6, 160))
    for m in range(6):
        for k in range(160):
            c = (int(W[m, k // 2]) >> (4 * (k % 2))) & 15
            w[m, k] = float(s[m, k // 64]) * (c - (8 if z is None else int(z[m, k // 64])))
    Y, B = deo.g4_matmul(W, s, z, 64, Xq)
    assert np.allclose(Y, x @ w.T, rtol=1e-12, atol=1e-12) and np.all(np.abs(Y) <= B * (1 + 1e-12))


def test_moe_is_the_chosen_matrix():
    rng = np.random.default_rng(2)
    W, s, z = g4_weights(rng, 4 * 5, 64, 32, True)
    Xq = q8_rows(rng, 3, 64)
    ids = np.array([[0, 3], [2, 2], [1, 0]])
    Y, _ = deo.moe_g4(W, s, z, 32, 4, ids, Xq, 5)
    for t in range(3):
        for j in range(2):
            r = slice(5 * ids[t, j], 5 * ids[t, j] + 5)
            assert np.allclose(Y[t, j], deo.g4_matmul(W[r], s[r], z[r], 32, Xq[t:t + 1])[0][0])
