"""kq_add_rmsnorm_q8_1 on rows whose squares pass fp32's range and on rows whose squares fall
below it. Against the fp64 definition."""
import numpy as np
import pytest

from oracle import decode_oracle as deo
import quantized_weight_matmul_q4_gb300 as kq
from _decodeutil import HALF, U32, assert_q8_blocks

pytestmark = pytest.mark.gpu

NORM_REL = 64 * U32      # of y before it is rounded, as in the norm's other tests


def _dtype(name):
    import torch
    return {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}[name]


def _check(X, R, gamma, eps, dtype, what):
    import torch
    H, Y, Xq = kq.kq_add_rmsnorm_q8_1(X, R, gamma, eps, Y=True)
    if R is not None:
        assert torch.equal(H, (X.float() + R.float()).to(X.dtype))
    f64 = lambda t: None if t is None else t.detach().cpu().double().numpy()  # noqa: E731
    _, y = deo.add_rmsnorm(f64(X), f64(R), f64(gamma), eps)
    # Rounding y to its type: half a step, and no less than half the type's smallest step.
    least = {"fp32": 2.0 ** -150, "fp16": 2.0 ** -25, "bf16": 2.0 ** -134}[dtype]
    err = np.abs(f64(Y) - y)
    assert np.all(err <= np.abs(y) * (NORM_REL + HALF[dtype] * 1.01) + 1.01 * least), what
    assert_q8_blocks(Xq.cpu().numpy(), y, NORM_REL, what)
    return y


# (rows that are held in registers by one, two and four runs a thread, an odd stride, and a row
# that is read twice)
SHAPES = [(3, 4096, 0), (1700, 1120, 0), (3, 1120, 1), (2, 16384, 0), (2, 33024, 0), (2, 33024, 1)]


@pytest.mark.parametrize("N,K,pad", SHAPES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", [3e17, 1e19, 3e19, 1e30, 5e37])
def test_rows_whose_squares_pass_the_range(N, K, pad, dtype, size):
    import torch
    rng = np.random.default_rng(K + pad)
    a = torch.from_numpy((size * np.clip(rng.standard_normal((N, K + pad)), -3, 3)).astype(np.float32)).cuda().to(_dtype(dtype))
    X = a[:, :K]
    gamma = torch.from_numpy((1 + 0.3 * rng.standard_normal(K)).astype(np.float32)).cuda()
    y = _check(X, None, gamma, 1e-5, dtype, f"{dtype} {N}x{K}+{pad} of {size}")
    assert 0.5 < np.sqrt(np.mean(y * y)) < 2
    _check(X, X.flip(0), gamma, 1e-5, dtype, f"{dtype} {N}x{K}+{pad} of {size}, residual")


@pytest.mark.parametrize("N,K,pad", SHAPES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size,eps", [(1e-19, 0.0), (1e-21, 0.0), (1e-24, 0.0), (1e-36, 0.0), (1e-39, 0.0), (1e-20, 1e-40),
                                      (1e-19, 1e-38), (1e-24, 1e-5)])
def test_rows_whose_squares_fall_below_the_range(N, K, pad, dtype, size, eps):
    import torch
    rng = np.random.default_rng(K + pad)
    a = torch.from_numpy((size * rng.standard_normal((N, K + pad))).astype(np.float32)).cuda().to(_dtype(dtype))
    gamma = torch.ones(K, device="cuda")
    eps = float(np.float32(eps))             # what the C call takes
    _check(a[:, :K], None, gamma, eps, dtype, f"{dtype} {N}x{K}+{pad} of {size}, eps {eps}")


def test_one_huge_value_in_an_ordinary_row():
    import torch
    rng = np.random.default_rng(1)
    for K in (4096, 33024):
        X = torch.from_numpy(rng.standard_normal((4, K)).astype(np.float32)).cuda()
        X[0, 5] = 1e25
        X[1, K - 1] = -3e38
        X[2, 77] = 2e19
        y = _check(X, None, torch.ones(K, device="cuda"), 1e-5, "fp32", f"{K}")
        assert abs(y[0, 5] - np.sqrt(K)) < 1e-3


def test_rows_of_zeros():
    import torch
    for K in (256, 33024):
        X = torch.zeros(2, K, device="cuda")
        gamma = torch.ones(K, device="cuda")
        for eps in (1e-5, 1e-40):
            _, Y, Xq = kq.kq_add_rmsnorm_q8_1(X, None, gamma, eps, Y=True)
            assert bool((Y == 0).all()) and bool((Xq == 0).all())
        _, Y, Xq = kq.kq_add_rmsnorm_q8_1(X, None, gamma, 0.0, Y=True)
        assert bool(torch.isnan(Y).all())                                # 0 / 0
        assert np.all(np.isnan(deo.unpack_q8_1(Xq.cpu().numpy())[0]))
