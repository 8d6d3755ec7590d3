"""kq_add_rmsnorm_q8_1 and kq_swiglu_q8_1 on the GPU against their fp64 definitions."""
import numpy as np
import pytest

from oracle import decode_oracle as deo
import quantized_weight_matmul_q4_gb300 as kq
from _decodeutil import HALF, U32, assert_q8_blocks

pytestmark = pytest.mark.gpu

# Relative error of y before it is rounded: h (1 rounding), the sum of squares
# (at most 100 roundings of positive terms, halved by the square root) and about
# eight single operations after it.
NORM_REL = 64 * U32
# expf (2 ulp), the sum, the division and the product.
SWIGLU_REL = 10 * U32


def _torch_dtype(name):
    import torch
    return {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}[name]


def _f64(t):
    return t.detach().cpu().double().numpy()


def _rows(rng, N, K, pad, dtype, scale=1.0):
    """[N, K] view with rows K + pad apart."""
    import torch
    a = torch.from_numpy((scale * rng.standard_normal((N, K + pad))).astype(np.float32)).cuda().to(dtype)
    return a[:, :K]


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("N,K,pad", [(1, 32, 0), (1, 4096, 0), (3, 96, 0), (5, 2080, 64), (7, 1120, 1), (2, 11008, 0),
                                     (3, 16384, 8), (2, 33024, 0), (310, 768, 0)])
def test_add_rmsnorm(dtype, N, K, pad):
    import torch
    t = _torch_dtype(dtype)
    rng = np.random.default_rng(N * 7 + K + pad)
    X, R = _rows(rng, N, K, pad, t), _rows(rng, N, K, 2 * pad, t, 3.0)
    gamma = torch.from_numpy((1 + 0.3 * rng.standard_normal(K)).astype(np.float32)).cuda()
    H, Y, Xq = kq.kq_add_rmsnorm_q8_1(X, R, gamma, 1e-5, Y=True)
    assert torch.equal(H, (X.float() + R.float()).to(t))
    _, y = deo.add_rmsnorm(_f64(X), _f64(R), _f64(gamma), 1e-5)
    assert np.all(np.abs(_f64(Y) - y) <= np.abs(y) * (NORM_REL + HALF[dtype] * 1.01) + (2.0 ** -25 if dtype == "fp16" else 0))
    assert_q8_blocks(Xq.cpu().numpy(), y, NORM_REL, f"{dtype} {N}x{K}")
    # Without the residual, and without the optional outputs: the same rows.
    H0, Y0, Xq0 = kq.kq_add_rmsnorm_q8_1(X, None, gamma, 1e-5)
    assert H0 is None and Y0 is None
    _, y0 = deo.add_rmsnorm(_f64(X), None, _f64(gamma), 1e-5)
    assert_q8_blocks(Xq0.cpu().numpy(), y0, NORM_REL, f"{dtype} {N}x{K} no residual")
    _, _, Xq1 = kq.kq_add_rmsnorm_q8_1(X, R, gamma, 1e-5)
    assert torch.equal(Xq1, Xq)


@pytest.mark.parametrize("which", ["X", "R"])
@pytest.mark.parametrize("K", [4096, 40960])
def test_add_rmsnorm_in_place(which, K):
    import torch
    rng = np.random.default_rng(5)
    X, R = _rows(rng, 9, K, 0, torch.bfloat16), _rows(rng, 9, K, 0, torch.bfloat16)
    gamma = torch.ones(K, device="cuda")
    H, Y, Xq = kq.kq_add_rmsnorm_q8_1(X, R, gamma, 1e-6, Y=True)
    X1, R1 = X.clone(), R.clone()
    out = X1 if which == "X" else R1
    H1, Y1, Xq1 = kq.kq_add_rmsnorm_q8_1(X1, R1, gamma, 1e-6, H=out, Y=True)
    assert H1 is out
    assert torch.equal(H1, H) and torch.equal(Y1, Y) and torch.equal(Xq1, Xq)


def test_add_rmsnorm_broadcast_row_and_zero_row():
    import torch
    K = 256
    rng = np.random.default_rng(8)
    X = _rows(rng, 4, K, 0, torch.float32).clone()
    X[2] = 0
    row = _rows(rng, 1, K, 0, torch.float32)
    gamma = torch.ones(K, device="cuda")
    H, _, Xq = kq.kq_add_rmsnorm_q8_1(X, row.expand(4, K), gamma, 1e-5)
    assert torch.equal(H, X + row)
    _, _, Xq2 = kq.kq_add_rmsnorm_q8_1(X, row.expand(4, K).contiguous(), gamma, 1e-5)
    assert torch.equal(Xq, Xq2)
    _, Y, Xz = kq.kq_add_rmsnorm_q8_1(X, None, gamma, 1e-5, Y=True)
    assert bool((Y[2] == 0).all()) and bool((Xz[2] == 0).all())


def test_add_rmsnorm_non_finite_rows_stay_visible():
    import torch
    K = 128
    X = torch.ones(4, K, device="cuda")
    X[1, 40] = float("nan")
    X[2, 3] = float("inf")
    gamma = torch.ones(K, device="cuda")
    gamma[100] = float("nan")
    _, _, Xq = kq.kq_add_rmsnorm_q8_1(X, None, gamma, 1e-5)
    d, _, _ = deo.unpack_q8_1(Xq.cpu().numpy())
    assert np.all(np.isnan(d[1]))                      # the whole row's norm is NaN
    assert np.isnan(d[2, 0])                           # inf * 0
    assert np.isnan(d[0, 3]) and np.all(np.isfinite(d[0, :3]))   # one channel: its block only
    assert np.isnan(d[3, 3]) and np.all(np.isfinite(d[3, :3]))


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("N,K,how", [(1, 32, "two"), (8, 768, "halves"), (5, 160, "halves"), (3, 4096, "two"),
                                     (7, 96, "odd"), (33, 11008, "halves")])
def test_swiglu(dtype, N, K, how):
    t = _torch_dtype(dtype)
    rng = np.random.default_rng(N + K)
    if how == "two":
        g, u = _rows(rng, N, K, 0, t, 3.0), _rows(rng, N, K, 0, t)
    elif how == "halves":
        gu = _rows(rng, N, 2 * K, 0, t, 3.0)
        g, u = gu[:, :K], gu[:, K:]
    else:
        g, u = _rows(rng, N, K, 3, t, 3.0), _rows(rng, N, K, 5, t)
    Xq = kq.kq_swiglu_q8_1(g, u)
    assert_q8_blocks(Xq.cpu().numpy(), deo.swiglu(_f64(g), _f64(u)), SWIGLU_REL, f"{dtype} {N}x{K} {how}")


def test_swiglu_extremes():
    import torch
    g = torch.zeros(1, 160, device="cuda")
    u = torch.ones(1, 160, device="cuda")
    g[0, :32] = -200.0                  # exp overflows: silu is -0
    g[0, 32:64] = 200.0
    g[0, 64] = float("nan")
    u[0, 96] = float("inf")
    g[0, 96:128] = 1.0
    d, _, q = deo.unpack_q8_1(kq.kq_swiglu_q8_1(g, u).cpu().numpy())
    assert d[0, 0] == 0 and np.all(q[0, 0] == 0)
    assert np.all(q[0, 1] == 127) and d[0, 1] == float(np.float16(200 / 127))
    assert np.isnan(d[0, 2]) and np.isinf(d[0, 3])
    assert d[0, 4] == 0


def test_offsets_beyond_32_bits():
    import torch
    N, K = 140_000, 16_384                  # 2.3e9 elements
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    X = torch.randn(N, K, generator=gen, device="cuda", dtype=torch.bfloat16)
    gamma = torch.ones(K, device="cuda")
    at = [0, 131_071, 131_072, N - 1]
    H, Y, Xq = kq.kq_add_rmsnorm_q8_1(X, X, gamma, 1e-5, Y=True)
    want = kq.kq_add_rmsnorm_q8_1(X[at], X[at], gamma, 1e-5, Y=True)
    for full, part in zip((H, Y, Xq), want):
        assert torch.equal(full[at], part)
    del H, Y, Xq
    got = kq.kq_swiglu_q8_1(X, X)
    assert torch.equal(got[at], kq.kq_swiglu_q8_1(X[at], X[at]))


def test_same_codes_as_the_quantiser():
    """SwiGLU with a gate whose silu is the gate itself: the codes kq_quantize_q8_1 makes."""
    import torch
    g = torch.full((6, 2048), 128.0, device="cuda")     # exp(-128) is below half a step of 1
    u = torch.from_numpy(np.random.default_rng(1).standard_normal((6, 2048)).astype(np.float32)).cuda()
    assert torch.equal(kq.kq_swiglu_q8_1(g, u), kq.kq_quantize_q8_1(128.0 * u))


def test_on_another_stream():
    import torch
    rng = np.random.default_rng(2)
    X = _rows(rng, 65, 4096, 0, torch.float32)
    gamma = torch.ones(4096, device="cuda")
    want = kq.kq_add_rmsnorm_q8_1(X, None, gamma, 1e-5)[2]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kq.kq_add_rmsnorm_q8_1(X, None, gamma, 1e-5, stream=side)[2]
    side.synchronize()
    assert torch.equal(got, want)
