"""kq_add_rmsnorm_q8_1 on rows so long that the order of the sum of squares counts. Against the
fp64 definition."""
import numpy as np
import pytest

from oracle import decode_oracle as deo
import quantized_weight_matmul_q4_gb300 as kq
from _decodeutil import U32, assert_q8_blocks

pytestmark = pytest.mark.gpu

NORM_REL = 64 * U32      # of y before it is rounded, as in the norm's other tests


@pytest.mark.parametrize("K", [32_800, 262_144, 1 << 20, (1 << 22) + 32])
@pytest.mark.parametrize("residual", [False, True])
def test_long_rows(K, residual):
    """Equal values whose squares, added one after the other, are rounded down every time:
    x^2 lies 0.9 of half a step above 1 when a thread's sum is at its largest."""
    import torch
    steps = 2.0 ** np.ceil(np.log2(K / 512))
    x = np.float32(np.sqrt(1 + 0.9 * steps * 2.0 ** -25))
    X = torch.full((2, K), float(x), device="cuda")
    R = None
    if residual:
        X = X * 0.5
        R = X.clone()
    X[1] = torch.from_numpy(np.random.default_rng(K).standard_normal(K).astype(np.float32)).cuda()
    _, Y, Xq = kq.kq_add_rmsnorm_q8_1(X, R, torch.ones(K, device="cuda"), 1e-5, Y=True)
    f64 = lambda t: None if t is None else t.cpu().double().numpy()  # noqa: E731
    _, y = deo.add_rmsnorm(f64(X), f64(R), np.ones(K), 1e-5)
    assert np.all(np.abs(f64(Y) - y) <= np.abs(y) * (NORM_REL + U32))
    assert_q8_blocks(Xq.cpu().numpy(), y, NORM_REL, f"K = {K}")
