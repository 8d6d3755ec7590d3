"""kq_sample where a bin of the first histogram is a few hundred keys of fp32, so that the search of a nucleus by several CTAs
ends with its first histogram of keys: logits far from 0, or low temperatures."""
import numpy as np
import pytest

import quantized_weight_matmul_q4_gb300 as kq
from _attnutil import torch_dtype
from oracle import attn_oracle as ao
from test_gpu_sample import _check

pytestmark = pytest.mark.gpu

F = np.float32


def keys_of_a_bin(top, T):
    """fp32 values within a sixteenth of an octave of weight, near `top`."""
    return T * np.log(2) / 16 / np.spacing(F(abs(top)))


@pytest.mark.parametrize("V", [40003, 152064])
@pytest.mark.parametrize("dtype,offset,spread,T", [
    ("fp32", 1000.0, 0.5, 1.0), ("fp32", -4096.0, 1.0, 1.0), ("fp32", 20.0, 0.02, 0.04), ("fp32", 4096.0, 0.0, 1.0),
    ("fp16", 1000.0, 1.0, 1.0), ("bf16", 4096.0, 20.0, 8.0), ("bf16", -600.0, 0.0, 1.0)])
def test_nucleus_of_logits_far_from_zero(dtype, offset, spread, T, V):
    rng = np.random.default_rng(V + int(abs(offset)))
    N = 3
    assert keys_of_a_bin(offset, T) < 1024
    L = (offset + spread * rng.standard_normal((N, V))).astype(F)
    x = _rows(L, dtype)
    for p in (0.3, 0.9):
        _check(x, rng.random(N).astype(F), top_p=np.full(N, p, F), temperature=np.full(N, T, F))
    # A top_k that leaves all tokens that there are takes the same way.
    x[:, 5] = float("-inf")
    _check(x, rng.random(N).astype(F), top_k=np.full(N, V - 1, np.int32), top_p=np.full(N, 0.7, F), temperature=np.full(N, T, F))


def _rows(L, dtype):
    import torch
    return torch.from_numpy(L).cuda().to(torch_dtype(dtype))


def test_the_same_tokens_every_time():
    """Many rows at once, so that the CTAs of a row are apart in time."""
    import torch
    rng = np.random.default_rng(11)
    N, V = 96, 90001
    x = _rows((1000.0 + 0.5 * rng.standard_normal((N, V))).astype(F), "fp32")
    u, p = (torch.from_numpy(a.astype(F)).cuda() for a in (rng.random(N), rng.uniform(0.2, 0.95, N)))
    want, probs = kq.kq_sample(x, u, top_p=p)
    for n in (0, 50, 95):
        ids, _ = ao.sample(x[n:n + 1].double().cpu().numpy(), u[n:n + 1].cpu().numpy(), top_p=p[n:n + 1].cpu().numpy())
        assert ids[0] == int(want[n])
    for _ in range(50):
        ids, again = kq.kq_sample(x, u, top_p=p)
        assert torch.equal(ids, want) and torch.equal(again, probs)
