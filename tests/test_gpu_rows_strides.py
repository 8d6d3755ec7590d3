"""kq_add_rmsnorm_q8_1 with outputs whose rows lie at odd element offsets, out of place and in
place, in each of the kernel's forms: the same rows as the aligned call's, and nothing written
between them."""
import numpy as np
import pytest

import quantized_weight_matmul_q4_gb300 as kq

pytestmark = pytest.mark.gpu


def _padded(src, pad, sentinel):
    """A copy of src [N, K] with `pad` elements of `sentinel` behind every row: (view, buffer)."""
    import torch
    N, K = src.shape
    buf = torch.full((N, K + pad), sentinel, dtype=src.dtype, device="cuda")
    buf[:, :K] = src
    return buf[:, :K], buf


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("N,K", [(5, 1120), (2000, 1120), (4, 12000), (3, 33024)])
@pytest.mark.parametrize("pad", [1, 2, 3])
@pytest.mark.parametrize("where", ["apart", "X", "R"])
def test_outputs_at_odd_offsets(dtype, N, K, pad, where):
    import torch
    t = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(K + pad)
    X = torch.randn(N, K, generator=gen, device="cuda").to(t)
    R = (3 * torch.randn(N, K, generator=gen, device="cuda")).to(t)
    gamma = 1 + 0.3 * torch.randn(K, generator=gen, device="cuda")
    H, Y, Xq = kq.kq_add_rmsnorm_q8_1(X, R, gamma, 1e-5, Y=True)
    x, xb = _padded(X, pad, 11.0)
    r, rb = _padded(R, pad + 1, 12.0)
    h, hb = {"X": (x, xb), "R": (r, rb), "apart": _padded(torch.zeros_like(X), pad, 13.0)}[where]
    y, yb = _padded(torch.zeros_like(X), pad, 14.0)
    got = kq.kq_add_rmsnorm_q8_1(x, r, gamma, 1e-5, H=h, Y=y)
    assert got[0] is h and got[1] is y
    assert torch.equal(h, H) and torch.equal(y, Y) and torch.equal(got[2], Xq)
    for buf, mark in ((xb, 11.0), (rb, 12.0), (yb, 14.0)) + (((hb, 13.0),) if where == "apart" else ()):
        assert bool((buf[:, K:] == mark).all())
    if where != "X":
        assert torch.equal(x, X)
    if where != "R":
        assert torch.equal(r, R)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("N,K", [(4, 96), (300, 1120)])
def test_swiglu_rows_at_odd_offsets(dtype, N, K):
    import torch
    t = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(K)
    g, u = (torch.randn(N, K, generator=gen, device="cuda").to(t) for _ in range(2))
    want = kq.kq_swiglu_q8_1(g, u)
    for pg, pu in ((1, 0), (0, 1), (1, 2), (3, 3)):
        assert torch.equal(kq.kq_swiglu_q8_1(_padded(g, pg, 5.0)[0], _padded(u, pu, 5.0)[0]), want), (pg, pu)
