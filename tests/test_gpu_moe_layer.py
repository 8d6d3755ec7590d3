"""The operators of a mixture-of-experts decode layer run together (the example's
layer), eagerly and from a CUDA graph: every stage against the fp64 oracle
applied to what the GPU produced before it, so that a stage that read its input
too early fails on its own."""
import os
import sys

import numpy as np
import pytest

from oracle import decode_oracle as deo
import quantized_weight_matmul_q4_gb300 as kq
from _decodeutil import U32, assert_g4, assert_q8_blocks

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _np(t):
    a = t.detach().cpu()
    return a.numpy() if a.dtype.is_floating_point is False else a.double().numpy()


def _g4(w):
    W, s, z = w
    return W.cpu().numpy(), s.cpu().double().numpy(), None if z is None else z.cpu().numpy()


def _check(layer, X, R, H, out):
    T, top_k, F, D, E = layer.T, layer.top_k, layer.F, layer.D, layer.E
    import torch
    assert torch.equal(H, X + R)
    _, y = deo.add_rmsnorm(_np(X), _np(R), _np(layer.gamma), layer.eps)
    rel = 64 * U32                                              # as in the norm's own test
    assert np.all(np.abs(_np(layer.Y) - y) <= np.abs(y) * (rel + U32))
    Xq = layer.Xq.cpu().numpy()
    assert_q8_blocks(Xq, y, rel, "norm")
    ids, p = deo.route(_np(layer.logits), top_k, score="sigmoid", bias=_np(layer.bias))
    got_ids = layer.ids.cpu().numpy()
    assert np.array_equal(got_ids, ids)
    assert np.all(np.abs(_np(layer.probs) - p) <= 120 * U32 * p)
    W, s, z = _g4(layer.up)
    Y, B = deo.moe_g4(W, s, z, layer.group, E, ids, Xq, 2 * F)
    assert_g4(layer.gu.cpu().numpy(), Y, B, D, "gate and up")
    gu = _np(layer.gu).reshape(T * top_k, 2 * F)
    Aq = layer.Aq.cpu().numpy()
    assert_q8_blocks(Aq, deo.swiglu(gu[:, :F], gu[:, F:]), 10 * U32, "swiglu")
    W, s, z = _g4(layer.down)
    Y, B = deo.moe_g4(W, s, z, layer.group, E, ids, Aq, D)
    assert_g4(layer.slots.cpu().numpy(), Y, B, F, "down")
    W, s, z = _g4(layer.shared)
    Y, B = deo.g4_matmul(W, s, z, layer.group, Xq)
    assert_g4(layer.dense.cpu().numpy(), Y, B, D, "dense")
    terms = _np(layer.slots) * _np(layer.probs)[..., None]
    total = terms.sum(1) + _np(layer.dense)
    bound = (np.abs(terms).sum(1) + np.abs(_np(layer.dense))) * (top_k + 2) * U32
    assert np.all(np.abs(_np(out) - total) <= bound)


@pytest.mark.parametrize("T", [1, 3, 40])
@pytest.mark.parametrize("graph", [False, True])
def test_moe_decode_layer(T, graph):
    import torch
    from moe_decode_layer import MoeDecodeLayer
    layer = MoeDecodeLayer(T, D=512, F=256, E=16, top_k=4, group=64, seed=T)
    X, R = torch.randn(T, 512, device="cuda"), torch.randn(T, 512, device="cuda")
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer(X, R)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            H, out = layer(X, R)
        X.copy_(torch.randn(T, 512, device="cuda"))             # other inputs than the capture saw
        g.replay()
        g.replay()                                              # back to back: the buffers are used again
    else:
        layer(X, R)
        H, out = layer(X, R)
    torch.cuda.synchronize()
    assert kq.kq_get_device_error() == 0
    _check(layer, X, R, H, out)
