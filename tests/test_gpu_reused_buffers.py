"""The example's decode layer run several times over in one CUDA graph, with other inputs every
time and the same intermediate buffers: each kernel begins while the one before it may still be
writing what it reads, over what the last run left there. The results are those of calls that
are waited for one by one."""
import os
import sys

import pytest

import quantized_weight_matmul_q4_gb300 as kq

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


class _Waited:
    """The package, every call followed by a wait for the GPU."""

    def __getattr__(self, name):
        import torch
        f = getattr(kq, name)

        def call(*args, **kw):
            torch.cuda.synchronize()
            r = f(*args, **kw)
            torch.cuda.synchronize()
            return r
        return call


@pytest.mark.parametrize("T", [1, 2, 3, 9, 40])
def test_layers_over_the_same_buffers(T, monkeypatch):
    import torch
    import moe_decode_layer as example
    RUNS, D = 6, 512
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    X = [torch.randn(T, D, generator=gen, device="cuda") * 3.0 ** i for i in range(RUNS)]
    R = [torch.randn(T, D, generator=gen, device="cuda") for _ in range(RUNS)]
    make = lambda: example.MoeDecodeLayer(T, D=D, F=256, E=16, top_k=4, group=64, seed=T)  # noqa: E731

    monkeypatch.setattr(example, "kq", _Waited())
    layer = make()
    want = [tuple(t.clone() for t in layer(x, r)) for x, r in zip(X, R)]
    monkeypatch.setattr(example, "kq", kq)

    layer = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(X[0], R[0])
    torch.cuda.current_stream().wait_stream(side)
    got = [(torch.empty_like(X[0]), torch.empty_like(X[0])) for _ in range(RUNS)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(RUNS):
            H, out = layer(X[i], R[i])
            got[i][0].copy_(H)
            got[i][1].copy_(out)
    for _ in range(20):
        for h, o in got:
            h.zero_(), o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i in range(RUNS):
            assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1]), i
    assert kq.kq_get_device_error() == 0


@pytest.mark.parametrize("N", [1, 2, 8])
def test_products_after_row_operators(N):
    """norm -> product -> SwiGLU -> product with nothing of PyTorch's between them."""
    import torch
    D, F, RUNS = 1024, 768, 6
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)

    def g4(M, K):
        return (torch.randint(0, 256, (M, K // 2), generator=gen, device="cuda", dtype=torch.uint8),
                (0.05 * torch.rand(M, K // 128, generator=gen, device="cuda") + 0.01).half())

    up, down = g4(2 * F, D), g4(D, F)
    gamma = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    X = [torch.randn(N, D, generator=gen, device="cuda") * 2.0 ** i for i in range(RUNS)]
    Xq = torch.empty(N, D // 32, 36, dtype=torch.uint8, device="cuda")
    Aq = torch.empty(N, F // 32, 36, dtype=torch.uint8, device="cuda")
    gu = torch.empty(N, 2 * F, device="cuda")

    def run(x, out, wait):
        for step in (lambda: kq.kq_add_rmsnorm_q8_1(x, None, gamma, 1e-6, Xq=Xq),
                     lambda: kq.kq_matvec_g4(*up, Xq, 2 * F, D, 128, Y=gu),
                     lambda: kq.kq_swiglu_q8_1(gu[:, :F], gu[:, F:], Xq=Aq),
                     lambda: kq.kq_matvec_g4(*down, Aq, D, F, 128, Y=out)):
            step()
            if wait:
                torch.cuda.synchronize()

    want, got = ([torch.empty(N, D, device="cuda") for _ in range(RUNS)] for _ in range(2))
    for x, w in zip(X, want):
        run(x, w, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, g in zip(X, got):
            run(x, g, False)
    for _ in range(50):
        for g in got:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
