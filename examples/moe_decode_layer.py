"""A mixture-of-experts decode layer on 4-bit experts, with the library's operators
from the residual stream back to the residual stream:

    kq_add_rmsnorm_q8_1   residual addition, RMSNorm, Q8_1 activations
    router logits         (a plain fp32 product of the normed rows)
    kq_moe_route          experts and weights of every token
    kq_moe_matvec_g4      gate and up rows of the chosen experts
    kq_swiglu_q8_1        SwiGLU, Q8_1 activations of every (token, slot)
    kq_moe_matvec_g4      down rows
    kq_moe_combine        weighted sum of a token's slots
    kq_matvec_g4          a dense 4-bit projection of the same activations (a shared expert's place)

    python examples/moe_decode_layer.py [tokens]

runs it on random weights, eagerly and as a CUDA graph, and prints the time of a
step. No step waits for the host, and none allocates inside the graph.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import quantized_weight_matmul_q4_gb300 as kq


def random_g4(rows: int, K: int, group: int, seed: int, zeros: bool = True):
    """(codes, scales, zero points) of `rows` rows of K 4-bit weights of about 1 / sqrt(K)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    groups = -(-K // group)
    W = torch.randint(0, 256, (rows, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s = (0.2 / K ** 0.5 * torch.exp(0.25 * torch.randn(rows, groups, generator=gen, device="cuda"))).to(torch.bfloat16)
    z = torch.randint(5, 11, (rows, groups), generator=gen, device="cuda", dtype=torch.uint8) if zeros else None
    return W, s, z


class MoeDecodeLayer:
    """Weights, and buffers for `tokens` tokens, of one layer (hidden size D, experts of F)."""

    def __init__(self, tokens: int, D: int = 2048, F: int = 768, E: int = 128, top_k: int = 8, group: int = 128,
                 eps: float = 1e-6, seed: int = 0):
        self.T, self.D, self.F, self.E, self.top_k, self.group, self.eps = tokens, D, F, E, top_k, group, eps
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.gamma = 1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        self.router = torch.randn(D, E, generator=gen, device="cuda") / D ** 0.5
        self.bias = 1e-3 * torch.round(20 * torch.randn(E, generator=gen, device="cuda"))
        self.up = random_g4(E * 2 * F, D, group, seed + 1)      # gate rows, then up rows, of every expert
        self.down = random_g4(E * D, F, group, seed + 2)
        self.shared = random_g4(D, D, group, seed + 3, zeros=False)
        f32, u8, dev = torch.float32, torch.uint8, "cuda"
        self.H = torch.empty(tokens, D, dtype=f32, device=dev)
        self.Y = torch.empty(tokens, D, dtype=f32, device=dev)
        self.Xq = torch.empty(tokens, D // 32, 36, dtype=u8, device=dev)
        self.logits = torch.empty(tokens, E, dtype=f32, device=dev)
        self.ids = torch.empty(tokens, top_k, dtype=torch.int32, device=dev)
        self.probs = torch.empty(tokens, top_k, dtype=f32, device=dev)
        self.gu = torch.empty(tokens, top_k, 2 * F, dtype=f32, device=dev)
        self.Aq = torch.empty(tokens * top_k, F // 32, 36, dtype=u8, device=dev)
        self.slots = torch.empty(tokens, top_k, D, dtype=f32, device=dev)
        self.out = torch.empty(tokens, D, dtype=f32, device=dev)
        self.dense = torch.empty(tokens, D, dtype=f32, device=dev)

    def __call__(self, X, R):
        """X: the layer's input rows, R: the residual rows (fp32 [T, D]); returns (residual, output) rows."""
        T, D, F, E, top_k, G = self.T, self.D, self.F, self.E, self.top_k, self.group
        kq.kq_add_rmsnorm_q8_1(X, R, self.gamma, self.eps, H=self.H, Y=self.Y, Xq=self.Xq)
        torch.matmul(self.Y, self.router, out=self.logits)
        kq.kq_moe_route(self.logits, top_k, score="sigmoid", bias=self.bias, ids=self.ids, probs=self.probs)
        W, s, z = self.up
        kq.kq_moe_matvec_g4(W, s, E, self.ids, self.Xq, 2 * F, D, G, zeros=z, Y=self.gu)
        gu = self.gu.view(T * top_k, 2 * F)
        kq.kq_swiglu_q8_1(gu[:, :F], gu[:, F:], Xq=self.Aq)
        W, s, z = self.down
        kq.kq_moe_matvec_g4(W, s, E, self.ids, self.Aq, D, F, G, zeros=z, Y=self.slots)
        kq.kq_moe_combine(self.slots, self.probs, out=self.out)
        W, s, z = self.shared
        kq.kq_matvec_g4(W, s, self.Xq, D, D, G, zeros=z, Y=self.dense)
        return self.H, self.out.add_(self.dense)


def main() -> None:
    T = int(sys.argv[1]) if len(sys.argv) > 1 else 1
    layer = MoeDecodeLayer(T)
    X, R = torch.randn(T, layer.D, device="cuda"), torch.randn(T, layer.D, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(X, R)                      # warm-up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(X, R)

    def ms(step, n=200):
        for _ in range(20):
            step()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            step()
        b.record()
        b.synchronize()
        return a.elapsed_time(b) / n

    print(f"{T} token(s): {1e3 * ms(lambda: layer(X, R)):.1f} us per layer eagerly, "
          f"{1e3 * ms(graph.replay):.1f} us as a CUDA graph")
    if kq.kq_get_device_error() != 0:
        raise RuntimeError("a kernel recorded an error")


if __name__ == "__main__":
    main()
