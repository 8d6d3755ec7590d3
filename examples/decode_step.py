"""Decode steps of a layer of attention on 4-bit weights and a 4-bit cache, from the tokens' rows to the next tokens:

    kq_add_rmsnorm_q8_1   RMSNorm of the tokens' rows, Q8_1 activations
    kq_matvec_g4          queries, keys and values
    kq_qk_norm_rope       the queries' heads normed and turned to their positions
    kq_kv_append_q4       keys (turned on the way) and values to the paged 4-bit cache
    kq_attn_q4            attention over the cache, its output as Q8_1 activations
    kq_matvec_g4          the output projection
    kq_add_rmsnorm_q8_1   residual addition, RMSNorm, Q8_1 activations
    kq_matvec_g4          logits
    kq_sample             the next tokens

    python examples/decode_step.py [sequences] [places]

runs it on random weights for sequences that already have so many places in the cache, eagerly and as a CUDA graph, and prints
the time of a step. Lengths, positions and tokens live on the GPU and are moved on by the step itself, so
that a graph of one step generates token after token. No step waits for the host.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import quantized_weight_matmul_q4_gb300 as kq
from moe_decode_layer import random_g4


def rope_table(n: int, rot: int, base: float = 10000.0):
    """fp32 [n, rot]: the cosines of every position's angles, then their sines."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


class DecodeStep:
    """Weights, a cache for `places` places of each of B sequences, and buffers for a step."""

    def __init__(self, B: int, places: int, D: int = 2048, heads: int = 16, kv_heads: int = 4, head_dim: int = 128,
                 vocab: int = 32000, page: int = 64, group: int = 128, eps: float = 1e-6, seed: int = 0):
        self.B, self.D, self.heads, self.kv_heads, self.head_dim = B, D, heads, kv_heads, head_dim
        self.vocab, self.group, self.eps = vocab, group, eps
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.rows = (heads + 2 * kv_heads) * head_dim
        self.qkv = random_g4(self.rows, D, group, seed + 1)
        self.out = random_g4(D, heads * head_dim, group, seed + 2)
        self.head = random_g4(vocab, D, group, seed + 3)
        self.embedding = torch.randn(vocab, D, generator=gen, device="cuda")
        self.gamma, self.gamma2, self.q_gamma = (1.0 + 0.1 * torch.randn(n, generator=gen, device="cuda")
                                                 for n in (D, D, head_dim))
        pages = -(-places // page)
        self.cos_sin = rope_table(pages * page, head_dim)
        self.cache = torch.zeros(kq.kv_cache_q4_shape(B * pages, kv_heads, page, head_dim), dtype=torch.uint8, device="cuda")
        self.table = torch.randperm(B * pages, generator=gen, device="cuda").to(torch.int32).view(B, pages)
        i32, f32, dev = torch.int32, torch.float32, "cuda"
        self.tokens = torch.zeros(B, dtype=i32, device=dev)
        self.probs = torch.zeros(B, dtype=f32, device=dev)
        self.kv_len = torch.zeros(B, dtype=i32, device=dev)      # places in the cache
        self.positions = torch.zeros(B, dtype=i32, device=dev)   # of the next token
        self.temperature = torch.full((B,), 0.8, device=dev)
        self.top_k = torch.full((B,), 50, dtype=i32, device=dev)
        self.top_p = torch.full((B,), 0.95, device=dev)
        self.Xq = torch.empty(B, D // 32, 36, dtype=torch.uint8, device=dev)
        self.Y = torch.empty(B, self.rows, dtype=f32, device=dev)
        self.Q = torch.empty(B, heads, head_dim, dtype=torch.bfloat16, device=dev)
        self.Aq = torch.empty(B, heads * head_dim // 32, 36, dtype=torch.uint8, device=dev)
        self.A = torch.empty(B, D, dtype=f32, device=dev)
        self.H = torch.empty(B, D, dtype=f32, device=dev)
        self.Hq = torch.empty_like(self.Xq)
        self.logits = torch.empty(B, vocab, dtype=f32, device=dev)
        self.ws = torch.empty(kq.kq_attn_q4_workspace_bytes(heads, kv_heads, head_dim, B, B), dtype=torch.uint8, device=dev)

    def prefill(self, K, V, lengths):
        """Writes prompts' keys and values [N, kv_heads, head_dim], packed one after the other, to the cache."""
        n = torch.tensor(lengths, device="cuda")
        seq = torch.repeat_interleave(torch.arange(self.B, device="cuda"), n, output_size=sum(lengths))
        pos = torch.arange(sum(lengths), device="cuda") - (torch.cumsum(n, 0) - n)[seq]
        kq.kq_kv_append_q4(K, V, self.cache, self.table, pos.to(torch.int32), seq_ids=seq.to(torch.int32),
                           cos_sin=self.cos_sin)
        self.kv_len.copy_(n)
        self.positions.copy_(n)

    def __call__(self, u):
        """One step for random numbers u fp32 [B]: the tokens become the next ones."""
        B, D, G, hd = self.B, self.D, self.group, self.head_dim
        X = self.embedding.index_select(0, self.tokens)
        kq.kq_add_rmsnorm_q8_1(X, None, self.gamma, self.eps, Xq=self.Xq)
        W, s, z = self.qkv
        kq.kq_matvec_g4(W, s, self.Xq, self.rows, D, G, zeros=z, Y=self.Y)
        heads = self.Y.view(B, -1, hd)
        q, k, v = heads[:, :self.heads], heads[:, self.heads:self.heads + self.kv_heads], heads[:, self.heads + self.kv_heads:]
        kq.kq_qk_norm_rope(q, None, self.cos_sin, self.positions, q_gamma=self.q_gamma, eps=self.eps, Qo=self.Q)
        kq.kq_kv_append_q4(k, v, self.cache, self.table, self.positions, cos_sin=self.cos_sin)
        self.kv_len.add_(1)
        kq.kq_attn_q4(self.Q, self.cache, self.table, self.kv_len, O=False, Xq=self.Aq, ws=self.ws)
        W, s, z = self.out
        kq.kq_matvec_g4(W, s, self.Aq, D, self.heads * hd, G, zeros=z, Y=self.A)
        kq.kq_add_rmsnorm_q8_1(self.A, X, self.gamma2, self.eps, H=self.H, Xq=self.Hq)
        W, s, z = self.head
        kq.kq_matvec_g4(W, s, self.Hq, self.vocab, D, G, zeros=z, Y=self.logits)
        kq.kq_sample(self.logits, u, temperature=self.temperature, top_k=self.top_k, top_p=self.top_p, ids=self.tokens,
                     probs=self.probs)
        self.positions.add_(1)
        return self.tokens, self.probs


def main() -> None:
    B = int(sys.argv[1]) if len(sys.argv) > 1 else 4
    have = int(sys.argv[2]) if len(sys.argv) > 2 else 2000
    steps = 200
    step = DecodeStep(B, have + 3 * steps)
    step.prefill(*(torch.randn(B * have, step.kv_heads, step.head_dim, device="cuda", dtype=torch.bfloat16) for _ in range(2)),
                 [have] * B)
    u = torch.rand(B, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(u)                          # warm-up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(u)

    def us(f):
        for _ in range(10):
            f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(steps):
            f()
        b.record()
        b.synchronize()
        return 1e3 * a.elapsed_time(b) / steps

    print(f"{B} sequence(s) of {have} places: {us(lambda: step(u)):.1f} us per step eagerly, {us(graph.replay):.1f} us as a CUDA graph")
    if kq.kq_get_device_error() != 0:
        raise RuntimeError("a kernel recorded an error")


if __name__ == "__main__":
    main()
