"""The attention-side operators together, as the example's decode step uses them: every stage against the oracle on the
GPU's previous output, and tokens generated by one CUDA graph against those of calls that are waited for."""
import os
import sys

import numpy as np
import pytest

import quantized_weight_matmul_q4_gb300 as kq
from _attnutil import U32, f64
from oracle import attn_oracle as ao
from oracle import decode_oracle as deo
from test_gpu_attn import _bound, _check_q8

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


class _Waited:
    """The package, every call followed by a wait for the GPU."""

    def __getattr__(self, name):
        import torch
        f = getattr(kq, name)
        if name.endswith(("_bytes", "_shape")):
            return f

        def call(*args, **kw):
            torch.cuda.synchronize()
            r = f(*args, **kw)
            torch.cuda.synchronize()
            return r
        return call


def _make(example, B, lengths, **kw):
    import torch
    torch.manual_seed(B)
    step = example.DecodeStep(B, max(lengths) + 40, D=512, heads=8, kv_heads=2, vocab=3001, page=16, group=64, seed=B, **kw)
    K, V = (torch.randn(sum(lengths), 2, step.head_dim, device="cuda") for _ in range(2))
    step.prefill(K.to(torch.bfloat16), V.to(torch.bfloat16), lengths)
    step.tokens.copy_(torch.arange(B, device="cuda"))
    return step


@pytest.mark.parametrize("head_dim", [64, 128])
def test_stages_against_the_oracle(head_dim):
    import decode_step as example
    import torch
    B, lengths = 3, [33, 0, 100]
    step = _make(example, B, lengths, head_dim=head_dim)
    before, pos = step.cache.cpu().numpy(), step.positions.cpu().numpy()
    u = torch.rand(B, device="cuda")
    tokens, probs = step(u)
    Y = f64(step.Y).reshape(B, 12, head_dim)
    cs = step.cos_sin.cpu().numpy()[pos]
    y, bnd = ao.norm_rope(Y[:, :8], f64(step.q_gamma), step.eps, cs, "half")
    assert np.all(np.abs(f64(step.Q) - y) <= 16 * U32 * bnd + 2.0 ** -8 * (np.abs(y) + 16 * U32 * bnd))
    table = step.table.cpu().numpy()
    Yf = step.Y.cpu().numpy().reshape(B, 12, head_dim)
    ao.append(before, table, 16, ao.turn_fp32(Yf[:, 8:10], cs, "half"), Yf[:, 10:], pos, np.arange(B))
    assert np.array_equal(step.cache.cpu().numpy(), before)
    lens = [n + 1 for n in lengths]
    assert step.kv_len.tolist() == lens and step.positions.tolist() == lens
    o, E, S = ao.attention(f64(step.Q), before, table, 16, lens)
    tol = _bound(o, E, S, "bf16", 101, True)
    _check_q8(step.Aq.cpu().numpy(), o.reshape(B, -1), tol.reshape(B, -1), "attention")
    W, s, z = (t.cpu() for t in step.head)
    L, bound = deo.g4_matmul(W.numpy(), s.double().numpy(), z.numpy(), 64, step.Hq.cpu().numpy())
    assert np.all(np.abs(f64(step.logits) - L) <= (512 // 32 + 12) * U32 * bound + 1e-30)
    ids, p = ao.sample(f64(step.logits), u.cpu().numpy(), temperature=np.full(B, np.float32(0.8)), top_k=[50] * B,
                       top_p=np.full(B, np.float32(0.95)))
    assert np.array_equal(tokens.cpu().numpy(), ids) and np.allclose(f64(probs), p, rtol=1e-6)
    assert kq.kq_get_device_error() == 0


@pytest.mark.parametrize("B,lengths", [(1, [70]), (5, [3, 0, 130, 64, 15]), (40, [(7 * i) % 50 for i in range(40)])])
def test_tokens_of_a_graph(B, lengths, monkeypatch):
    import decode_step as example
    import torch
    steps = 12
    U = torch.rand(steps, B, device="cuda")
    monkeypatch.setattr(example, "kq", _Waited())
    one = _make(example, B, lengths)
    want = [tuple(t.clone() for t in one(u)) for u in U]
    monkeypatch.setattr(example, "kq", kq)

    two = _make(example, B, lengths)                     # calls one after the other, nothing waited for
    got = [tuple(t.clone() for t in two(u)) for u in U]
    for (i, p), (j, r) in zip(want, got):
        assert torch.equal(i, j) and torch.equal(p, r)

    three = _make(example, B, lengths)
    state = [t.clone() for t in (three.tokens, three.kv_len, three.positions, three.cache)]
    u = U[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        three(u)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        three(u)
    for t, s in zip((three.tokens, three.kv_len, three.positions, three.cache), state):
        t.copy_(s)
    for k in range(steps):
        u.copy_(U[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(three.tokens, want[k][0]) and torch.equal(three.probs, want[k][1]), k
    assert torch.equal(three.cache, one.cache)
    assert kq.kq_get_device_error() == 0


def test_two_graphs_with_a_workspace_each():
    """Two captured attention calls at once on two streams, each with its own workspace."""
    import torch
    import decode_step as example
    steps = [_make(example, 5, [300, 20, 7, 0, 150]) for _ in range(2)]
    steps[1].Q.normal_(), steps[0].Q.normal_()
    for s in steps:
        s.kv_len.clamp_(min=1)
    want = [kq.kq_attn_q4(s.Q, s.cache, s.table, s.kv_len, O=False, Xq=True)[1] for s in steps]
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in steps]
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                kq.kq_attn_q4(s.Q, s.cache, s.table, s.kv_len, O=False, Xq=s.Aq, ws=s.ws)
        graphs.append(g)
    for _ in range(10):
        for s in steps:
            s.Aq.zero_()
        torch.cuda.synchronize()
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s.Aq, w) for s, w in zip(steps, want))


def test_prompt_in_chunks():
    """A prompt whose rows attend to the cache in chunks as they are written: as all at once, and read back from it."""
    import torch
    torch.manual_seed(3)
    L, H, Hq, D, P = 150, 2, 6, 128, 32
    K, V, Q = (torch.randn(L, h, D, device="cuda", dtype=torch.bfloat16) for h in (H, H, Hq))
    cache = torch.zeros(kq.kv_cache_q4_shape(5, H, P, D), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[4, 0, 3, 1, 2]], dtype=torch.int32, device="cuda")
    pos, seq = torch.arange(L, dtype=torch.int32, device="cuda"), torch.zeros(L, dtype=torch.int32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    parts, at = [], 0
    for n in (1, 31, 64, 54):
        rows = slice(at, at + n)
        kq.kq_kv_append_q4(K[rows], V[rows], cache, table, pos[rows].contiguous(), seq_ids=seq[:n])
        at += n
        parts.append(kq.kq_attn_q4(Q[rows], cache, table, i32(at), q_start=i32(0, n))[0])
    O, _ = kq.kq_attn_q4(Q, cache, table, i32(L), q_start=i32(0, L))
    o, E, S = ao.attention(f64(Q), cache.cpu().numpy(), table.cpu().numpy(), P, [L], q_start=[0, L])
    tol = _bound(o, E, S, "bf16", L)
    tol = tol + 2.0 ** -8 * (np.abs(o) + tol)
    assert np.all(np.abs(f64(O) - o) <= tol) and np.all(np.abs(f64(torch.cat(parts)) - o) <= tol)
    k, v = kq.kq_kv_gather_q4(cache, table, pos, seq_ids=seq, dtype=torch.float32)
    q = Q.float().view(L, H, Hq // H, D).permute(1, 2, 0, 3)
    s = torch.matmul(q, k.permute(1, 2, 0)[:, None]) * D ** -0.5
    s = s.masked_fill(torch.triu(torch.ones(L, L, dtype=torch.bool, device="cuda"), 1), float("-inf"))
    again = torch.matmul(torch.softmax(s, -1), v.permute(1, 0, 2)[:, None]).permute(2, 0, 1, 3).reshape(L, Hq, D)
    assert np.all(np.abs(f64(O) - f64(again)) <= 2 * tol + 1e-5)


@pytest.mark.parametrize("args", [[], ["1", "70"]])
def test_example_runs(args, monkeypatch, capsys):
    import decode_step as example
    monkeypatch.setattr(sys, "argv", ["decode_step.py", *args])
    example.main()
    assert "us as a CUDA graph" in capsys.readouterr().out
