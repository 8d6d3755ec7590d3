"""kq_sample on the GPU against its definition in 64 bits."""
import numpy as np
import pytest

import quantized_weight_matmul_q4_gb300 as kq
from _attnutil import f64, torch_dtype
from oracle import attn_oracle as ao

pytestmark = pytest.mark.gpu


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda() if a is not None else None


def _check(L, u, **kw):
    """ids and probabilities of rows L (a CUDA tensor) against the oracle."""
    dev = {k: _dev(v) for k, v in kw.items()}
    ids, probs = kq.kq_sample(L, _dev(u), **dev)
    want, p = ao.sample(f64(L), u, **kw)
    assert np.array_equal(ids.cpu().numpy(), want)
    # The share of two sums of weights, each within 2^-30, and its rounding.
    assert np.all(np.abs(f64(probs) - p) <= p * (2.0 ** -28 + 2.0 ** -24) + 1e-30)
    return ids


def _params(rng, N, k=True, p=True, m=True, T=True, V=1000):
    f = np.float32
    return {"temperature": rng.uniform(0.3, 1.5, N).astype(f) if T else None,
            "top_k": rng.integers(1, V + 1, N).astype(np.int32) if k else None,
            "top_p": rng.uniform(0.05, 1.0, N).astype(f) if p else None,
            "min_p": rng.uniform(0.0, 0.3, N).astype(f) if m else None}


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (5, 31), (40, 1000), (7, 1537), (2, 32003), (17, 4096)])
def test_all_limits(dtype, N, V):
    rng = np.random.default_rng(N + V)
    L = _dev((2.5 * rng.standard_normal((N, V))).astype(np.float32)).to(torch_dtype(dtype))
    for k in (False, True):
        for p in (False, True):
            for m in (False, True):
                for T in (False, True):
                    _check(L, rng.random(N).astype(np.float32), **_params(rng, N, k, p, m, T, min(V, 300)))


@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.3, 8.0, 60.0])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_flat_and_peaked_rows(dtype, spread):
    rng = np.random.default_rng(int(spread * 10))
    N, V = 24, 5003
    L = _dev((spread * rng.standard_normal((N, V)) + 4).astype(np.float32)).to(torch_dtype(dtype))
    for k, p in ((0, 1), (1, 0), (1, 1), (0, 0)):
        _check(L, rng.random(N).astype(np.float32), **_params(rng, N, k, p, False, True, V))


def test_large_vocabularies():
    rng = np.random.default_rng(2)
    for N, V in ((2, 152064), (1, 524288), (4, 100001)):
        L = _dev((2.5 * rng.standard_normal((N, V))).astype(np.float32))
        for k, p in ((1, 0), (0, 1), (1, 1)):
            _check(L, rng.random(N).astype(np.float32), **_params(rng, N, k, p, True, True, 50000))


def test_ties_go_to_the_lowest_index():
    """Whole numbers of equal logits at every limit; sums that are exact in 64 bits."""
    rng = np.random.default_rng(3)
    N, V = 64, 777
    L = rng.integers(-2, 3, (N, V)).astype(np.float32)
    k = rng.integers(1, V, N).astype(np.int32)
    _check(_dev(L), rng.random(N).astype(np.float32), top_k=k)
    _check(_dev(L), rng.random(N).astype(np.float32), top_p=rng.uniform(0.01, 0.99, N).astype(np.float32))
    _check(_dev(L), rng.random(N).astype(np.float32), top_k=k, top_p=rng.uniform(0.01, 0.99, N).astype(np.float32))
    same = np.full((N, 512), 1.25, np.float32)            # 512 equal weights: the prefix ends exactly where p says
    p = (rng.integers(1, 512, N) / 512).astype(np.float32)
    u = (rng.integers(0, 512, N) / 512).astype(np.float32)
    ids = _check(_dev(same), u, top_p=p)
    assert np.array_equal(ids.cpu().numpy(), np.floor(u * (p * 512)).astype(np.int64))
    ids = _check(_dev(same), u, top_k=k)
    assert np.all(ids.cpu().numpy() < k)
    zero = np.where(rng.random((N, 99)) < 0.5, 0.0, -0.0).astype(np.float32)      # both zeros are one value
    _check(_dev(zero), rng.random(N).astype(np.float32), top_k=np.full(N, 40, np.int32))


def test_greedy():
    import torch
    rng = np.random.default_rng(4)
    L = rng.integers(0, 50, (9, 20011)).astype(np.float32)
    for T in (0.0, -1.0, float("nan")):
        ids, probs = kq.kq_sample(_dev(L), torch.rand(9, device="cuda"), temperature=torch.full((9,), T, device="cuda"),
                                  top_p=torch.full((9,), 0.5, device="cuda"))
        assert np.array_equal(ids.cpu().numpy(), L.argmax(1)) and bool((probs == 1).all())
    ids, _ = kq.kq_sample(_dev(L), torch.rand(9, device="cuda"), top_k=torch.ones(9, dtype=torch.int32, device="cuda"))
    assert np.array_equal(ids.cpu().numpy(), L.argmax(1))
    # One greedy row among others.
    T = np.ones(9, np.float32)
    T[4] = 0
    _check(_dev(L), rng.random(9).astype(np.float32), temperature=T, top_k=np.full(9, 7, np.int32))


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_masked_rows(dtype):
    import torch
    rng = np.random.default_rng(5)
    N, V = 30, 3001
    L = (2 * rng.standard_normal((N, V))).astype(np.float32)
    L[rng.random((N, V)) < 0.98] = -np.inf
    L[3], L[4] = -np.inf, np.nan
    L[5] = -np.inf
    L[5, 2999] = -50.0
    L[6, ::7], L[7, 11], L[8] = np.nan, np.inf, -np.inf
    L[8, 100:102] = np.inf
    t = _dev(L).to(torch_dtype(dtype))
    low = torch.finfo(t.dtype).min
    t[9] = low                                            # the type's lowest value is a logit like any other
    t[10, 5:] = low
    for k, p, m in ((0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)):
        ids = _check(t, rng.random(N).astype(np.float32), **_params(rng, N, k, p, m, True, 60))
        assert ids[3] == 0 and ids[4] == 0 and ids[5] == 2999


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("masked", [0.5, 0.99])
def test_masked_rows_of_many_tokens(dtype, masked):
    """Rows that several CTAs share, of odd length: limits above what the mask leaves, few and many tokens left."""
    rng = np.random.default_rng(8)
    N, V = 6, 40003
    L = (2 * rng.standard_normal((N, V))).astype(np.float32)
    L[rng.random((N, V)) < masked] = -np.inf
    L[4, 7] = 30.0
    L[5, :-1] = -np.inf
    t = _dev(L).to(torch_dtype(dtype))
    u = rng.random(N).astype(np.float32)
    for k in (3, 300, 2048, 3000, 30000):
        K = np.full(N, k, np.int32)
        _check(t, u, top_k=K)
        for p in (0.3, 0.9, 0.999):
            _check(t, u, top_k=K, top_p=np.full(N, p, np.float32), temperature=np.full(N, 1.7, np.float32))
    for p in (0.5, 0.95):
        _check(t, u, top_p=np.full(N, p, np.float32), min_p=np.full(N, 0.01, np.float32))
    _check(t, u, min_p=np.full(N, 0.05, np.float32))
    _check(t, u)


def test_limits_at_their_ends():
    import torch
    rng = np.random.default_rng(6)
    N, V = 16, 900
    L = _dev((2 * rng.standard_normal((N, V))).astype(np.float32))
    u = rng.random(N).astype(np.float32)
    plain = _check(L, u)
    for kw in (dict(top_k=0), dict(top_k=-5), dict(top_k=V), dict(top_k=1 << 30), dict(top_p=1.0), dict(top_p=2.0), dict(min_p=0.0),
               dict(min_p=-1.0), dict(top_p=float("nan")), dict(min_p=float("nan"))):
        (name, v), = kw.items()
        t = torch.full((N,), v, dtype=torch.int32 if name == "top_k" else torch.float32, device="cuda")
        assert torch.equal(kq.kq_sample(L, _dev(u), **{name: t})[0], plain), kw
    best = L.argmax(1).to(torch.int32)
    for kw in (dict(top_p=0.0), dict(top_p=-1.0), dict(min_p=1.0), dict(min_p=7.0)):
        (name, v), = kw.items()
        ids, probs = kq.kq_sample(L, _dev(u), **{name: torch.full((N,), v, device="cuda")})
        assert torch.equal(ids, best) and bool((probs == 1).all()), kw
    for v in (0.0, 1.0 - 2.0 ** -24):
        _check(L, np.full(N, v, np.float32), **_params(rng, N, V=V))
    ids, _ = kq.kq_sample(L, torch.full((N,), 1.0, device="cuda"))     # beyond the range: the last token
    assert bool((ids == V - 1).all())
    for T in (1e-3, 1e-30, 1e-42, 1e4):
        _check(L, u, temperature=np.full(N, T, np.float32))


def test_strides_outputs_streams_and_graphs():
    import torch
    rng = np.random.default_rng(7)
    N, V = 6, 5000
    wide = torch.randn(N, V + 13, device="cuda") * 3
    L = wide[:, :V]
    u = torch.rand(N, device="cuda")
    want, p = kq.kq_sample(L.contiguous(), u)
    ids, probs = kq.kq_sample(L, u)
    assert torch.equal(ids, want) and torch.equal(probs, p)
    half = wide.bfloat16()
    a, _ = kq.kq_sample(half[:, :V], u)
    b, _ = kq.kq_sample(half[:, :V].contiguous(), u)
    assert torch.equal(a, b)
    one, _ = kq.kq_sample(wide[:1, :V].expand(N, V), u)
    many, _ = kq.kq_sample(wide[:1, :V].repeat(N, 1), u)
    assert torch.equal(one, many)
    ids2, none = kq.kq_sample(L, u, probs=False)
    assert none is None and torch.equal(ids2, want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other, _ = kq.kq_sample(L, u, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
    ids = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kq.kq_sample(L, u, ids=ids, probs=probs)
    for _ in range(4):
        wide.normal_(0, 3), u.uniform_()
        g.replay()
        torch.cuda.synchronize()
        x, y = kq.kq_sample(L, u)
        assert torch.equal(ids, x) and torch.equal(probs, y)


def test_frequencies():
    """Tokens come up as often as their probabilities say."""
    import torch
    n = 20000
    l = torch.log(torch.tensor([0.5, 0.05, 0.25, 0.2], device="cuda"))
    u = (torch.arange(n, device="cuda") + 0.5) / n
    ids, probs = kq.kq_sample(l.expand(n, 4).contiguous(), u)
    got = torch.bincount(ids.long(), minlength=4).double() / n
    assert torch.allclose(got.cpu(), torch.tensor([0.5, 0.05, 0.25, 0.2], dtype=torch.float64), atol=2 / n)
