"""Refusals of the attention-side operators, on the CPU: the C ABI's argument checks (fake
addresses, none is dereferenced) and the binding's."""
import ctypes

import numpy as np
import pytest

import quantized_weight_matmul_q4_gb300 as kq
from quantized_weight_matmul_q4_gb300 import _native as nat
from quantized_weight_matmul_q4_gb300.build import build


@pytest.fixture(scope="module")
def L():
    build()
    return nat.lib()


A = 1 << 20          # 16-byte aligned
W = A + 4            # 4-byte aligned
U = A + 2
f = ctypes.c_float
NAMES = ("kq_qk_norm_rope", "kq_kv_append_q4", "kq_kv_gather_q4", "kq_attn_q4", "kq_sample")


def _rope(L, dtype=nat.KQ_F32, Q=A, ldq=256, nq=2, K=A, ldk=128, nk=1, D=128, qg=A, kg=A, eps=1e-6, cs=A, rot=64, npos=9,
          pairing=1, pos=A, out=nat.KQ_BF16, Qo=A, ldqo=256, Ko=A, ldko=128, N=3):
    return L.kq_qk_norm_rope(dtype, Q, ldq, nq, K, ldk, nk, D, qg, kg, f(eps), cs, rot, npos, pairing, pos, out, Qo, ldqo,
                             Ko, ldko, N, None)


def test_norm_rope_argument_checks(L):
    for kw in (dict(dtype=0), dict(out=5), dict(dtype=nat.KQ_F16), dict(dtype=nat.KQ_BF16, out=nat.KQ_F32), dict(pairing=0),
               dict(pairing=3)):
        assert _rope(L, **kw) == nat.KQ_ERR_TYPE, kw
    for name in ("Q", "K", "Qo", "Ko"):
        assert _rope(L, **{name: None}) == nat.KQ_ERR_NULL
    for kw in (dict(nq=0), dict(nk=-1), dict(D=0), dict(D=8), dict(D=120), dict(D=272), dict(rot=0), dict(rot=8), dict(rot=144),
               dict(rot=40), dict(npos=0), dict(N=0), dict(N=-1), dict(ldq=255), dict(ldk=127), dict(ldqo=0), dict(ldko=64),
               dict(ldq=-256), dict(eps=-1.0), dict(eps=float("nan")), dict(N=1 << 31)):
        assert _rope(L, **kw) == nat.KQ_ERR_SHAPE, kw
    for name in ("Q", "K", "Qo", "Ko", "qg", "kg", "cs"):
        assert _rope(L, **{name: W}) == nat.KQ_ERR_ALIGN, name
    assert _rope(L, pos=U) == nat.KQ_ERR_ALIGN
    # What belongs to operands that are not there is not looked at.
    assert _rope(L, nk=0, K=None, Ko=None, ldk=-3, ldko=-3, kg=U, Q=W) == nat.KQ_ERR_ALIGN
    assert _rope(L, cs=None, rot=7, npos=-1, pairing=9, Q=W) == nat.KQ_ERR_ALIGN


def _append(L, dtype=nat.KQ_F16, K=A, ldk=256, V=A, ldv=256, H=2, D=128, cs=A, rot=128, npos=9, pairing=2, pos=A, seq=A,
            table=A, ldt=4, seqs=3, cache=A, pages=8, page=16, N=3):
    return L.kq_kv_append_q4(dtype, K, ldk, V, ldv, H, D, cs, rot, npos, pairing, pos, seq, table, ldt, seqs, cache, pages,
                             page, N, None)


def _gather(L, dtype=nat.KQ_F16, K=A, ldk=256, V=A, ldv=256, H=2, D=128, pos=A, seq=A, table=A, ldt=4, seqs=3, cache=A,
            pages=8, page=16, N=3):
    return L.kq_kv_gather_q4(cache, pages, page, H, D, table, ldt, seqs, pos, seq, dtype, K, ldk, V, ldv, N, None)


def _attn(L, dtype=nat.KQ_F16, Q=A, ldq=512, Hq=4, cache=A, pages=8, page=16, H=2, D=128, table=A, ldt=4, seqs=3, kv=A,
          start=A, scale=0.1, window=0, O=A, ldo=512, Xq=A, N=7, ws=A, nbytes=1 << 40):
    return L.kq_attn_q4(dtype, Q, ldq, Hq, cache, pages, page, H, D, table, ldt, seqs, kv, start, f(scale), window, O, ldo,
                        Xq, N, ws, nbytes, None)


CACHE = (dict(H=0), dict(H=5000), dict(D=96), dict(D=32), dict(D=0), dict(page=8), dict(page=24), dict(page=0), dict(page=1 << 17),
         dict(pages=0), dict(ldt=0), dict(seqs=0), dict(N=0), dict(N=-4), dict(N=1 << 31))


@pytest.mark.parametrize("call,rows,ints", [(_append, ("K", "V"), ("pos", "seq", "table")),
                                            (_gather, ("K", "V"), ("pos", "seq", "table")),
                                            (_attn, ("Q", "O", "Xq", "ws"), ("kv", "start", "table"))])
def test_cache_argument_checks(L, call, rows, ints):
    for bad in (0, 4, -1):
        assert call(L, dtype=bad) == nat.KQ_ERR_TYPE
    for name in (*rows, "cache", "table"):
        if name not in ("O", "Xq"):
            assert call(L, **{name: None}) == nat.KQ_ERR_NULL, name
        if name != "table":
            assert call(L, **{name: W}) == nat.KQ_ERR_ALIGN, name
    for name in ints:
        assert call(L, **{name: U}) == nat.KQ_ERR_ALIGN, name
    for kw in CACHE:
        assert call(L, **kw) == nat.KQ_ERR_SHAPE, kw


def test_append_and_gather_argument_checks(L):
    for call in (_append, _gather):
        assert call(L, pos=None) == nat.KQ_ERR_NULL
        assert call(L, seq=None, N=4) == nat.KQ_ERR_SHAPE          # more tokens than sequences
        for kw in (dict(ldk=255), dict(ldv=1), dict(ldk=-1)):
            assert call(L, **kw) == nat.KQ_ERR_SHAPE, kw
    assert _gather(L, ldk=0) == nat.KQ_ERR_SHAPE
    for kw in (dict(rot=0), dict(rot=24), dict(rot=256), dict(npos=0)):
        assert _append(L, **kw) == nat.KQ_ERR_SHAPE, kw
    assert _append(L, pairing=7) == nat.KQ_ERR_TYPE
    assert _append(L, cs=W) == nat.KQ_ERR_ALIGN
    assert _append(L, cs=None, rot=3, pairing=7, K=W) == nat.KQ_ERR_ALIGN


def test_attention_argument_checks(L):
    assert _attn(L, kv=None) == nat.KQ_ERR_NULL
    assert _attn(L, O=None, Xq=None) == nat.KQ_ERR_NULL
    for kw in (dict(Hq=0), dict(Hq=3), dict(ldq=511), dict(ldo=0), dict(window=-1), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(start=None)):
        assert _attn(L, **kw) == nat.KQ_ERR_SHAPE, kw
    assert _attn(L, O=None, ldo=-1, Q=W) == nat.KQ_ERR_ALIGN


def test_attention_workspace(L):
    ws = L.kq_attn_q4_workspace_bytes
    assert ws(32, 8, 128, 4, 4) > 0
    for bad in ((32, 0, 128, 4, 4), (30, 8, 128, 4, 4), (32, 8, 96, 4, 4), (32, 8, 128, 0, 4), (32, 8, 128, 4, 0),
                (0, 8, 128, 4, 4)):
        assert ws(*bad) == 0, bad


def test_sample_argument_checks(L):
    def call(dtype=nat.KQ_F32, x=A, ld=1000, T=A, k=A, p=A, m=A, u=A, ids=A, probs=A, V=1000, N=2):
        return L.kq_sample(dtype, x, ld, T, k, p, m, u, ids, probs, V, N, None)
    assert call(dtype=9) == nat.KQ_ERR_TYPE
    for name in ("x", "u", "ids"):
        assert call(**{name: None}) == nat.KQ_ERR_NULL
    for kw in (dict(V=0), dict(V=(1 << 19) + 1, ld=1 << 20), dict(N=0), dict(ld=999), dict(ld=-1), dict(N=1 << 31)):
        assert call(**kw) == nat.KQ_ERR_SHAPE, kw
    assert call(x=W) == nat.KQ_ERR_ALIGN
    for name in ("T", "k", "p", "m", "u", "ids", "probs"):
        assert call(**{name: U}) == nat.KQ_ERR_ALIGN, name


def test_binding_refuses_cpu_tensors_and_non_tensors():
    torch = pytest.importorskip("torch")
    x, i = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32)
    cache, t = torch.zeros(*kq.kv_cache_q4_shape(2, 4, 16, 64), dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: kq.kq_qk_norm_rope(x, None),
                 lambda: kq.kq_kv_append_q4(x, x, cache, t, i),
                 lambda: kq.kq_kv_gather_q4(cache, t, i),
                 lambda: kq.kq_attn_q4(x, cache, t, i),
                 lambda: kq.kq_sample(x[0], x[0, 0]),
                 lambda: kq.kq_sample(np.zeros((2, 8), np.float32), x[0, 0]),
                 lambda: kq.kq_qk_norm_rope(x.double(), None),
                 lambda: kq.kq_attn_q4(x.int(), cache, t, i)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()


def test_names_are_exported():
    for n in NAMES:
        assert n in kq.__all__ and n in nat.header_symbols()
    assert kq.kv_cache_q4_shape(3, 8, 64, 128) == (3, 8, 4, 2560)
