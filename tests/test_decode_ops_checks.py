"""Refusals of the decode-step operators, on the CPU: the C ABI's argument checks
(fake addresses, none is dereferenced) and the binding's."""
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
U = A + 4            # misaligned
f = ctypes.c_float


def _norm(L, dtype=nat.KQ_F32, X=A, ldx=64, R=A, ldr=64, gamma=A, eps=1e-5, H=A, ldh=64, Y=A, ldy=64, Xq=A, K=64, N=2):
    return L.kq_add_rmsnorm_q8_1(dtype, X, ldx, R, ldr, gamma, f(eps), H, ldh, Y, ldy, Xq, K, N, None)


def test_add_rmsnorm_argument_checks(L):
    for bad in (0, 4, -1):
        assert _norm(L, dtype=bad) == nat.KQ_ERR_TYPE
    for name in ("X", "gamma", "Xq"):
        assert _norm(L, **{name: None}) == nat.KQ_ERR_NULL
    for kw in (dict(K=48), dict(K=0), dict(N=0), dict(N=-1), dict(ldx=63), dict(ldx=-64), dict(ldr=1), dict(ldh=0),
               dict(ldy=32), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(K=1 << 31),
               dict(ldx=1 << 31)):
        assert _norm(L, **kw) == nat.KQ_ERR_SHAPE, kw
    for name in ("X", "R", "gamma", "H", "Y", "Xq"):
        assert _norm(L, **{name: U}) == nat.KQ_ERR_ALIGN
    # A stride of an operand that is not there is not looked at.
    assert _norm(L, R=None, ldr=-5, X=U) == nat.KQ_ERR_ALIGN


def test_swiglu_argument_checks(L):
    def call(dtype=nat.KQ_F16, g=A, ldg=64, u=A, ldu=64, Xq=A, K=64, N=2):
        return L.kq_swiglu_q8_1(dtype, g, ldg, u, ldu, Xq, K, N, None)
    assert call(dtype=7) == nat.KQ_ERR_TYPE
    for name in ("g", "u", "Xq"):
        assert call(**{name: None}) == nat.KQ_ERR_NULL
        assert call(**{name: U}) == nat.KQ_ERR_ALIGN
    for kw in (dict(K=33), dict(N=0), dict(ldg=32), dict(ldu=-1), dict(K=-32)):
        assert call(**kw) == nat.KQ_ERR_SHAPE, kw


def test_route_argument_checks(L):
    def call(dtype=nat.KQ_BF16, x=A, ld=64, bias=A, score=1, ng=4, kg=2, gt=2, k=8, scale=1.0, ids=A, probs=A, E=64, T=3):
        return L.kq_moe_route(dtype, x, ld, bias, score, ng, kg, gt, k, 1, f(scale), ids, probs, E, T, None)
    assert call(dtype=0) == nat.KQ_ERR_TYPE
    assert call(score=3) == nat.KQ_ERR_TYPE
    for name in ("x", "ids", "probs"):
        assert call(**{name: None}) == nat.KQ_ERR_NULL
    for name in ("x", "bias", "ids", "probs"):
        assert call(**{name: U}) == nat.KQ_ERR_ALIGN
    for kw in (dict(E=0), dict(E=513, ng=1, kg=1), dict(T=0), dict(ng=0), dict(ng=5), dict(kg=0), dict(kg=5), dict(gt=0),
               dict(gt=3), dict(k=0), dict(k=33), dict(ld=63), dict(ld=-1), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert call(**kw) == nat.KQ_ERR_SHAPE, kw


def _g4(L, W=A, s=A, sd=nat.KQ_F16, z=A, group=128, Xq=A, Y=A, M=16, K=256, N=1):
    return L.kq_matvec_g4(W, s, sd, z, group, Xq, Y, M, K, N, None)


def _moe(L, W=A, s=A, sd=nat.KQ_F16, z=A, group=128, E=8, ids=A, k=2, Xq=A, Y=A, M=16, K=256, N=1):
    return L.kq_moe_matvec_g4(W, s, sd, z, group, E, ids, k, 0, Xq, Y, M, K, N, None)


@pytest.mark.parametrize("call", [_g4, _moe])
def test_g4_argument_checks(L, call):
    for sd in (nat.KQ_F32, 0, 9):
        assert call(L, sd=sd) == nat.KQ_ERR_TYPE
    for name in ("W", "s", "Xq", "Y"):
        assert call(L, **{name: None}) == nat.KQ_ERR_NULL
    for name in ("W", "s", "z", "Xq", "Y"):
        assert call(L, **{name: U}) == nat.KQ_ERR_ALIGN
    for kw in (dict(M=0), dict(K=0), dict(K=40), dict(N=0), dict(group=16), dict(group=96), dict(group=0),
               dict(group=-32), dict(M=1 << 31), dict(K=1 << 31), dict(N=1 << 31)):
        assert call(L, **kw) == nat.KQ_ERR_SHAPE, kw


def test_moe_g4_argument_checks(L):
    assert _moe(L, ids=None) == nat.KQ_ERR_NULL
    assert _moe(L, ids=U) == nat.KQ_ERR_ALIGN
    for kw in (dict(E=0), dict(E=513), dict(k=0), dict(k=9), dict(M=1 << 30)):
        assert _moe(L, **kw) == nat.KQ_ERR_SHAPE, kw


def test_binding_refuses_cpu_tensors_and_non_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64)
    u8 = torch.zeros(2, 2, 36, dtype=torch.uint8)
    for call in (lambda: kq.kq_add_rmsnorm_q8_1(x, None, torch.ones(64), 1e-5),
                 lambda: kq.kq_swiglu_q8_1(x, x),
                 lambda: kq.kq_moe_route(x, 2),
                 lambda: kq.kq_matvec_g4(u8, x.half(), u8, 16, 64, 64),
                 lambda: kq.kq_moe_matvec_g4(u8, x.half(), 1, u8, u8, 16, 64, 64),
                 lambda: kq.kq_moe_route(np.zeros((2, 64), np.float32), 2),
                 lambda: kq.kq_add_rmsnorm_q8_1(x.double(), None, x[0], 1e-5),
                 lambda: kq.kq_swiglu_q8_1(x.int(), x)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()


def test_names_are_exported():
    for n in ("kq_add_rmsnorm_q8_1", "kq_swiglu_q8_1", "kq_moe_route", "kq_matvec_g4", "kq_moe_matvec_g4"):
        assert n in kq.__all__ and n in nat.header_symbols()
