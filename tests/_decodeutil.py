"""Inputs and checks shared by the tests of the decode-step operators."""
import numpy as np

from oracle import decode_oracle as deo

U32 = 2.0 ** -24      # half a step of fp32, relative
HALF = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


def q8_rows(rng, N, K):
    """Random Q8_1 rows, uint8 [N, K/32, 36]: codes over the whole int8 range, varied scales."""
    d = np.abs(0.02 * np.exp(rng.standard_normal((N, K // 32, 1)))).astype(np.float16)
    q = rng.integers(-128, 128, (N, K // 32, 32)).astype(np.int8)
    s = (d.astype(np.float32) * q.astype(np.int32).sum(-1, keepdims=True)).astype(np.float16)
    return np.ascontiguousarray(np.concatenate([d.view(np.uint8), s.view(np.uint8), q.view(np.uint8)], -1))


def g4_weights(rng, rows, K, group, zeros):
    groups = -(-K // group)
    W = rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)
    s = (0.02 * np.exp(0.5 * rng.standard_normal((rows, groups))) * rng.choice([-1.0, 1.0], (rows, groups))).astype(np.float32)
    z = rng.integers(0, 16, (rows, groups), dtype=np.uint8) if zeros else None
    return W, s, z


def assert_g4(got, Y, B, K, what):
    """fp32 error bound for the sum over K / 32 blocks in any order: each block's exact
    integer is multiplied by two scales (3 roundings) and passes through at most
    K / 32 + 8 additions."""
    tol = (K // 32 + 12) * U32 * B + 1e-30
    err = np.abs(got.astype(np.float64) - Y)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first at {np.argwhere(bad)[0]}"


def assert_q8_blocks(Xq, v, rel, what):
    """The blocks hold Q8_1 of values within a relative error `rel` of v (fp64 [N, K])."""
    N, K = v.shape
    b = v.reshape(N, K // 32, 32)
    d_h, s_h, q = deo.unpack_q8_1(Xq)
    amax = np.abs(b).max(-1)
    d = amax / 127.0
    # d_h: fp32 error, then one rounding to fp16 (half a step is 2^-25 below fp16's normal range)
    assert np.all(np.abs(d_h - d) <= d * (2.0 ** -11 + 2 * rel + 4 * U32) + 2.0 ** -25), what
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(d[..., None] > 1e-36, b / d[..., None], 0.0)
    # A code is the integer nearest to t; t itself may be off by |t| (2 rel + 4 roundings).
    slack = np.abs(t) * (2 * rel + 4 * U32)
    live = (d > 1e-36)[..., None]
    assert np.all(np.abs(q - t)[np.broadcast_to(live, q.shape)] <= (0.5 + slack)[np.broadcast_to(live, q.shape)]), what
    want = (d_h.astype(np.float32) * q.sum(-1).astype(np.float32)).astype(np.float16).astype(np.float64)
    assert np.array_equal(s_h, want), what
