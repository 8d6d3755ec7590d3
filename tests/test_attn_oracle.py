"""The oracle of the attention-side operators against closed forms and brute force. CPU only."""
import numpy as np
import pytest

from _attnutil import page_table, random_cache, table
from oracle import attn_oracle as ao


@pytest.mark.parametrize("pairing", ["half", "pairs"])
def test_rotation_is_a_rotation(pairing):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 48))
    cs = table(5, 32)
    y, _ = ao.norm_rope(x, None, 0.0, cs, pairing)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-6)     # the table is fp32
    assert np.array_equal(y[..., 32:], x[..., 32:])
    assert np.array_equal(y[0], x[0])                                     # position 0 turns nothing
    a, b = ao.rope_pairs(32, pairing)
    back, _ = ao.norm_rope(y, None, 0.0, np.concatenate([cs[:, :16], -cs[:, 16:]], 1), pairing)
    assert np.allclose(back, x, atol=1e-6)
    z = (x[1, 0, a[3]] + 1j * x[1, 0, b[3]]) * np.exp(1j * 10000.0 ** (-6 / 32))
    assert np.allclose([y[1, 0, a[3]], y[1, 0, b[3]]], [z.real, z.imag], atol=1e-6)


def test_products_depend_on_the_distance_of_positions():
    rng = np.random.default_rng(1)
    q, k, cs = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32)), table(200, 32)
    at = lambda x, p: ao.norm_rope(x, None, 0.0, cs[p:p + 1], "half")[0][0, 0]  # noqa: E731
    assert abs(at(q, 150) @ at(k, 140) - at(q, 60) @ at(k, 50)) < 1e-5


def test_norm_closed_form():
    x = np.array([[[3.0, 4.0] * 8]])
    y, _ = ao.norm_rope(x, np.full(16, 2.0), 0.0, None, "half")
    assert np.allclose(y, 2 * x / np.sqrt(12.5))


def test_blocks_by_hand():
    v = np.arange(32, dtype=np.float32)
    s, m, c = ao.blocks4(v)
    assert float(m) == 0.0 and float(s) == float(np.float16(np.float32(31) * np.float32(1 / 15)))
    assert c.tolist() == [min(15, int(np.rint(np.float32(i) / np.float32(s)))) for i in range(32)]
    s, m, c = ao.blocks4(np.full(32, 1.5, np.float32))
    assert (float(s), float(m)) == (0.0, 1.5) and not c.any()
    for bad in (np.inf, -np.inf, np.nan, 2e6, -70000.0):
        v[5] = bad
        s, m, c = ao.blocks4(v)
        assert np.isnan(s) and m == 0 and not c.any(), bad


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("values", [0, 1])
def test_codes_fill_a_row_once(D, values):
    byte, high = ao.code_bytes(D, values)
    assert sorted(2 * byte + high) == list(range(D))


@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (256, 16)])
def test_append_then_read(D, P):
    rng = np.random.default_rng(D)
    H, lens = 2, [P + 3, 0, 5]
    pages, t = page_table(rng, lens, P)
    cache = random_cache(rng, pages, H, P, D)
    seq = np.repeat(np.arange(3), lens)
    pos = np.concatenate([np.arange(n) for n in lens])
    K, V = (rng.standard_normal((len(seq), H, D)).astype(np.float32) for _ in range(2))
    ao.append(cache, t, P, K, V, pos, seq)
    for b, n in enumerate(lens):
        for x, (s, m, c) in zip((K, V), ao.read(cache, t[b], P, np.arange(n))):
            got = (m[..., None] + s[..., None] * c).reshape(n, H, D)
            step = np.repeat(s, 32, -1)
            # Half a step, the rounding of s over 15 steps, and that of m.
            assert np.all(np.abs(got - x[seq == b]) <= step * (0.5 + 15 * 2.0 ** -11) + 2.0 ** -11 * np.abs(np.repeat(m, 32, -1)) + 1e-7)


def test_attention_against_brute_force():
    rng = np.random.default_rng(3)
    D, H, Hq, P, L, n = 64, 2, 6, 16, 21, 3
    pages, t = page_table(rng, [L], P)
    cache = random_cache(rng, pages, H, P, D)
    Q = rng.standard_normal((n, Hq, D))
    (ks, km, kc), (vs, vm, vc) = ao.read(cache, t[0], P, np.arange(L))
    o, _, _ = ao.attention(Q, cache, t, P, [L], q_start=[0, n], window=5)
    for i in range(n):
        for h in range(Hq):
            num, den = np.zeros(D), 0.0
            for p in range(L):
                if p <= L - n + i and p > L - n + i - 5:
                    k = (km[p, h // 3][:, None] + ks[p, h // 3][:, None] * kc[p, h // 3]).reshape(D)
                    v = (vm[p, h // 3][:, None] + vs[p, h // 3][:, None] * vc[p, h // 3]).reshape(D)
                    e = np.exp(k @ Q[i, h] / 8.0)
                    num, den = num + e * v, den + e
            assert np.allclose(o[i, h], num / den, rtol=1e-12)
    o, _, _ = ao.attention(Q[:1], cache, t, P, [0])
    assert not o.any()


def test_sample_by_hand():
    l = np.log(np.array([[0.1, 0.4, 0.2, 0.3]]))
    for u, want in ((0.0, 0), (0.09, 0), (0.11, 1), (0.51, 2), (0.69, 2), (0.71, 3), (0.999, 3)):
        assert ao.sample(l, [u])[0][0] == want
    assert ao.sample(l, [0.0], top_k=[2])[0][0] == 1 and ao.sample(l, [0.58], top_k=[2])[0][0] == 3    # 4/7
    ids, probs = ao.sample(l, [0.99], top_p=[0.69])
    assert ids[0] == 3 and np.isclose(probs[0], 3 / 7)
    ids, probs = ao.sample(l, [0.99], top_p=[0.71])            # 1, 3 and 2
    assert ids[0] == 3 and np.isclose(probs[0], 3 / 9)
    ids, probs = ao.sample(l, [0.3], min_p=[0.6])              # 1 and 3
    assert ids[0] == 1 and np.isclose(probs[0], 4 / 7)
    assert ao.sample(l, [0.5], temperature=[0.0])[0][0] == 1
    ids, probs = ao.sample(l, [0.5], temperature=[0.5])        # the squares: 1, 16, 4, 9 of 30
    assert ids[0] == 1 and np.isclose(probs[0], 16 / 30)
    ids, probs = ao.sample(np.array([[1.0, np.nan, 2.0, 2.0], [-np.inf] * 4]), [0.0, 0.5], top_k=[1, 1])
    assert ids.tolist() == [2, 0] and probs.tolist() == [1.0, 0.0]
