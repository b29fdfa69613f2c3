"""The oracle of attention, the residual norm and the 8-bit activation format, against closed forms,
finite differences and exact rationals."""
from fractions import Fraction

import numpy as np
import pytest

import oracle


def _rng(*key):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence(entropy=7, spawn_key=key)))


def _bf16(a):
    return oracle.f32_from_bf16_bits(oracle.bf16_bits_from_f32(np.asarray(a, dtype=np.float32))).astype(np.float64)


def test_attention_closed_forms():
    g = _rng(1)
    v = g.standard_normal((5, 3))
    see = oracle.visible(2, 5, False, 0)
    # equal scores: the mean of the values, lse = ln n
    o, lse, P = oracle.attention_head(np.zeros((2, 3)), g.standard_normal((5, 3)), v, 0.7, see)
    assert np.allclose(o, v.mean(axis=0)) and np.allclose(lse, np.log(5)) and np.allclose(P, 0.2)
    # causal with as many queries as keys: the first query sees one key
    o, lse, _ = oracle.attention_head(g.standard_normal((5, 3)), v, v, 1.0, oracle.visible(5, 5, True, 0))
    assert np.allclose(o[0], v[0])
    # more queries than keys: the first rows see nothing
    see = oracle.visible(5, 2, True, 0)
    assert see.sum(axis=1).tolist() == [0, 0, 0, 1, 2]
    o, lse, _ = oracle.attention_head(g.standard_normal((5, 3)), v[:2], v[:2], 1.0, see)
    assert np.all(o[:3] == 0) and np.all(np.isneginf(lse[:3])) and np.all(np.isfinite(lse[3:]))
    # a window of w keys, the own one among them
    assert oracle.visible(6, 6, True, 2).sum(axis=1).tolist() == [1, 2, 2, 2, 2, 2]


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3)])
def test_attention_gradients_against_differences(causal, window):
    g = _rng(2, int(causal), window)
    seqs = [(0, 4, 0, 6), (4, 3, 6, 2), (7, 1, 8, 1)]
    q, k, v = g.standard_normal((8, 4, 5)), g.standard_normal((9, 2, 5)), g.standard_normal((9, 2, 5))
    do = g.standard_normal(q.shape)
    f = lambda a, b, c: (oracle.attention(a, b, c, seqs, 0.4, causal, window)["o"] * do).sum()  # noqa: E731
    r = oracle.attention(q, k, v, seqs, 0.4, causal, window, do=do)
    e = 1e-6
    for name, x, at in (("dq", q, 0), ("dk", k, 1), ("dv", v, 2)):
        for _ in range(12):
            i = tuple(int(g.integers(n)) for n in x.shape)
            hi, lo = [q, k, v], [q, k, v]
            hi[at], lo[at] = x.copy(), x.copy()
            hi[at][i] += e
            lo[at][i] -= e
            assert abs((f(*hi) - f(*lo)) / (2 * e) - r[name][i]) < 1e-7, (name, i)
        assert np.all(r[name + "_terms"] >= np.abs(r[name]) - 1e-12)


@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_gradients_against_differences(residual):
    g = _rng(3, int(residual))
    x, w = g.standard_normal((3, 16)), 1 + 0.2 * g.standard_normal(16)
    res = g.standard_normal((3, 16)) if residual else None
    dy, dh = g.standard_normal((3, 16)), g.standard_normal((3, 16))

    def f(x_, w_):
        h, y, _ = oracle.rmsnorm(x_, res, w_, 1e-5)
        return (y * dy).sum() + (h * dh).sum()
    h, y, rstd = oracle.rmsnorm(x, res, w, 1e-5)
    assert np.allclose((y / w * (y / w)).mean(axis=1), 1.0, atol=1e-4)
    dx, dw, terms, _ = oracle.rmsnorm_bwd(dy, dh, h, w, rstd)
    assert np.all(terms >= np.abs(dx) - 1e-12)
    e = 1e-6
    for _ in range(20):
        i = (int(g.integers(3)), int(g.integers(16)))
        up, dn = x.copy(), x.copy()
        up[i] += e
        dn[i] -= e
        assert abs((f(up, w) - f(dn, w)) / (2 * e) - dx[i]) < 1e-7
        up, dn = w.copy(), w.copy()
        up[i[1]] += e
        dn[i[1]] -= e
        assert abs((f(x, up) - f(x, dn)) / (2 * e) - dw[i[1]]) < 1e-7


def test_act8_against_exact_rationals():
    g = _rng(4)
    x = _bf16(g.standard_normal((6, 128)) * np.exp(3 * g.standard_normal((6, 1))))
    x[1, :64] = 0.0
    x[2, 3] = 4096.0                              # a value that stands out
    x[3, :64] = _bf16(np.arange(64) / 64.0)
    x[4, :64] = np.tile([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 63.5, -126.5], 8)   # absmax 127: exact ties
    codes, a = oracle.act8(x)
    assert codes[4, :8].tolist() == [127, 0, 2, 2, 0, -2, 64, -126]
    for m in range(6):
        for c in range(128):
            top = Fraction(float(a[m, c // 64]))
            if top == 0:
                assert codes[m, c] == 0
                continue
            r = 127 * Fraction(float(x[m, c])) / top
            assert codes[m, c] == round(r), (m, c)   # Fraction rounds ties to even
    assert np.all(np.abs(oracle.act8_values(codes, a) - x) <= np.repeat(a, 64, axis=1) / 254 * (1 + 1e-12))
