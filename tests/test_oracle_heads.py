"""Pins of the oracle's rotary positions, head norms and 4-bit key/value format: complex products, differences, exact
rationals, brute force over all codes."""
from fractions import Fraction

import numpy as np
import pytest

import oracle
from layer_helpers import bf16, rng


@pytest.mark.parametrize("interleaved", [False, True])
def test_turn_is_a_complex_product(interleaved):
    g = rng(1, int(interleaved))
    x, pos, f = g.standard_normal((5, 3, 24)), np.array([0, 1, 7, -3, 1000]), 10000.0 ** (-np.arange(8) / 8)
    y, _ = oracle.rope_turn(x, pos, f, interleaved, factor=1.5)
    a, b = (slice(0, 16, 2), slice(1, 16, 2)) if interleaved else (slice(0, 8), slice(8, 16))
    z = (x[..., a] + 1j * x[..., b]) * 1.5 * np.exp(1j * pos[:, None, None] * f)
    assert np.allclose(y[..., a], z.real, atol=1e-12) and np.allclose(y[..., b], z.imag, atol=1e-12)
    assert np.array_equal(y[..., 16:], x[..., 16:])
    back, _ = oracle.rope_turn(y, pos, f, interleaved, factor=1.5, back=True)
    assert np.allclose(back[..., :16], 2.25 * x[..., :16], atol=1e-12)


def test_scores_depend_on_distance_alone():
    g = rng(2)
    q, k, f = g.standard_normal((1, 1, 64)), g.standard_normal((1, 1, 64)), 10000.0 ** (-np.arange(32) / 32)
    dot = lambda m, n: (oracle.rope_turn(q, [m], f, False)[0] * oracle.rope_turn(k, [n], f, False)[0]).sum()  # noqa: E731
    assert abs(dot(17, 5) - dot(1012, 1000)) < 1e-11


@pytest.mark.parametrize("weighted", [False, True])
def test_gradients_against_differences(weighted):
    g = rng(3, int(weighted))
    x, dy, w = g.standard_normal((3, 2, 16)), g.standard_normal((3, 2, 16)), 1 + 0.1 * g.standard_normal(16)
    pos, f, eps = np.array([2, 50, 9]), 100.0 ** (-np.arange(4) / 4), 1e-3
    w = w if weighted else None
    loss = lambda x, w: (oracle.rope_fwd(x, pos, f, False, w, eps, 1.25)[0] * dy).sum()  # noqa: E731
    dx, _, dw, _ = oracle.rope_bwd(dy, pos, f, False, x, w, eps, 1.25)
    h = 1e-6
    for i in range(x.size):
        e = np.zeros(x.size)
        e[i] = h
        e = e.reshape(x.shape)
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx.flat[i]) < 1e-7
    for i in range(16 if weighted else 0):
        e = np.zeros(16)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


@pytest.mark.parametrize("name", ["nf4", "fp4", "int4"])
def test_nearest_code_by_exact_rationals(name):
    t, top, order = oracle.kv4_book(name)
    x = bf16(rng(4).standard_normal((6, 40)))
    x[0, :15] = [3, 14, 1, -1, -3, 5, -5, 7, 9, -9, 11, -11, 13, -13, 2]     # ties of INT4 at absmax 14
    x[1, :9] = [6, 0.25, -0.25, 0.75, -0.75, 2.5, -2.5, 5, -5]                 # ties of FP4 at absmax 6
    codes, absmax = oracle.kv4(x, name)
    for r in range(6):
        for i in range(40):
            a = Fraction(float(absmax[r, i // 32]))
            p = (int(codes[r, i // 32, i % 32 // 2]) >> (0 if i % 2 else 4)) & 15
            q = Fraction(float(x[r, i])) / a * Fraction(top)
            dist = [(abs(q - Fraction(float(t[c]))), t[c], c) for c in order]
            assert p == min(dist)[2], (r, i)
        assert absmax[r, 1] == np.abs(x[r, 32:]).max()
    zero = {"nf4": 0x77, "fp4": 0, "int4": 0x77}[name]
    assert np.all(codes[:, 1, 4:] == zero)     # the filling


@pytest.mark.parametrize("name", ["nf4", "fp4", "int4"])
def test_values(name):
    t, top, order = oracle.kv4_book(name)
    codes = np.array([(i * 16 + (i + 1) % 16) for i in range(16)], dtype=np.uint8).reshape(1, 1, 16)
    v = oracle.kv4_values(codes, np.array([[2.5]]), 32, name)[0]
    for i in range(16):
        for at, c in ((2 * i, i), (2 * i + 1, (i + 1) % 16)):
            assert abs(v[at] - 2.5 * t[c] / top) <= 2 ** -8 * abs(2.5 * t[c] / top) + 1e-30
    assert np.max(np.abs(v)) == 2.5
    assert np.isnan(oracle.kv4_values(codes, np.array([[np.inf]]), 32, name)).all()


def test_zero_and_lost_blocks():
    for name in ("nf4", "fp4", "int4"):
        x = np.zeros((4, 32))
        x[1, 3], x[2, 5], x[3, 0] = np.nan, np.inf, -2.0
        codes, absmax = oracle.kv4(x, name)
        zero = {"nf4": 0x77, "fp4": 0, "int4": 0x77}[name]
        assert absmax[0, 0] == 0 and np.all(codes[:3] == zero) and np.isnan(absmax[1, 0]) and np.isinf(absmax[2, 0])
        v = oracle.kv4_values(codes, absmax, 32, name)
        assert np.array_equal(v[0], np.zeros(32)) and np.isnan(v[1:3]).all() and v[3, 0] == -2.0 and not v[3, 1:].any()


def test_no_quotient_of_bf16_values_is_near_an_nf4_midpoint():
    """What lets the kernel decide by an approximate quotient: values of 8 significant bits over maxima of 8."""
    code = oracle.codebook().astype(np.float64)
    p = np.arange(1, 256, dtype=np.float64)     # 128..255 are the significands; below, subnormal ones
    r = p[:, None] / p[None, :]
    for m in np.abs(code[1:] + code[:-1]) / 2:
        assert min((np.abs(r * 2.0 ** k - m) / m).min() for k in range(-9, 9)) > 1.4e-6
