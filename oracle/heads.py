"""What runs between a layer's projections and its attention, in float64: rotary positions and norms of the query
and key heads with their gradients, and the 4-bit key/value format. TEST INFRASTRUCTURE ONLY.

Written from the formulas. The ``*_terms`` results are the sums of the absolute values of the same terms, which the
rounding-error bounds of the tests are made of."""
from __future__ import annotations

import numpy as np

from .nf4 import bf16_bits_from_f32, codebook, f32_from_bf16_bits


def rope_turn(x, positions, inv_freq, interleaved: bool, factor: float = 1.0, back: bool = False):
    """The first 2 len(inv_freq) features of rows [tokens, heads, d] turned by position * inv_freq, or back (the
    transpose). The angle is reduced in extended precision. Returns the result and its terms."""
    x = np.asarray(x, dtype=np.float64)
    half = len(inv_freq)
    turn = 2 * np.longdouble("3.14159265358979323846264338327950288")
    angle = np.asarray(positions).astype(np.longdouble)[:, None] * np.asarray(inv_freq, dtype=np.float64).astype(np.longdouble)
    angle = np.fmod(angle, turn).astype(np.float64)[:, None, :]
    c, s = factor * np.cos(angle), factor * np.sin(angle) * (-1.0 if back else 1.0)
    a, b = (np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if interleaved else (np.arange(half), np.arange(half, 2 * half))
    y, terms = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    both = abs(factor) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    terms[..., a], terms[..., b] = both, both
    return y, terms


def head_norm(x, w, eps: float):
    """n = x rsqrt(mean(x^2) + eps) over the last dimension, rstd, and n w."""
    rstd = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    return x * rstd, rstd, x * rstd * w


def rope_fwd(x, positions, inv_freq, interleaved, w=None, eps=0.0, factor=1.0):
    z = x if w is None else head_norm(x, w, eps)[2]
    return rope_turn(z, positions, inv_freq, interleaved, factor)


def rope_bwd(dy, positions, inv_freq, interleaved, x=None, w=None, eps=0.0, factor=1.0):
    """dx, its terms, dw and its terms (None without a weight)."""
    g, mag = rope_turn(dy, positions, inv_freq, interleaved, factor, back=True)
    if w is None:
        return g, mag, None, None
    n, rstd, _ = head_norm(x, w, eps)
    wg, wm = w * g, np.abs(w) * mag
    dx = rstd * (wg - n * (wg * n).mean(axis=-1, keepdims=True))
    terms = rstd * (wm + np.abs(n) * (wm * np.abs(n)).mean(axis=-1, keepdims=True))
    return dx, terms, (g * n).sum(axis=(0, 1)), (mag * np.abs(n)).sum(axis=(0, 1))


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def kv4_book(name: str):
    """The value of each nibble, the largest, and the nibbles in the order of their values (-0 left out)."""
    if name == "nf4":
        return codebook().astype(np.float64), 1.0, np.arange(16)
    if name == "int4":
        return np.minimum(np.arange(16) - 7, 7).astype(np.float64), 7.0, np.arange(15)
    return np.concatenate([E2M1, -E2M1]), 6.0, np.array([15, 14, 13, 12, 11, 10, 9, 0, 1, 2, 3, 4, 5, 6, 7])


def kv4(x, name: str):
    """4-bit blocks of [..., d] values that bf16 holds: codes uint8 [..., blocks, 16] and absmax [..., blocks]. Every
    comparison is exact in float64: 8 significant bits against 8 times the at most 25 of a midpoint."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    nb = -(-d // 32)
    b = np.zeros(x.shape[:-1] + (nb * 32,))
    b[..., :d] = x
    b = b.reshape(x.shape[:-1] + (nb, 32))
    a = np.abs(b).max(axis=-1)
    t, top, order = kv4_book(name)
    v = t[order]
    fine = np.isfinite(a)[..., None]
    bb, aa = np.where(fine, b, 0.0), np.where(fine, a[..., None], 0.0)
    at = np.zeros(b.shape, dtype=np.int64)
    for i in range(len(v) - 1):     # a tie takes the lower value
        at += top * bb > (v[i] + v[i + 1]) / 2 * aa
    at = np.where(aa == 0, int(np.flatnonzero(v == 0)[0]), at)
    p = order[at]
    return (p[..., 0::2] * 16 + p[..., 1::2]).astype(np.uint8), a


def kv4_values(codes, absmax, d: int, name: str):
    """The bf16 values that blocks stand for."""
    t, top, _ = kv4_book(name)
    with np.errstate(invalid="ignore", over="ignore"):
        step = absmax.astype(np.float32) * np.float32(1.0 / top)
        p = np.stack([codes >> 4, codes & 15], axis=-1).reshape(codes.shape[:-1] + (32,))
        v = t.astype(np.float32)[p] * step[..., None]
    lost = ~np.isfinite(absmax)
    bits = bf16_bits_from_f32(np.where(lost[..., None], np.float32(0), v))
    v = np.where(lost[..., None], np.nan, f32_from_bf16_bits(bits).astype(np.float64))
    return v.reshape(codes.shape[:-2] + (-1,))[..., :d]
