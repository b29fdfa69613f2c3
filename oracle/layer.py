"""What runs around the adapted linears, in float64: attention with its gradients, the residual norm
with its gradients, and the 8-bit activation format. TEST INFRASTRUCTURE ONLY.

Written from the formulas, sequence by sequence and head by head. The ``*_terms`` results are the sums
of the absolute values of the same terms, which the rounding-error bounds of the tests are made of.
"""
from __future__ import annotations

import numpy as np


def visible(nq: int, nk: int, causal: bool, window: int) -> np.ndarray:
    """[nq, nk] truth values: query i at position nk - nq + i sees key j."""
    p = np.arange(nq)[:, None] + (nk - nq)
    j = np.arange(nk)[None, :]
    see = np.ones((nq, nk), dtype=bool)
    if causal:
        see &= j <= p
    if window:
        see &= j > p - window
    return see


def attention_head(q, k, v, scale: float, see):
    """One head of one sequence: o [nq, d], lse [nq], P [nq, nk]; a row that sees nothing gives 0, -inf."""
    z = np.where(see, scale * (q @ k.T), -np.inf)
    top = z.max(axis=1, initial=-np.inf)
    e = np.exp(z - np.where(np.isinf(top), 0.0, top)[:, None])
    total = e.sum(axis=1)
    with np.errstate(divide="ignore"):
        lse = np.where(np.isinf(top), 0.0, top) + np.log(total)
    P = e / np.where(total > 0, total, 1.0)[:, None]
    return P @ v, lse, P


def attention(q, k, v, seqs, scale: float, causal: bool, window: int, do=None):
    """Attention of [tokens, heads, d] arrays over sequences (q0, nq, k0, nk), query heads sharing key
    heads in turn. Returns a dict of o, lse [heads, tokens], o_terms and, given do, dq, dk, dv and their
    *_terms; rows outside every sequence stay 0 (lse too)."""
    T, H, d = q.shape
    G = H // k.shape[1]
    out = {"o": np.zeros((T, H, d)), "o_terms": np.zeros((T, H, d)), "lse": np.zeros((H, T))}
    if do is not None:
        for n, like in (("dq", q), ("dk", k), ("dv", k)):
            out[n], out[n + "_terms"] = np.zeros(like.shape), np.zeros(like.shape)
    for q0, nq, k0, nk in seqs:
        see = visible(nq, nk, causal, window)
        a, b = slice(q0, q0 + nq), slice(k0, k0 + nk)
        for h in range(H):
            g = h // G
            o, lse, P = attention_head(q[a, h], k[b, g], v[b, g], scale, see)
            out["o"][a, h], out["lse"][h, a] = o, lse
            out["o_terms"][a, h] = P @ np.abs(v[b, g])
            if do is None:
                continue
            dp = do[a, h] @ v[b, g].T
            delta = (do[a, h] * o).sum(axis=1, keepdims=True)
            ds = P * (dp - delta)
            mag = P * (np.abs(dp) + (np.abs(do[a, h]) * np.abs(o)).sum(axis=1, keepdims=True))
            out["dq"][a, h] = scale * (ds @ k[b, g])
            out["dk"][b, g] += scale * (ds.T @ q[a, h])
            out["dv"][b, g] += P.T @ do[a, h]
            out["dq_terms"][a, h] = scale * (mag @ np.abs(k[b, g]))
            out["dk_terms"][b, g] += scale * (mag.T @ np.abs(q[a, h]))
            out["dv_terms"][b, g] += P.T @ np.abs(do[a, h])
    return out


def rmsnorm(x, residual, w, eps: float):
    """h = x + residual, rstd per row, y = h rstd w (all float64)."""
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h, h * rstd[:, None] * w, rstd


def rmsnorm_bwd(dy, dh, h, w, rstd):
    """dx and dw of the norm at a given h and rstd, with their *_terms."""
    n = h * rstd[:, None]
    wd = dy * w
    dx = rstd[:, None] * (wd - n * (wd * n).mean(axis=1, keepdims=True))
    terms = rstd[:, None] * (np.abs(wd) + np.abs(n) * np.abs(wd * n).mean(axis=1, keepdims=True))
    if dh is not None:
        dx, terms = dx + dh, terms + np.abs(dh)
    return dx, (dy * n).sum(axis=0), terms, np.abs(dy * n).sum(axis=0)


def act8(x):
    """8-bit codes (int8) and block maxima of [M, K] values that bf16 holds: absmax over blocks of 64,
    codes the integers nearest to 127 x / absmax, ties to even. The float64 quotient decides rightly: a
    quotient of bf16 values times 127 is a tie (which float64 holds) or further than 2^-20 from one. A block
    with a NaN or an infinity has that as its maximum and codes 0."""
    b = np.asarray(x, dtype=np.float64).reshape(x.shape[0], -1, 64)
    a = np.abs(b).max(axis=2)
    b = np.where(np.isfinite(a)[:, :, None], b, 0.0)
    codes = np.rint(127.0 * b / np.where((a > 0) & np.isfinite(a), a, 1.0)[:, :, None])
    return codes.astype(np.int8).reshape(x.shape), a


def act8_values(codes, absmax):
    """The values codes stand for: code * absmax / 127."""
    with np.errstate(invalid="ignore"):   # 0 times infinity: NaN
        return codes.astype(np.float64) * np.repeat(absmax, 64, axis=1) / 127.0
