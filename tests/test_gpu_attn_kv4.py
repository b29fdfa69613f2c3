"""Attention over a 4-bit cache against the float64 oracle over the values that the cache stands for.

Bounds (element by element; U = 2^-8 is bf16's unit roundoff): the values are bf16 numbers, exact operands; every
probability is rounded once (relative U) and the result once: U |o| + (U + E) sum_j P |v|, with E = 1e-4 for fp32
scores, sums and the hardware exponential (arguments below 50 in magnitude: 50 * 2^-24 * 8). lse is fp32:
2e-5 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import U, bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu
E = 1e-4
BOOKS = ["nf4", "fp4", "int4"]


def _cache(codes, absmax, d, book, layout="heads"):
    import bit_nf4_quantised_amd as nf4
    c, a = torch.from_numpy(codes).to("cuda:0"), dev(absmax)
    if layout == "heads":
        c, a = c.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3), a.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    return nf4.Kv4(c, a, d, book)


def _run(name, seqs, heads, kv, d, book="nf4", causal=True, window=0, tq=None, tk=None, scale=None, std=1.5, layout="heads",
         spoil=None, vstd=1.0):
    import bit_nf4_quantised_amd as nf4
    log(f"[attn kv4] {name}: seqs={seqs[:8]}{'...' if len(seqs) > 8 else ''} heads={heads}/{kv} d={d} {book} causal={causal} window={window} {layout}")
    tq = max([s[0] + s[1] for s in seqs], default=0) if tq is None else tq
    tk = max([s[2] + s[3] for s in seqs], default=0) if tk is None else tk
    g = rng(len(seqs), heads, kv, d, int(causal), window, tq, tk)
    q = bf16(std * g.standard_normal((tq, heads, d)))
    k, v = bf16(g.standard_normal((tk, kv, d))), bf16(vstd * g.standard_normal((tk, kv, d)))
    kc, ka = oracle.kv4(k, book)
    vc, va = oracle.kv4(v, book)
    kd, vd = oracle.kv4_values(kc, ka, d, book), oracle.kv4_values(vc, va, d, book)
    scale = d ** -0.5 if scale is None else scale
    want = oracle.attention(q, kd, vd, seqs, scale, causal, window)
    seen, rows = np.zeros(tk, bool), np.zeros(tq, bool)
    for q0, nq, k0, nk in seqs:
        rows[q0:q0 + nq] = True
        seen[k0:k0 + nk] |= oracle.visible(nq, nk, causal, window).any(axis=0) if nq else False
    if spoil:       # what no query sees may hold anything
        for a in (ka, va):
            a[~seen] = spoil
    q[~rows] = np.nan
    K4, V4 = _cache(kc, ka, d, book, layout), _cache(vc, va, d, book, layout)

    def place(a):
        t = dev(a)
        if layout == "tokens":      # a slice of a wider row
            wide = torch.full((a.shape[0], a.shape[1] + 3, d + 8), 7.0, dtype=t.dtype, device=t.device)
            wide[:, 1:1 + a.shape[1], :d] = t
            return wide[:, 1:1 + a.shape[1], :d]
        return t
    Q, O = place(q), place(np.full(q.shape, 3.0))
    lse = torch.full((heads, tq), 5.0, dtype=torch.float32, device="cuda:0")
    nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs(seqs, causal=causal, window=window), Q, K4, V4, O, lse, scale=scale)
    torch.cuda.synchronize()
    assert np.all(host(O)[~rows] == 3.0) and np.all(host(lse)[:, ~rows] == 5.0), "a row outside the sequences was written"
    within("o", host(O)[rows], want["o"][rows], (U * np.abs(want["o"]) + (U + E) * want["o_terms"])[rows])
    within("lse", host(lse)[:, rows], want["lse"][:, rows], 2e-5 * (1 + np.abs(np.where(np.isfinite(want["lse"]), want["lse"], 0)))[:, rows])


def _caches(nq, *nk, room=None):
    room = max(nk) if room is None else room
    return [(i * nq, nq, i * room, n) for i, n in enumerate(nk)]


@pytest.mark.parametrize("book", BOOKS)
@pytest.mark.parametrize("nk", [1, 2, 31, 32, 33, 127, 128, 129, 300, 1025])
def test_one_token(nk, book):
    _run("one token", _caches(1, nk), 8, 2, 128, book)
    _run("one token", _caches(1, nk), 4, 4, 64, book)


@pytest.mark.parametrize("d", [8, 24, 32, 40, 72, 80, 96, 104, 120])
@pytest.mark.parametrize("book", BOOKS)
def test_head_sizes(d, book):
    _run("head size", _caches(1, 70, 3), 2, 1, d, book)
    _run("head size", _caches(9, 70, 40), 3, 3, d, book)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (6, 2), (8, 8), (64, 8), (12, 1), (33, 1), (40, 8)])
def test_shared_heads(heads, kv):
    _run("heads", _caches(1, 97, 240), heads, kv, 64)
    _run("heads", _caches(3, 97, 240), heads, kv, 128)


@pytest.mark.parametrize("book", BOOKS)
def test_ragged_batch(book):
    _run("ragged", _caches(1, 1000, 1, 33, 640, 255, 7, 2048, 64), 16, 4, 128, book)


@pytest.mark.parametrize("nq", [2, 5, 16, 33, 100, 200])
@pytest.mark.parametrize("d", [64, 128])
def test_several_tokens(nq, d):
    _run("several", _caches(nq, 300, nq, nq + 31), 8, 2, d, "fp4")
    _run("several", _caches(nq, 700, 260), 4, 4, d, "nf4")


@pytest.mark.parametrize("window", [1, 2, 31, 32, 64, 65, 200, 1 << 40])
def test_window(window):
    _run("window", _caches(1, 700, 40), 4, 2, 128, window=window, spoil=np.nan)
    _run("window", _caches(40, 260, 47), 4, 2, 64, "int4", window=window, spoil=np.nan)


def test_not_causal():
    _run("not causal", _caches(5, 129, 64, 4), 4, 4, 64, causal=False)
    _run("not causal", [(0, 70, 0, 33), (70, 3, 33, 200)], 4, 2, 128, causal=False, window=50)


def test_rows_that_see_nothing():
    _run("empty rows", [(0, 200, 0, 60), (200, 40, 60, 0), (240, 0, 60, 50), (240, 70, 110, 1)], 4, 2, 64)
    _run("empty rows", [(0, 5, 0, 2), (5, 1, 2, 0)], 4, 1, 128)
    _run("nothing at all", [], 2, 1, 64, tq=4, tk=4)


@pytest.mark.parametrize("spoil", [np.nan, np.inf])
def test_what_no_query_sees_may_hold_anything(spoil):
    _run("gaps", [(1, 1, 7, 300), (3, 1, 400, 33), (4, 20, 450, 40)], 8, 2, 128, tq=30, tk=500, spoil=spoil)
    _run("shared keys", [(0, 4, 0, 100), (4, 4, 0, 90), (8, 1, 50, 60)], 2, 1, 64, tk=130, spoil=spoil)


def test_token_major_cache():
    _run("token-major", _caches(1, 300, 20), 8, 4, 128, layout="tokens")
    _run("token-major", _caches(30, 300, 50), 8, 4, 80, "fp4", layout="tokens")


@pytest.mark.parametrize("vstd", [1e-30, 1e30])
def test_magnitudes(vstd):
    _run("magnitudes", _caches(2, 300), 4, 2, 128, "fp4", vstd=vstd)


@pytest.mark.parametrize("std", [0.0, 1e-20, 12.0])
def test_scores(std):
    """Equal scores, and scores of tens: exp's argument reaches 12 * 11.3 / 11.3 * 4 = 50."""
    _run("scores", _caches(2, 600), 4, 2, 128, std=std)


def test_more_sequences_than_a_launch_holds():
    _run("many", [(i, 1, 20 * i, 1 + i % 20) for i in range(150)], 2, 1, 64)


def test_nan_reaches_the_queries_that_see_it_and_no_other():
    import bit_nf4_quantised_amd as nf4
    g = rng(77)
    nq, nk, heads, kv, d = 40, 300, 4, 2, 128
    q = bf16(g.standard_normal((nq, heads, d)))
    for book in BOOKS:
        for which, bad in (("k", np.nan), ("v", np.nan), ("v", np.inf), ("k", -np.inf)):
            x = {n: bf16(g.standard_normal((nk, kv, d))) for n in ("k", "v")}
            clean = {n: oracle.kv4_values(*oracle.kv4(x[n], book), d, book) for n in x}
            want = oracle.attention(q, clean["k"], clean["v"], [(0, nq, 0, nk)], d ** -0.5, True, 0)
            at = nk - nq + 25           # seen by queries 25 .. 39, of key head 1 alone
            x[which][at, 1, 70] = bad
            caches = [_cache(*oracle.kv4(x[n], book), d, book) for n in ("k", "v")]
            O, lse = dev(np.zeros(q.shape)), torch.zeros(heads, nq, device="cuda:0")
            nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs([(0, nq, 0, nk)]), dev(q), *caches, O, lse)
            o, l = host(O), host(lse)
            assert np.isnan(o[25:, 2:]).all() and np.isnan(l[2:, 25:]).all()
            ok = np.ones((nq, heads), bool)
            ok[25:, 2:] = False
            within("o", o[ok], want["o"][ok], (U * np.abs(want["o"]) + (U + E) * want["o_terms"])[ok])
            assert np.isfinite(l[:2]).all() and np.isfinite(l[:, :25]).all()


def test_nan_in_a_query():
    import bit_nf4_quantised_amd as nf4
    g = rng(78)
    q = bf16(g.standard_normal((3, 4, 64)))
    q[1, 2, 9] = np.nan
    for nk in (40, 5000):
        k, v = (_cache(*oracle.kv4(bf16(g.standard_normal((nk, 2, 64))), "nf4"), 64, "nf4") for _ in range(2))
        O, lse = dev(np.zeros(q.shape)), torch.zeros(4, 3, device="cuda:0")
        nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs([(0, 3, 0, nk)]), dev(q), k, v, O, lse)
        bad = np.zeros((3, 4), bool)
        bad[1, 2] = True
        assert np.isnan(host(O)[bad]).all() and np.isnan(host(lse).T[bad]).all()
        assert np.isfinite(host(O)[~bad]).all() and np.isfinite(host(lse).T[~bad]).all()
