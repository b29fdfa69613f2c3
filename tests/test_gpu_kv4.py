"""Keys and values into a 4-bit cache and back: codes, maxima and values bit for bit those of the oracle."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import bf16, dev, host, rng

pytestmark = pytest.mark.gpu
BOOKS = ["nf4", "fp4", "int4"]


def _empty(tokens, kv, d, book, layout="heads"):
    import bit_nf4_quantised_amd as nf4
    nb = (d + 31) // 32
    if layout == "heads":
        c = nf4.empty_kv4(tokens, kv, d, codebook=book)
    elif layout == "tokens":
        c = nf4.Kv4(torch.empty(tokens, kv, nb, 16, dtype=torch.uint8, device="cuda:0"),
                    torch.empty(tokens, kv, nb, dtype=torch.bfloat16, device="cuda:0"), d, book)
    else:                       # a layer's part of all layers' cache, and tokens from 3 on
        c = nf4.Kv4(torch.empty(2, kv, tokens + 3, nb, 16, dtype=torch.uint8, device="cuda:0")[1].permute(1, 0, 2, 3)[3:],
                    torch.empty(2, kv, tokens + 3, nb, dtype=torch.bfloat16, device="cuda:0")[1].permute(1, 0, 2)[3:], d, book)
    c.codes.fill_(0x5A)
    c.absmax.fill_(2.0)
    return c


def _run(seqs, kv, d, book, tokens=None, layout="heads", source="tokens", x=None, std=1.0):
    import bit_nf4_quantised_amd as nf4
    log(f"[kv4] seqs={seqs[:6]} kv={kv} d={d} {book} {layout} {source}")
    tq = max(s[0] + s[1] for s in seqs)
    tk = max(s[2] + s[3] for s in seqs) if tokens is None else tokens
    g = rng(tq, tk, kv, d)
    k, v = (bf16(std * g.standard_normal((tq, kv, d))) for _ in range(2))
    if x is not None:
        k.reshape(-1)[:x.size] = x
        v.reshape(-1)[-x.size:] = x

    def place(a):
        t = dev(a)
        if source == "fused":
            wide = torch.full((tq, kv + 2, d + 8), 9.0, dtype=t.dtype, device=t.device)
            wide[:, 1:1 + kv, :d] = t
            return wide[:, 1:1 + kv, :d]
        return t
    k4, v4 = _empty(tk, kv, d, book, layout), _empty(tk, kv, d, book, layout)
    batch = nf4.AttnSeqs(seqs)
    nf4.qlora_kv4_write(batch, place(k), place(v), k4, v4)
    ko, vo = place(np.full(k.shape, 3.0)), place(np.full(k.shape, 3.0))
    nf4.qlora_kv4_read(batch, k4, v4, ko, vo)
    torch.cuda.synchronize()
    inside, rows = np.zeros(tk, bool), np.zeros(tq, bool)
    for q0, nq, k0, nk in seqs:
        inside[k0 + nk - nq:k0 + nk] = rows[q0:q0 + nq] = True
    for src, c, out in ((k, k4, ko), (v, v4, vo)):
        codes, absmax = oracle.kv4(src, book)
        got_c, got_a = c.codes.cpu().numpy(), host(c.absmax)
        assert np.all(got_c[~inside] == 0x5A) and np.all(got_a[~inside] == 2.0), "a token outside was written"
        for q0, nq, k0, nk in seqs:
            a, b = slice(q0, q0 + nq), slice(k0 + nk - nq, k0 + nk)
            assert np.array_equal(got_a[b], absmax[a], equal_nan=True)
            assert np.array_equal(got_c[b], codes[a])
        want = oracle.kv4_values(codes, absmax, d, book)
        assert np.array_equal(host(out)[rows], want[rows], equal_nan=True) and np.all(host(out)[~rows] == 3.0)


@pytest.mark.parametrize("book", BOOKS)
@pytest.mark.parametrize("d", [8, 32, 40, 64, 72, 80, 96, 120, 128])
def test_head_sizes(d, book):
    _run([(0, 37, 0, 37)], 2, d, book)


@pytest.mark.parametrize("book", BOOKS)
def test_behind_what_a_sequence_holds(book):
    _run([(0, 1, 0, 1), (1, 1, 100, 50), (2, 20, 200, 300)], 3, 64, book, tokens=600)
    _run([(i, 1, 64 * i, 1 + i) for i in range(40)], 8, 128, book)
    _run([(i, 1, 20 * i, 5 + i % 7) for i in range(150)], 1, 96, book)      # more than one launch holds
    _run([(2, 3, 40, 4), (9, 0, 10, 6), (9, 2, 0, 2)], 2, 64, book, tokens=50)


@pytest.mark.parametrize("layout", ["tokens", "part"])
@pytest.mark.parametrize("source", ["tokens", "fused"])
def test_layouts(layout, source):
    _run([(0, 50, 0, 50), (50, 7, 60, 30)], 4, 128, "nf4", layout=layout, source=source)
    _run([(0, 50, 0, 50), (50, 7, 60, 30)], 1, 72, "fp4", layout=layout, source=source)


@pytest.mark.parametrize("book", BOOKS)
def test_ties_and_every_quotient(book):
    """All quotients of two 8-bit significands, among them every tie; 31 of them a block beside the maximum."""
    p = np.arange(128, 256, dtype=np.float64)
    num, den = np.meshgrid(p, p)
    blocks = []
    for e in (0, 1, 2, 3, 4, 5):
        n, a = (num * 2.0 ** -e).reshape(-1), den.reshape(-1)
        n = np.where(np.arange(n.size) % 2, -n, n)
        take = np.abs(n) <= a
        for top in p:
            q = n[take & (a == top)]
            q = np.concatenate([q, np.zeros(-len(q) % 31)]).reshape(-1, 31)
            blocks.append(np.concatenate([np.full((len(q), 1), top), q], axis=1))
    x = np.concatenate(blocks)
    x = np.concatenate([x, np.zeros((-len(x) % 4, 32))])
    # midpoints of INT4 and FP4 over every absmax that makes them bf16 values
    mid = []
    for a in range(1, 256):
        for m in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            mid.append((a, m * a / 6))
        for k in range(7):
            mid.append((a, (2 * k + 1) * a / 14))
    mid = np.array([(a, m) for a, m in mid if bf16(m) == m])
    t = np.zeros((len(mid) + (-len(mid) % 4), 32))
    t[:len(mid), 0], t[:len(mid), 1], t[:len(mid), 2] = mid[:, 0], mid[:, 1], -mid[:, 1]
    x = np.concatenate([x, t]).reshape(-1, 1, 128)
    import bit_nf4_quantised_amd as nf4
    log(f"[kv4] {x.size // 32} blocks {book}")
    k4, v4 = _empty(len(x), 1, 128, book), _empty(len(x), 1, 128, book)
    X = dev(x)
    nf4.qlora_kv4_write(nf4.AttnSeqs([(0, len(x), 0, len(x))]), X, X, k4, v4)
    torch.cuda.synchronize()
    codes, absmax = oracle.kv4(x, book)
    assert np.array_equal(k4.codes.cpu().numpy(), codes) and np.array_equal(v4.codes.cpu().numpy(), codes)
    assert np.array_equal(host(k4.absmax), absmax)


@pytest.mark.parametrize("book", BOOKS)
@pytest.mark.parametrize("std", [1e-36, 1e-20, 1e-4, 1e4, 1e20, 1e37])
def test_magnitudes(std, book):
    _run([(0, 20, 0, 20)], 1, 128, book, std=std)


@pytest.mark.parametrize("book", BOOKS)
def test_zeros_nan_and_infinities(book):
    x = np.zeros(3 * 128)
    x[5], x[40], x[100], x[128 + 7], x[128 + 70], x[300] = np.nan, np.inf, -np.inf, -0.0, -3.0, 1e-30
    x[300 + 1] = np.nan
    fine = np.isfinite(x)
    x[fine] = bf16(x[fine])
    _run([(0, 9, 0, 9)], 2, 128, book, x=x)


def test_offsets_past_32_bits():
    """A cache of more than 4 GiB of codes: rows at its end."""
    import bit_nf4_quantised_amd as nf4
    tokens, kv, d = (1 << 25) + 100, 3, 128         # 64 bytes a row: 6.4 GiB
    k4, v4 = nf4.empty_kv4(tokens, kv, d), nf4.empty_kv4(tokens, kv, d)
    g = rng(8)
    k, v = bf16(g.standard_normal((70, kv, d))), bf16(g.standard_normal((70, kv, d)))
    batch = nf4.AttnSeqs([(0, 70, tokens - 200, 200)])
    nf4.qlora_kv4_write(batch, dev(k), dev(v), k4, v4)
    ko, vo = dev(np.zeros(k.shape)), dev(np.zeros(k.shape))
    nf4.qlora_kv4_read(batch, k4, v4, ko, vo)
    torch.cuda.synchronize()
    for src, c, out in ((k, k4, ko), (v, v4, vo)):
        codes, absmax = oracle.kv4(src, "nf4")
        assert np.array_equal(c.codes[tokens - 70:].cpu().numpy(), codes)
        assert np.array_equal(host(out), oracle.kv4_values(codes, absmax, d, "nf4"))
