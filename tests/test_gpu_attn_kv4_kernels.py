"""Every kernel of the attention over a 4-bit cache against the float64 oracle: over whole caches, and over caches with a block
that stands for NaN, which has to reach exactly the queries that see it, whatever kernel, range and lane holds it.

Bounds (element by element; U = 2^-8 is bf16's unit roundoff): every probability and the result are rounded once, U |o| + (U + E)
sum_j P |v|. E = 1e-4 for what is fp32: scores of up to 128 products (exact in fp32, added 16 and 32 at a time: 16 * 2^-24 of sums of
magnitudes below 20), the exponential of arguments below 50 (50 * 2^-24 * 8), sums over 4100 keys (16 at a time and more, and
up to 64 lanes, waves and ranges: 330 * 2^-24): 7e-5 together. lse is fp32: 2e-5 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from kv4_cases import CASES, name_of, sequences
from layer_helpers import U, bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu
E = 1e-4


class Batch:
    """A case's inputs, what the oracle makes of them, and what lies in no query's sight made NaN."""

    def __init__(self, c):
        self.c, self.seqs = c, sequences(c)
        tq, tk = c.nq * len(c.nks), self.seqs[-1][2] + self.seqs[-1][3] + 2
        g = rng(CASES.index(c), 3)
        self.q = bf16(1.5 * g.standard_normal((tq, c.heads, c.d)))
        self.x = {n: bf16(g.standard_normal((tk, c.kv, c.d))) for n in "kv"}
        blocks = {n: oracle.kv4(self.x[n], c.book) for n in "kv"}
        values = {n: oracle.kv4_values(*blocks[n], c.d, c.book) for n in "kv"}
        self.want = oracle.attention(self.q, values["k"], values["v"], self.seqs, c.d ** -0.5, c.causal, c.window)
        seen = np.zeros(tk, bool)
        for _, nq, k0, nk in self.seqs:
            seen[k0:k0 + nk] |= self.see(nq, nk).any(axis=0)
        for _, absmax in blocks.values():
            absmax[~seen] = np.nan
        self.blocks = blocks

    def see(self, nq, nk):
        return oracle.visible(nq, nk, self.c.causal, self.c.window)

    def run(self, blocks):
        import bit_nf4_quantised_amd as nf4
        c = self.c

        def cache(codes, absmax):
            return nf4.Kv4(torch.from_numpy(codes).to("cuda:0").permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3),
                           dev(absmax).permute(1, 0, 2).contiguous().permute(1, 0, 2), c.d, c.book)
        k4, v4, q = cache(*blocks["k"]), cache(*blocks["v"]), dev(self.q)
        batch = nf4.AttnSeqs(self.seqs, causal=c.causal, window=c.window)
        outs = []
        for _ in range(2):
            o, lse = torch.full_like(q, 3.0), torch.full((c.heads, q.shape[0]), 5.0, device="cuda:0")
            nf4.qlora_attn_kv4_fwd(batch, q, k4, v4, o, lse)
            torch.cuda.synchronize()
            outs.append((o.view(torch.int16), lse.view(torch.int32), o, lse))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1]), "two calls differ"
        return host(outs[0][2]), host(outs[0][3])

    def check(self, o, lse, lost):
        """lost [tokens, heads]: the rows that have to be NaN."""
        assert np.isnan(o[lost]).all() and np.isnan(lse.T[lost]).all(), "a lost block did not reach a query that sees it"
        w, ok = self.want, ~lost
        within("o", o[ok], w["o"][ok], (U * np.abs(w["o"]) + (U + E) * w["o_terms"])[ok])
        fine = np.where(np.isfinite(w["lse"]), w["lse"], 0.0)
        within("lse", lse.T[ok], w["lse"].T[ok], (2e-5 * (1 + np.abs(fine))).T[ok])


@pytest.fixture(scope="module", params=CASES, ids=name_of)
def batch(request):
    return Batch(request.param)


def test_against_the_oracle(batch):
    log(f"[attn kv4 kernels] {batch.c}")
    batch.check(*batch.run(batch.blocks), np.zeros(batch.q.shape[:2], bool))


@pytest.mark.parametrize("which,bad,first_block,last_sequence", [("k", np.nan, True, False), ("k", -np.inf, False, True),
                                                                 ("v", np.nan, False, False), ("v", np.inf, True, True)])
def test_a_lost_block_reaches_the_queries_that_see_it_and_no_other(batch, which, bad, first_block, last_sequence):
    c = batch.c
    log(f"[attn kv4 lost] {which} {bad} {c}")
    q0, nq, k0, nk = batch.seqs[-1 if last_sequence else 0]
    see = batch.see(nq, nk)
    keys = np.flatnonzero(see.any(axis=0))
    j = int(keys[0]) if last_sequence else max(int(keys[0]), nk - nq + nq // 2)      # an early key; one that some queries see
    head, column = (0, 0) if first_block else (c.kv - 1, c.d - 1)
    row = batch.x[which][k0 + j, head].copy()
    row[column] = bad
    blocks = {n: (a.copy(), b.copy()) for n, (a, b) in batch.blocks.items()}
    for old, new in zip(blocks[which], oracle.kv4(row, c.book)):
        old[k0 + j, head] = new
    lost, G = np.zeros(batch.q.shape[:2], bool), c.heads // c.kv
    lost[q0:q0 + nq, head * G:(head + 1) * G] = see[:, j, None]
    assert lost.any()
    batch.check(*batch.run(blocks), lost)
