"""Attention over more keys than 64 ranges hold, and with large scores in the backward.

Bounds: as in test_gpu_attn.py, where E = 1e-4 covers scores below 50. Scores are sums of exact products in fp32, scaled
by fp32 factors: with Z the largest sum of absolute terms of a score (scale sum_d |q_d k_d|), a score is off by up to
2^-23 (Z d + 3 Z) at worst; the additions' errors are independent, so sqrt(d) stands for d, four times over. lse is off
by as much, and the exponential of the difference by twice that, relatively: E(Z) = 1e-4 + 2 * 2^-23 Z (4 sqrt(d) + 3).
The bounds are relative: they hold while no probability that counts falls below fp32's normal numbers (2^-126)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import U, bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq,nk,heads,kv,d", [(1, 70000, 4, 1, 128), (3, 40000, 8, 1, 64), (2, 131072, 8, 2, 128)])
@pytest.mark.parametrize("window", [0, 36000])
def test_one_token_over_a_long_cache(nq, nk, heads, kv, d, window):
    import bit_nf4_quantised_amd as nf4
    g = rng(61, nk, window)
    q, k, v = bf16(1.5 * g.standard_normal((nq, heads, d))), bf16(g.standard_normal((nk, kv, d))), bf16(g.standard_normal((nk, kv, d)))
    seqs = nf4.AttnSeqs([(0, nq, 0, nk)], window=window)
    o, lse = torch.zeros(nq, heads, d, dtype=torch.bfloat16, device="cuda:0"), torch.zeros(heads, nq, device="cuda:0")
    Q, K, V = dev(q), dev(k), dev(v)
    ranges = seqs.workspace_bytes(Q, K) // (4 * nq * heads * (d + 8))
    log(f"[attn long] {nq} queries over {nk} keys, window {window}: {ranges} ranges")
    assert ranges > 64
    nf4.qlora_attn_fwd(seqs, Q, K, V, o, lse)
    torch.cuda.synchronize()
    want = oracle.attention(q, k, v, [(0, nq, 0, nk)], d ** -0.5, True, window)
    within("o", o, want["o"], U * np.abs(want["o"]) + (U + 1e-4) * want["o_terms"])
    within("lse", lse, want["lse"], 2e-5 * (1 + np.abs(want["lse"])))


@pytest.mark.parametrize("lens,heads,kv,d", [((300,), 2, 1, 64), ((300, 257, 311), 8, 2, 128)])
def test_large_scores_in_the_backward(lens, heads, kv, d):
    import bit_nf4_quantised_amd as nf4
    log(f"[attn long] scores of std 20, {len(lens)} sequences, heads={heads}/{kv} d={d}")
    T = sum(lens)
    g = rng(62, T, heads)
    q, do = bf16(20 * g.standard_normal((T, heads, d))), bf16(g.standard_normal((T, heads, d)))
    k, v = bf16(g.standard_normal((T, kv, d))), bf16(g.standard_normal((T, kv, d)))
    seqs = [(sum(lens[:i]), n, sum(lens[:i]), n) for i, n in enumerate(lens)]
    want = oracle.attention(q, k, v, seqs, d ** -0.5, True, 0, do=do)
    Z = 0.0
    for q0, nq, _, _ in seqs:
        for h in range(heads):
            Z = max(Z, d ** -0.5 * (np.abs(q[q0:q0 + nq, h]) @ np.abs(k[q0:q0 + nq, h // (heads // kv)]).T).max())
    E = 1e-4 + 2 * 2.0 ** -23 * Z * (4 * np.sqrt(d) + 3)
    Q, K, V, DO = dev(q), dev(k), dev(v), dev(do)
    batch, O, lse = nf4.AttnSeqs(seqs), torch.empty_like(Q), torch.empty(heads, T, device="cuda:0")
    DQ, DK, DV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
    nf4.qlora_attn_fwd(batch, Q, K, V, O, lse)
    nf4.qlora_attn_bwd(batch, Q, K, V, O, lse, DO, DQ, DK, DV)
    torch.cuda.synchronize()
    log(f"[attn long] largest score terms {Z:.0f}, E = {E:.2e}")
    within("o", O, want["o"], U * np.abs(want["o"]) + (U + E) * want["o_terms"])
    for name, t, f in (("dq", DQ, 2), ("dk", DK, 2), ("dv", DV, 1)):
        within(name, t, want[name], U * np.abs(want[name]) + (f * U + E) * want[name + "_terms"])
