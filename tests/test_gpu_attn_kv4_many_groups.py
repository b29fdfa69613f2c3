"""Attention over a 4-bit cache whose workgroups of 512 threads do not fit one launch: 65528 heads that share one head's
queries, keys and values through a head stride of 0, over 64 sequences of three row tiles. Every head equals the first, bit for
bit, and the first the oracle. Bounds as in test_gpu_attn_kv4.py."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import U, bf16, dev, rng, within

pytestmark = pytest.mark.gpu
E = 1e-4


def test_more_workgroups_of_512_threads_than_a_launch_holds():
    import bit_nf4_quantised_amd as nf4
    heads, d, n, nk, count = 65528, 8, 768, 70, 64
    seqs = [(n * i, n, 0, nk) for i in range(count)]
    T = n * count
    g = rng(52)
    q, k, v = bf16(g.standard_normal((T, 1, d))), bf16(g.standard_normal((nk, 1, d))), bf16(g.standard_normal((nk, 1, d)))
    blocks = [oracle.kv4(x, "nf4") for x in (k, v)]
    values = [oracle.kv4_values(*b, d, "nf4") for b in blocks]
    want = oracle.attention(q, *values, seqs, d ** -0.5, False, 0)
    caches = [nf4.Kv4(torch.from_numpy(c).to("cuda:0").expand(nk, heads, 1, 16), dev(a).expand(nk, heads, 1), d) for c, a in blocks]
    o = torch.zeros(T, heads, d, dtype=torch.bfloat16, device="cuda:0")
    log("[attn kv4 wide] forward")
    nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs(seqs, causal=False), dev(q).expand(T, heads, d), *caches, o)
    torch.cuda.synchronize()
    log("[attn kv4 wide] done")
    within("o", o[:, :1], want["o"], U * np.abs(want["o"]) + (U + E) * want["o_terms"])
    for h in range(0, heads, 2048):
        assert (o[:, h:h + 2048] == o[:, :1]).all(), h
    del o
    torch.cuda.empty_cache()
