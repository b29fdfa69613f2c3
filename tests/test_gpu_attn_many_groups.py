"""Attention whose workgroups do not fit one launch (2^24 of 256 threads): 65528 heads, which share one head's q, k, v
and dout through a head stride of 0, over 64 sequences of five tiles. Every head equals the first, bit for bit, and the
first the oracle. Bounds as in test_gpu_attn.py."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import U, bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu
E = 1e-4


def test_more_workgroups_than_a_launch_holds():
    import bit_nf4_quantised_amd as nf4
    heads, d, n, count = 65528, 8, 513, 64
    seqs = [(n * i, n, n * i, n) for i in range(count)]
    T = n * count
    assert 5 * heads * count > (1 << 24) - 1 > 5 * heads
    g = rng(51)
    q, k, v, do = (bf16(g.standard_normal((T, 1, d))) for _ in range(4))
    want = oracle.attention(q, k, v, seqs, d ** -0.5, True, 0, do=do)
    wide = [dev(a).expand(T, heads, d) for a in (q, k, v, do)]
    new = lambda: torch.zeros(T, heads, d, dtype=torch.bfloat16, device="cuda:0")  # noqa: E731
    batch, lse = nf4.AttnSeqs(seqs), torch.zeros(heads, T, device="cuda:0")
    out = {"o": new()}
    log("[attn wide] forward")
    nf4.qlora_attn_fwd(batch, *wide[:3], out["o"], lse)
    torch.cuda.synchronize()
    out.update(dq=new(), dk=new(), dv=new())
    log("[attn wide] backward")
    nf4.qlora_attn_bwd(batch, *wide[:3], out["o"], lse, wide[3], out["dq"], out["dk"], out["dv"])
    torch.cuda.synchronize()
    log("[attn wide] done")
    for name, t in out.items():
        f = {"o": 1, "dq": 2, "dk": 2, "dv": 1}[name]
        within(name, t[:, :1], want[name], U * np.abs(want[name]) + (f * U + E) * want[name + "_terms"])
        for h in range(0, heads, 2048):
            assert (t[:, h:h + 2048] == t[:, :1]).all(), (name, h)
    within("lse", lse[:1], want["lse"], 2e-5 * (1 + np.abs(want["lse"])))
    for h in range(0, heads, 2048):
        assert (lse[h:h + 2048] == lse[:1]).all(), h
    del out, lse, t
    torch.cuda.empty_cache()
