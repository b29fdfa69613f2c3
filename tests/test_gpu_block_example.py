"""The example's attention block, forward and backward, against the same block in float64 on the CPU.

Tolerances: every stage rounds its result to bf16 once (relative error up to 2^-8, independent over
elements: about 1.7e-3 of a tensor's norm); the output passes 5 such stages and the gradients up to 9,
and the 8-bit checkpoints put an error of absmax / 254 at most, about 6e-3 of the norm of Gaussian
values, on the operand of dA. 5e-3 sqrt(5) and 5e-3 sqrt(9) + 6e-3 bound them: 1.2e-2 and 2.1e-2."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import gpu_dequant, log
from layer_helpers import bf16, dev, host, rng

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def test_block_against_the_oracle():
    import bit_nf4_quantised_amd as nf4
    from attention_block import EPS, AttentionBlock
    log("[block] forward and backward")
    blk = AttentionBlock(hidden=256, heads=4, kv_heads=2, d=64)
    lens = [40, 1, 23]
    M, d, s = sum(lens), blk.d, blk.scale
    g = rng(77)
    x, res = bf16(g.standard_normal((M, 256))), bf16(g.standard_normal((M, 256)))
    dout, dh = bf16(g.standard_normal((M, 256))), bf16(g.standard_normal((M, 256)))
    out, h = blk.forward(dev(x), dev(res), nf4.AttnSeqs.packed(lens))
    dx = blk.backward(dev(dout), dev(dh))
    torch.cuda.synchronize()

    W = [oracle.f32_from_bf16_bits(gpu_dequant(w)).astype(np.float64).reshape(w.N, w.K) for w in blk.weights]
    A, B = [host(t) for t in blk.A], [host(t) for t in blk.B]
    w = host(blk.norm_weight)
    hh, n, rstd = oracle.rmsnorm(x, res, w, EPS)
    q, k, v = (n @ W[i].T + s * (n @ A[i].T) @ B[i].T for i in range(3))
    q, k, v = q.reshape(M, 4, d), k.reshape(M, 2, d), v.reshape(M, 2, d)
    seqs = [(sum(lens[:i]), m, sum(lens[:i]), m) for i, m in enumerate(lens)]
    a = oracle.attention(q, k, v, seqs, d ** -0.5, True, 0)["o"].reshape(M, -1)
    want = a @ W[3].T + s * (a @ A[3].T) @ B[3].T
    assert _rel(host(out), want) < 1.2e-2 and _rel(host(h), hh) < 4e-3

    bwd = lambda i, y, inp: (y @ W[i] + s * (y @ B[i]) @ A[i], s * (y @ B[i]).T @ inp, s * y.T @ (inp @ A[i].T))  # noqa: E731
    da, dA3, dB3 = bwd(3, dout, a)
    t = oracle.attention(q, k, v, seqs, d ** -0.5, True, 0, do=da.reshape(M, 4, d))
    parts = [bwd(i, t[m].reshape(M, -1), n) for i, m in enumerate(("dq", "dk", "dv"))]
    dn = sum(p[0] for p in parts)
    dxw = oracle.rmsnorm_bwd(dn, dh, hh, w, rstd)[0]
    assert _rel(host(dx), dxw) < 2.1e-2
    for i, (_, dA, dB) in enumerate(parts + [(None, dA3, dB3)]):
        assert _rel(host(blk.grads[2 * i]), dA) < 2.1e-2, ("dA", i)
        assert _rel(host(blk.grads[2 * i + 1]), dB) < 2.1e-2, ("dB", i)


def test_decoding_matches_the_packed_forward():
    import bit_nf4_quantised_amd as nf4
    from attention_block import AttentionBlock
    log("[block] decode")
    blk = AttentionBlock()
    g = rng(78)
    x, res = dev(bf16(g.standard_normal((20, 512)))), dev(bf16(g.standard_normal((20, 512))))
    out, _ = blk.forward(x, res, nf4.AttnSeqs.packed([20]))
    kc = torch.zeros(1, 32, blk.kv_heads, blk.d, dtype=torch.bfloat16, device="cuda:0")
    vc = torch.zeros_like(kc)
    one = torch.cat([blk.decode(x[i:i + 1], res[i:i + 1], kc, vc, [i]) for i in range(20)])
    assert _rel(host(one), host(out)) < 1.2e-2


def test_training_lowers_the_loss():
    import bit_nf4_quantised_amd as nf4
    from attention_block import AttentionBlock
    log("[block] training")
    blk = AttentionBlock(hidden=256, heads=4, kv_heads=2, d=64)
    g = rng(79)
    x, res, target = (dev(bf16(g.standard_normal((64, 256)))) for _ in range(3))
    losses = []
    for step in range(1, 31):
        out, h = blk.forward(x, res, nf4.AttnSeqs.packed([50, 14]))
        diff = out.float() - target.float()
        losses.append(diff.square().sum().item())
        blk.backward((diff / 64).to(torch.bfloat16), torch.zeros_like(h))
        blk.plan.step(step)
    assert losses[-1] < 0.9 * losses[0] and all(np.isfinite(losses)), losses[::5]
