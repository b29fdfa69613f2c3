"""The residual norm, forward and backward, against the float64 oracle.

Bounds: every bf16 output is an fp32 value rounded once (relative U = 2^-8); fp32 arithmetic over at
most 16384 columns in sums of 8 to 32 terms per lane and trees above loses under 1e-5 of the sum of
absolute terms. rstd and dw are fp32: 1e-5 relative, 2e-5 of the absolute terms (sums over rows)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import U, bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _inputs(M, K, residual):
    g = rng(M, K, int(residual))
    x = bf16(g.standard_normal((M, K)))
    res = bf16(2 * g.standard_normal((M, K))) if residual else None
    w = bf16(1 + 0.2 * g.standard_normal(K))
    return g, x, res, w


@pytest.mark.parametrize("M", [1, 3, 130])
@pytest.mark.parametrize("K", [8, 64, 72, 512, 520, 1024, 2048, 2056, 4096, 5120, 8192, 11008, 16384])
def test_forward_and_backward(M, K):
    import bit_nf4_quantised_amd as nf4
    residual = K % 3 != 0
    log(f"[norm] M={M} K={K} residual={residual}")
    g, x, res, w = _inputs(M, K, residual)
    h, y, rstd = oracle.rmsnorm(x, res, w, EPS)
    kept = nf4.empty_act8(M, K) if K % 64 == 0 else None
    H, Y = dev(np.zeros((M, K))), dev(np.zeros((M, K)))
    R = torch.zeros(M, device="cuda:0")
    nf4.qlora_rmsnorm_fwd(dev(x), dev(w), EPS, Y, residual=None if res is None else dev(res), h=H, rstd=R, act8=kept)
    torch.cuda.synchronize()
    within("h", H, h, (U + 1e-6) * np.abs(h))
    within("y", Y, y, (U + 1e-5) * np.abs(y))
    within("rstd", R, rstd, 1e-5 * rstd)
    if kept is not None:   # the checkpoint is exactly that of the y written
        codes, a = oracle.act8(host(Y))
        assert np.array_equal(kept.codes.cpu().numpy(), codes) and np.array_equal(host(kept.absmax), a)
        alone = nf4.empty_act8(M, K)
        nf4.qlora_act8_pack(Y, alone)
        assert torch.equal(alone.codes, kept.codes) and torch.equal(alone.absmax, kept.absmax)
    # backward at the stored h and rstd
    dy, dh = bf16(g.standard_normal((M, K))), bf16(g.standard_normal((M, K)))
    for with_dh, accumulate in ((True, False), (False, True)):
        hs, rs = host(H), host(R)
        dx, dw, dx_terms, dw_terms = oracle.rmsnorm_bwd(dy, dh if with_dh else None, hs, w, rs)
        DX = dev(np.zeros((M, K)))
        DW = torch.full((K,), 2.0 if accumulate else float("nan"), device="cuda:0")
        nf4.qlora_rmsnorm_bwd(dev(dy), H, dev(w), R, DX, dw=DW, dh=dev(dh) if with_dh else None, accumulate=accumulate)
        only = dev(np.zeros((M, K)))
        nf4.qlora_rmsnorm_bwd(dev(dy), H, dev(w), R, only, dh=dev(dh) if with_dh else None)
        torch.cuda.synchronize()
        within("dx", DX, dx, (U + 1e-6) * np.abs(dx) + 1e-5 * dx_terms)
        within("dw", DW, dw + (2.0 if accumulate else 0.0), 2e-5 * dw_terms + (1e-6 if accumulate else 0.0))
        assert torch.equal(only, DX), "dx without dw differs"


def test_many_rows_and_repeated_results():
    import bit_nf4_quantised_amd as nf4
    M, K = 1500, 768
    log(f"[norm] M={M} K={K}")
    g, x, res, w = _inputs(M, K, True)
    dy = bf16(g.standard_normal((M, K)))
    h, y, rstd = oracle.rmsnorm(x, res, w, EPS)
    H, Y, R = dev(np.zeros((M, K))), dev(np.zeros((M, K))), torch.zeros(M, device="cuda:0")
    nf4.qlora_rmsnorm_fwd(dev(x), dev(w), EPS, Y, residual=dev(res), h=H, rstd=R)
    within("y", Y, y, (U + 1e-5) * np.abs(y))
    got = []
    for _ in range(3):
        DX, DW = dev(np.zeros((M, K))), torch.zeros(K, device="cuda:0")
        nf4.qlora_rmsnorm_bwd(dev(dy), H, dev(w), R, DX, dw=DW)
        got.append((DX, DW))
    dx, dw, dx_terms, dw_terms = oracle.rmsnorm_bwd(dy, None, host(H), w, host(R))
    within("dx", got[0][0], dx, (U + 1e-6) * np.abs(dx) + 1e-5 * dx_terms)
    within("dw", got[0][1], dw, 2e-5 * dw_terms)
    assert all(torch.equal(a, got[0][0]) and torch.equal(b, got[0][1]) for a, b in got)


def test_in_place_and_rows_of_zeros():
    import bit_nf4_quantised_amd as nf4
    M, K = 5, 4096
    log("[norm] in place")
    _, x, res, w = _inputs(M, K, True)
    x[2] = 0
    res[2] = 0
    h, y, _ = oracle.rmsnorm(x, res, w, EPS)
    X, R = dev(x), dev(res)
    kept = nf4.empty_act8(M, K)
    nf4.qlora_rmsnorm_fwd(X, dev(w), EPS, X, residual=R, h=R, act8=kept)   # y over x, h over the residual
    torch.cuda.synchronize()
    within("y", X, y, (U + 1e-5) * np.abs(y))
    within("h", R, h, (U + 1e-6) * np.abs(h))
    assert not kept.codes[2].any() and not kept.absmax[2].any()
