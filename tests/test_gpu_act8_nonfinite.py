"""8-bit checkpoints of activations that hold a NaN or an infinity: such a block keeps it as its absmax, stands for
NaN throughout, and the gradient that reads it is NaN in the block's columns and right everywhere else."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
M, K = 5, 192


def _input():
    """Rows of three blocks, with the places of what is not finite."""
    x = bf16(rng(31).standard_normal((M, K)))
    x[0, 5] = NAN                 # among numbers
    x[1, 64:128] = NAN            # a whole block
    x[2, 130] = INF
    x[2, 140] = -INF
    x[3, 63], x[3, 0] = -INF, NAN     # both
    x[4, 70], x[4, 71] = -NAN, 3e38
    return x, [(0, 0), (1, 1), (2, 2), (3, 0), (4, 1)]


def _bad(places):
    b = np.zeros((M, K // 64), bool)
    for p in places:
        b[p] = True
    return b


def _check(kept, x, places):
    """kept against the oracle's checkpoint of x, bit for bit apart from which NaN it is."""
    codes, a = oracle.act8(x)
    bad = _bad(places)
    assert np.array_equal(~np.isfinite(a), bad) and not codes.reshape(M, -1, 64)[bad].any()
    assert np.array_equal(kept.codes.cpu().numpy(), codes)
    assert np.array_equal(host(kept.absmax), a, equal_nan=True)


def test_pack_and_unpack():
    import bit_nf4_quantised_amd as nf4
    log("[act8] not finite: pack")
    x, places = _input()
    kept = nf4.empty_act8(M, K)
    nf4.qlora_act8_pack(dev(x), kept)
    out = torch.empty(M, K, dtype=torch.bfloat16, device="cuda:0")
    nf4.qlora_act8_unpack(kept, out)
    torch.cuda.synchronize()
    _check(kept, x, places)
    a = host(kept.absmax)
    assert np.isnan(a[0, 0]) and np.isnan(a[1, 1]) and a[2, 2] == INF and np.isnan(a[3, 0]) and np.isnan(a[4, 1])
    got, bad = host(out).reshape(M, -1, 64), _bad(places)
    assert np.isnan(got[bad]).all()
    v = oracle.act8_values(*oracle.act8(x)).reshape(M, -1, 64)
    within("restored", got[~bad], v[~bad], (2.0 ** -8 + 1e-6) * np.abs(v[~bad]) + 1e-39)


def test_norm_with_a_checkpoint():
    """The norm's codes are those of the y it writes; a row with a NaN or an infinity in it is lost whole."""
    import bit_nf4_quantised_amd as nf4
    log("[act8] not finite: norm")
    for k in (192, 4160):        # a wave and a workgroup a row
        x = bf16(rng(32).standard_normal((M, k)))
        x[1, 7], x[3, k - 1] = NAN, INF
        y, y8, alone = torch.empty(M, k, dtype=torch.bfloat16, device="cuda:0"), nf4.empty_act8(M, k), nf4.empty_act8(M, k)
        nf4.qlora_rmsnorm_fwd(dev(x), dev(np.ones(k)), 1e-5, y, act8=y8)
        nf4.qlora_act8_pack(y, alone)
        torch.cuda.synchronize()
        assert torch.equal(y8.codes, alone.codes)
        assert torch.equal(y8.absmax.view(torch.int16), alone.absmax.view(torch.int16))
        a = host(y8.absmax)
        assert np.isnan(a[1]).all() and np.isnan(a[3, -1]) and np.isfinite(a[[0, 2, 4]]).all()


@pytest.mark.parametrize("rows", [M, 300])       # one range of rows, and several with their sum
def test_gradient_from_a_checkpoint(rows):
    import bit_nf4_quantised_amd as nf4
    log(f"[act8] not finite: dA of {rows} rows")
    g = rng(33, rows)
    x = bf16(g.standard_normal((rows, K)))
    x[0, 70], x[rows - 1, 130] = NAN, INF
    kept = nf4.empty_act8(rows, K)
    nf4.qlora_act8_pack(dev(x), kept)
    N, r = 64, 32
    W = nf4.quantize_weight(torch.from_numpy(g.standard_normal((N, K)).astype(np.float32)).cuda())
    dY, A, B = bf16(g.standard_normal((rows, N))), bf16(g.standard_normal((r, K))), bf16(g.standard_normal((N, r)))
    u = torch.from_numpy(g.standard_normal((rows, r)).astype(np.float32)).cuda()
    dA, dB = torch.empty(r, K, device="cuda:0"), torch.empty(N, r, device="cuda:0")
    nf4.qlora_linear_bwd_act8([W], kept, [dev(dY)], [dev(A)], [dev(B)], 0.5, [u], None, [dA], [dB])
    torch.cuda.synchronize()
    got = host(dA)
    assert np.isnan(got[:, 64:]).all()
    x8 = oracle.act8_values(*oracle.act8(x))[:, :64]
    want, terms = 0.5 * (dY @ B).T @ x8, 0.5 * (np.abs(dY) @ np.abs(B)).T @ np.abs(x8)
    within("dA", got[:, :64], want, 2.0 ** -14 * terms)
    assert torch.isfinite(dB).all()
