"""8-bit activation checkpoints: codes bit for bit, and the adapted linears' backward that reads them.

Bounds of dA (element by element): v = dY B is an fp32 sum of exact products, and enters as a bf16 pair
(relative 2^-17 after scaling): 2^-14 of scale * sum_m (sum |dY||B|) |x8| covers both."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu


def _check_pack(x):
    import bit_nf4_quantised_amd as nf4
    M, K = x.shape
    codes, a = oracle.act8(x)
    kept = nf4.empty_act8(M, K)
    X = dev(x)
    assert np.array_equal(host(X), x)
    nf4.qlora_act8_pack(X, kept)
    out = torch.empty_like(X)
    nf4.qlora_act8_unpack(kept, out)
    torch.cuda.synchronize()
    got = kept.codes.cpu().numpy()
    bad = np.argwhere(got != codes)
    assert not len(bad), (len(bad), [(tuple(i), got[tuple(i)], codes[tuple(i)], x[tuple(i)]) for i in bad[:4]])
    assert np.array_equal(host(kept.absmax), a)
    v = oracle.act8_values(codes, a)
    within("restored", out, v, (2.0 ** -8 + 1e-6) * np.abs(v) + 1e-39)


@pytest.mark.parametrize("M,K", [(1, 64), (3, 128), (77, 4096), (5, 64 * 333), (2100, 512)])
def test_pack_is_exact(M, K):
    log(f"[act8] pack {M} x {K}")
    g = rng(M, K)
    x = bf16(g.standard_normal((M, K)) * np.exp(2 * g.standard_normal((M, 1))))
    x.reshape(-1)[:: 97] *= 32
    _check_pack(bf16(x))


def test_pack_of_every_quotient_of_one_binade():
    """Every 8-bit significand over every 8-bit significand of the maximum, ties among them."""
    log("[act8] quotients")
    rows = []
    for a in range(128, 256):
        for e in (0, -1, -2, -5):
            s = np.arange(128, 256) * 2.0 ** e
            s = s[s <= a]
            block = np.zeros(-(-(len(s) + 1) // 63) * 63)
            block[:len(s)] = s * np.where(np.arange(len(s)) % 2, -1, 1)
            for part in block.reshape(-1, 63):
                rows.append(np.concatenate([[a], part]))
    _check_pack(np.array(rows))


def test_pack_of_very_small_and_large_values():
    log("[act8] range")
    g = rng(8)
    x = g.standard_normal((6, 64))
    for i, e in enumerate((-120, -100, -126, 100, 126, 0)):
        x[i] *= 2.0 ** e
    x[5] = 0
    x[4] = np.clip(x[4], -3e38, 3e38)
    x[3, 0] = 3.3e38        # the rest of the row is far below
    _check_pack(bf16(x))


def _weight(nf4, N, K, seed):
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    nb = N * K // 64
    return nf4.NF4Weight(torch.randint(0, 256, (N * K // 2,), generator=g, device="cuda:0", dtype=torch.uint8),
                         torch.randint(0x28, 0x39, (nb,), generator=g, device="cuda:0", dtype=torch.uint8),
                         0.05 + 0.01 * torch.rand((nb + 255) // 256, generator=g, device="cuda:0"), N, K)


@pytest.mark.parametrize("M,Ns,K,r", [(1, (16,), 64, 16), (5, (64, 16), 192, 32), (77, (256, 64, 64), 512, 16),
                                      (130, (128,), 64, 128), (300, (64, 64), 1088, 48), (513, (96, 32, 32, 160), 320, 64),
                                      (2049, (512,), 128, 16)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_from_a_checkpoint(M, Ns, K, r, accumulate):
    import bit_nf4_quantised_amd as nf4
    log(f"[act8] backward M={M} N={Ns} K={K} r={r} accumulate={accumulate}")
    g = rng(M, K, r, len(Ns))
    x = bf16(g.standard_normal((M, K)))
    codes, a = oracle.act8(x)
    x8 = oracle.act8_values(codes, a)
    kept = nf4.Act8(torch.from_numpy(codes).cuda(), dev(a), M, K)
    scale = 0.5
    ws = [_weight(nf4, n, K, i) for i, n in enumerate(Ns)]
    A = [bf16(0.01 * g.standard_normal((r, K))) for _ in Ns]
    B = [bf16(0.01 * g.standard_normal((n, r))) for n in Ns]
    dY = [bf16(g.standard_normal((M, n))) for n in Ns]
    u = [(x @ m.T).astype(np.float32) for m in A]
    dA0 = [g.standard_normal((r, K)).astype(np.float32) for _ in Ns]
    args = (list(map(dev, dY)), list(map(dev, A)), list(map(dev, B)), scale, [torch.from_numpy(t).cuda() for t in u])

    def outputs():
        return ([torch.empty(M, K, dtype=torch.bfloat16, device="cuda:0") for _ in Ns],
                [torch.from_numpy(t).cuda() for t in dA0], [torch.full((n, r), 0.25, device="cuda:0") for n in Ns])
    dx, dA, dB = outputs()
    nf4.qlora_linear_bwd_act8(ws, kept, *args, dx, dA, dB, accumulate=accumulate)
    ref_x, _, ref_B = got = outputs()
    nf4.qlora_linear_bwd_group(ws, dev(x), *args, *got, accumulate=accumulate)
    _, dA2, dB2 = outputs()
    nf4.qlora_linear_bwd_act8(ws, kept, *args, None, dA2, dB2, accumulate=accumulate)
    torch.cuda.synchronize()
    for i in range(len(Ns)):
        assert torch.equal(dx[i], ref_x[i]) and torch.equal(dB[i], ref_B[i]), "dX or dB differs from the bf16 call's"
        assert torch.equal(dA[i], dA2[i]) and torch.equal(dB[i], dB2[i]), "skipping dX changes dA or dB"
        want = scale * (dY[i] @ B[i]).T @ x8 + (dA0[i] if accumulate else 0.0)
        terms = scale * (np.abs(dY[i]) @ np.abs(B[i])).T @ np.abs(x8) + (np.abs(dA0[i]) if accumulate else 0.0)
        within(f"dA[{i}]", dA[i], want, 2.0 ** -14 * terms)
        assert np.linalg.norm(host(dA[i]) - want) <= 1e-5 * np.linalg.norm(want)
