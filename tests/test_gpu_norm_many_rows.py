"""The norm's forward over more rows than one launch holds threads for (2^26 short rows; per-head norms of a few
million tokens have as many), on both sides of the launches' borders and at the end. Rows repeat with a period of 1009,
so that every row of the result can be compared with the same rows in a small call, bit for bit."""
import pytest
import torch

from gpu_helpers import log

pytestmark = pytest.mark.gpu
PERIOD = 1009


def _tiled(small, M):
    return small.repeat(-(-M // PERIOD), 1)[:M].contiguous()


@pytest.mark.parametrize("K,M,residual,act8", [(8, (1 << 26) + 77, True, False), (64, (1 << 26) + 5, False, True),
                                              (2056, (1 << 24) + 3, False, False)])
def test_more_rows_than_a_launch_holds(K, M, residual, act8):
    import bit_nf4_quantised_amd as nf4
    log(f"[norm] {M} rows of {K}")
    g = torch.Generator(device="cuda:0").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    x, res, w = r(PERIOD, K), r(PERIOD, K) if residual else None, r(K)
    y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(PERIOD, device="cuda:0")
    kept = nf4.empty_act8(PERIOD, K) if act8 else None
    nf4.qlora_rmsnorm_fwd(x, w, 1e-5, y, residual=res, h=h, rstd=rstd, act8=kept)
    X = _tiled(x, M)
    R = _tiled(res, M) if residual else None
    Y, H = torch.zeros_like(X), torch.zeros_like(X) if residual else None
    S, kept_all = torch.zeros(M, device="cuda:0"), nf4.empty_act8(M, K) if act8 else None
    nf4.qlora_rmsnorm_fwd(X, w, 1e-5, Y, residual=R, h=H, rstd=S, act8=kept_all)
    torch.cuda.synchronize()
    log("[norm] done")
    del X, R
    pairs = [(Y, y), (S[:, None], rstd[:, None])] + ([(H, h)] if residual else [])
    if act8:
        pairs += [(kept_all.codes, kept.codes), (kept_all.absmax, kept.absmax)]
    step = PERIOD << 12
    for at in range(0, M, step):
        for j, (big, small) in enumerate(pairs):
            part = big[at:at + step]
            assert torch.equal(part, small.repeat(-(-part.shape[0] // PERIOD), 1)[:part.shape[0]]), (j, at)
    del Y, H, S, kept_all, pairs, big, part
    torch.cuda.empty_cache()
