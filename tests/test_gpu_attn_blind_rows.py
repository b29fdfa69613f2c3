"""Queries that see no key have no gradient and give none: what their rows of q and dout hold does not reach dk, dv or
any other row, NaN included."""
import pytest
import torch

from gpu_helpers import log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,heads,kv,d", [
    ([(0, 200, 0, 60), (200, 40, 60, 0), (240, 70, 60, 1)], 4, 2, 64),
    ([(0, 200, 0, 60), (200, 40, 60, 0), (240, 70, 60, 1)], 4, 2, 128),      # one wave a SIMD
    ([(0, 333, 0, 300), (333, 1, 300, 1)], 8, 2, 80),
    ([(150 * i, 150, 129 * i, 129) for i in range(16)], 64, 64, 128),        # two waves a SIMD
    ([(150 * i, 150, 129 * i, 129) for i in range(16)], 64, 64, 64),
])
@pytest.mark.parametrize("window", [0, 40])
def test_rows_without_keys_give_no_gradient(seqs, heads, kv, d, window):
    import bit_nf4_quantised_amd as nf4
    log(f"[attn blind] {seqs[:3]} heads={heads}/{kv} d={d} window={window}")
    tq, tk = max(s[0] + s[1] for s in seqs), max(s[2] + s[3] for s in seqs)
    g = torch.Generator(device="cuda:0").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    q, k, v, do = r(tq, heads, d), r(tk, kv, d), r(tk, kv, d), r(tq, heads, d)
    blind = torch.cat([torch.arange(nq) + (nk - nq) < 0 for _, nq, _, nk in seqs]).cuda()
    assert blind.any() and not blind.all()
    batch, got = nf4.AttnSeqs(seqs, window=window), []
    for junk in (None, float("nan")):
        if junk is not None:
            q, do = q.clone(), do.clone()
            q[blind], do[blind] = junk, junk
        o, lse, dq = torch.empty_like(q), torch.empty(heads, tq, device="cuda:0"), torch.empty_like(q)
        dk, dv = torch.empty_like(k), torch.empty_like(v)
        nf4.qlora_attn_fwd(batch, q, k, v, o, lse)
        nf4.qlora_attn_bwd(batch, q, k, v, o, lse, do, dq, dk, dv)
        torch.cuda.synchronize()
        assert not o[blind].any() and (lse[:, blind] == float("-inf")).all() and not dq[blind].any()
        got.append([o, lse, dq, dk, dv])
    for j, (a, b) in enumerate(zip(*got)):
        assert torch.isfinite(a).all() or j == 1
        assert torch.equal(a, b), j
