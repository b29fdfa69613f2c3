"""NaN in a query or in a key that it sees: o and lse are NaN for the rows concerned, on every path of the forward
(one range of keys, several, tiles of query rows with one and two groups of waves), and right for all others.
Bounds as in test_gpu_attn.py."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import U, bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu
E = 1e-4


def _packed(*lens):
    return [(sum(lens[:i]), n, sum(lens[:i]), n) for i, n in enumerate(lens)]


CASES = {
    "one range": ([(0, 1, 0, 200), (1, 3, 200, 90)], 8, 2, 128),
    "one range, small heads": ([(0, 1, 0, 200), (1, 3, 200, 90)], 8, 2, 64),
    "several ranges": ([(0, 1, 0, 9000), (1, 2, 9000, 4000)], 8, 1, 128),
    "several ranges, small heads": ([(0, 2, 0, 9000)], 6, 2, 40),
    "ranges past 64": ([(0, 1, 0, 70000)], 4, 1, 128),
    "rows split over the keys": ([(0, 128, 0, 4096)], 32, 8, 128),
    "tiles of rows, two groups": (_packed(300, 257, 311), 8, 2, 128),
    "tiles of rows": (_packed(*([130] * 20)), 16, 4, 128),
    "tiles of rows, small heads": (_packed(*([130] * 20)), 16, 16, 64),
}


@pytest.mark.parametrize("where", ["query", "key", "value"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_nan(name, where):
    import bit_nf4_quantised_amd as nf4
    seqs, heads, kv, d = CASES[name]
    log(f"[attn nan] {name}: NaN in a {where}")
    tq, tk = max(s[0] + s[1] for s in seqs), max(s[2] + s[3] for s in seqs)
    g = rng(41, tq, tk, heads, kv, d)
    q, k, v = bf16(1.5 * g.standard_normal((tq, heads, d))), bf16(g.standard_normal((tk, kv, d))), bf16(g.standard_normal((tk, kv, d)))
    want = oracle.attention(q, k, v, seqs, d ** -0.5, True, 0)
    lost = np.zeros((tq, heads), bool)        # rows whose o is NaN
    maybe = np.zeros((tq, heads), bool)       # rows of which nothing is said
    for i, (q0, nq, k0, nk) in enumerate(seqs):
        if where == "query":
            q[q0 + nq // 2, i % heads, 3] = np.nan
            lost[q0 + nq // 2, i % heads] = True
            continue
        at, head = nk - 1 - (nk // 3 if nq > 1 else nk // 5), i % kv
        if where == "key":
            k[k0 + at, head, 1] = np.nan
        else:
            v[k0 + at, head, :] = np.nan
        sees = np.arange(nq) + (nk - nq) >= at
        group = slice(head * (heads // kv), (head + 1) * (heads // kv))
        lost[q0:q0 + nq, group] = sees[:, None]
        if where == "value":
            maybe[q0:q0 + nq, group] = ~sees[:, None]
    o, lse = torch.zeros(tq, heads, d, dtype=torch.bfloat16, device="cuda:0"), torch.zeros(heads, tq, device="cuda:0")
    nf4.qlora_attn_fwd(nf4.AttnSeqs(seqs), dev(q), dev(k), dev(v), o, lse)
    torch.cuda.synchronize()
    got, got_lse, sure = host(o), host(lse).T, ~lost & ~maybe
    assert lost.any() and np.isnan(got[lost]).all()
    if where == "value":
        assert np.isfinite(got_lse).all()
    else:
        assert np.isnan(got_lse[lost]).all()
    bound = U * np.abs(want["o"]) + (U + E) * want["o_terms"]
    within("o", got[sure], want["o"][sure], bound[sure])
    w = want["lse"].T
    within("lse", got_lse[sure], w[sure], 2e-5 * (1 + np.abs(w[sure])))


def test_rows_without_keys_are_not_lost():
    """A NaN query that sees no key gives 0 and -inf like any other."""
    import bit_nf4_quantised_amd as nf4
    log("[attn nan] rows without keys")
    for seqs, heads, kv in (([(0, 200, 0, 60), (200, 40, 60, 0)], 4, 2), ([(0, 5, 0, 2), (5, 1, 2, 0)], 4, 1)):
        tq, tk = max(s[0] + s[1] for s in seqs), max(s[2] + s[3] for s in seqs)
        g = rng(42, tq)
        q, k, v = bf16(g.standard_normal((tq, heads, 64))), bf16(g.standard_normal((tk, kv, 64))), bf16(g.standard_normal((tk, kv, 64)))
        blind = np.concatenate([np.arange(nq) + (nk - nq) < 0 for _, nq, _, nk in seqs])
        q[blind] = np.nan
        o, lse = torch.ones(tq, heads, 64, dtype=torch.bfloat16, device="cuda:0"), torch.zeros(heads, tq, device="cuda:0")
        nf4.qlora_attn_fwd(nf4.AttnSeqs(seqs), dev(q), dev(k), dev(v), o, lse)
        torch.cuda.synchronize()
        assert not host(o)[blind].any() and (host(lse)[:, blind] == -np.inf).all()
        assert np.isfinite(host(o)[~blind]).all() and np.isfinite(host(lse)[:, ~blind]).all()
