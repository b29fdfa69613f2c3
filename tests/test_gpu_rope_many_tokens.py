"""The rotation over more items than the largest grid takes at a time, with rows of 16 lanes (d over 64): groups of queries and of
keys go on to further tokens, forward, backward and with the weights' gradients.

Of 450000 tokens, 5 query heads (two items a token, one where gradients of weights are summed) and one key head, the queries' 54613
workgroups of 16 groups take 873808 of 900000 items at a time and the keys' 10923 174768 of 450000; with sums the queries' 3413
take 54608 of 450000 and the keys' 683 10928. A weight's gradient adds 9 items of 5 heads a lane (keys: 42 of one), 16 groups, 27
workgroups a slice, 16 and 8 slices: 112 * 2^-24 = 6.7e-6 of the terms, beside 4e-6 for the terms themselves: 1.1e-5."""
import pytest
import torch

from gpu_helpers import log

pytestmark = pytest.mark.gpu
TOKENS, HEADS, KV, D = 450000, 5, 1, 128


def _dw(dy, x, pos, freq, eps):
    """The weight's gradient of rows [tokens, heads, D] in float64, and its terms' magnitudes."""
    total, terms = (torch.zeros(D, dtype=torch.float64, device="cuda:0") for _ in range(2))
    half = D // 2
    for a in range(0, dy.shape[0], 25000):
        s = slice(a, a + 25000)
        angle = pos[s].double()[:, None, None] * freq
        c, n = torch.cos(angle), torch.sin(angle)
        g, xx = dy[s].double(), x[s].double()
        back = torch.cat([g[..., :half] * c + g[..., half:] * n, g[..., half:] * c - g[..., :half] * n], -1)
        mag = (g[..., :half].abs() + g[..., half:].abs()).repeat(1, 1, 2)
        unit = xx * torch.rsqrt(xx.square().mean(-1, keepdim=True) + eps)
        total += (back * unit).sum((0, 1))
        terms += (mag * unit.abs()).sum((0, 1))
    return total, terms


def test_groups_go_on_to_further_tokens():
    import bit_nf4_quantised_amd as nf4
    log("[rope] 450000 tokens")
    gen = torch.Generator(device="cuda:0").manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    q, k, gq, gk, wq, wk = r(TOKENS, HEADS, D), r(TOKENS, KV, D), r(TOKENS, HEADS, D), r(TOKENS, KV, D), r(D), r(D)
    pos, rope, eps = torch.arange(TOKENS, device="cuda:0"), nf4.Rope(D, 500000.0), 1e-6
    new = lambda: [torch.full_like(t, 3.0) for t in (q, k)]  # noqa: E731
    (y, yk), (dx, dk), (dx2, dk2), dw = new(), new(), new(), torch.full((2, D), 5.0, device="cuda:0")
    kw = dict(q=q, k=k, q_weight=wq, k_weight=wk)
    nf4.qlora_rope_fwd(rope, pos, q, k, y, yk, q_weight=wq, k_weight=wk)
    nf4.qlora_rope_bwd(rope, pos, gq, gk, dx, dk, **kw)
    nf4.qlora_rope_bwd(rope, pos, gq, gk, dx2, dk2, dq_weight=dw[0], dk_weight=dw[1], **kw)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dk, dk2)
    # parts, of few enough tokens for one item a group, give the same bits
    n = 5000
    one, onek = torch.empty_like(q[:n]), torch.empty_like(k[:n])
    for a in range(0, TOKENS, n):
        s = slice(a, a + n)
        nf4.qlora_rope_fwd(rope, pos[s], q[s], k[s], one, onek, q_weight=wq, k_weight=wk)
        assert torch.equal(one, y[s]) and torch.equal(onek, yk[s]), a
        nf4.qlora_rope_bwd(rope, pos[s], gq[s], gk[s], one, onek, q=q[s], k=k[s], q_weight=wq, k_weight=wk)
        assert torch.equal(one, dx[s]) and torch.equal(onek, dk[s]), a
    freq = torch.tensor(rope.inv_freq, dtype=torch.float64, device="cuda:0")
    for i, (g, x) in enumerate(((gq, q), (gk, k))):
        want, terms = _dw(g, x, pos, freq, eps)
        assert torch.all((dw[i].double() - want).abs() <= 1.1e-5 * terms)
    del q, k, gq, gk, y, yk, dx, dk, dx2, dk2
    torch.cuda.empty_cache()
