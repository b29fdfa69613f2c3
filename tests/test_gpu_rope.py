"""Rotary positions and head norms, forward and backward, against the float64 oracle.

Bounds (element by element; U = 2^-8 is bf16's unit roundoff): every output is rounded once, U |y|. What comes before is
fp32: the angle is exact to 2^-25 of a turn (1.9e-7), sine and cosine to 1.2e-7, the mean of squares and the
reciprocal root to 12 * 2^-24 and 3 * 2^-24, the products to 6 * 2^-24; together below 2e-6 of the terms, and E = 4e-6
stands for it. The backward has two such sums: 2 E. A weight's gradient adds, in fp32, at most 64 values a lane and
48 partial sums here, 112 * 2^-24 = 7e-6 of the terms, beside the error of each: 1e-5."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import U, bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu
E = 4e-6


def _place(a, layout):
    t = dev(a)
    if layout == "heads":      # [heads][tokens][d]
        return t.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    if layout == "fused":      # a slice of a wider row
        wide = torch.full((a.shape[0], a.shape[1] + 3, a.shape[2] + 8), 7.0, dtype=t.dtype, device=t.device)
        wide[:, 1:1 + a.shape[1], :a.shape[2]] = t
        return wide[:, 1:1 + a.shape[1], :a.shape[2]]
    return t


def _run(tokens, heads, kv, d, rot, interleaved=False, norm=(True, True), start=0, base=10000.0, factor=1.0, eps=1e-6, layout="tokens",
         inplace=False, std=1.5, positions=None, stretch=1.0, trained=0):
    import bit_nf4_quantised_amd as nf4
    log(f"[rope] tokens={tokens} heads={heads}/{kv} d={d} rot={rot} interleaved={interleaved} norm={norm} start={start} {layout} inplace={inplace}")
    g = rng(tokens, heads, kv, d, rot, int(interleaved))
    rope = nf4.Rope(rot, base, interleaved, stretch=stretch, trained=trained, factor=factor)
    pos = start + np.arange(tokens) if positions is None else np.asarray(positions)
    P = torch.from_numpy(pos.astype(np.int64)).to("cuda:0")
    names = ["q", "k"] if kv else ["q"]
    H = dict(q=heads, k=kv)
    x = {n: bf16(std * g.standard_normal((tokens, H[n], d))) for n in names}
    dy = {n: bf16(g.standard_normal((tokens, H[n], d))) for n in names}
    w = {n: bf16(1 + 0.2 * g.standard_normal(d)) if norm[i] else None for i, n in enumerate(names)}
    X, DY = ({n: _place(a[n], layout) for n in names} for a in (x, dy))
    W = {n: None if w[n] is None else dev(w[n]) for n in names}
    keep = {n: X[n].clone() for n in names}
    Y = X if inplace else {n: _place(np.full(x[n].shape, 3.0), layout) for n in names}
    nf4.qlora_rope_fwd(rope, P, X["q"], X.get("k"), Y["q"], Y.get("k"), q_weight=W["q"], k_weight=W.get("k"), eps=eps)
    torch.cuda.synchronize()
    for n in names:
        want, terms = oracle.rope_fwd(x[n], pos, rope.inv_freq, interleaved, w[n], eps, factor)
        within("y " + n, Y[n], want, U * np.abs(want) + E * terms)
    DX = DY if inplace else {n: _place(np.full(x[n].shape, 3.0), layout) for n in names}
    DW = {n: None if w[n] is None else torch.full((d,), 0.5, device="cuda:0") for n in names}
    src = keep if inplace else X
    for accumulate in ([False] if inplace else [False, True]):
        nf4.qlora_rope_bwd(rope, P, DY["q"], DY.get("k"), DX["q"], DX.get("k"), q=src["q"] if norm[0] else None,
                           k=src.get("k") if norm[1] else None, q_weight=W["q"], k_weight=W.get("k"), dq_weight=DW["q"],
                           dk_weight=DW.get("k"), eps=eps, accumulate=accumulate)
    torch.cuda.synchronize()
    for n in names:
        dx, terms, dw, dwt = oracle.rope_bwd(dy[n], pos, rope.inv_freq, interleaved, x[n], w[n], eps, factor)
        within("dx " + n, DX[n], dx, U * np.abs(dx) + 2 * E * terms)
        if w[n] is not None:
            times = 1 if inplace else 2
            within("dw " + n, DW[n], times * dw, times * 1e-5 * dwt)
    if layout == "fused" and not inplace:   # what lies around the slices stays
        assert torch.all(Y["q"]._base[:, 0] == 7) and torch.all(DX["q"]._base[:, :, d:] == 7)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(8, 8), (64, 64), (64, 16), (72, 72), (80, 32), (80, 40), (96, 96), (120, 8), (128, 128), (128, 64)])
def test_head_sizes(d, rot, interleaved):
    _run(37, 4, 2, d, rot, interleaved)


@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norms_of_either(norm, interleaved):
    _run(19, 6, 3, 64, 64, interleaved, norm=norm)
    _run(19, 5, 1, 128, 96, interleaved, norm=norm)


@pytest.mark.parametrize("tokens,heads,kv", [(1, 1, 0), (1, 32, 8), (2, 3, 3), (5, 7, 0), (333, 9, 2), (1100, 1, 1)])
def test_tokens_and_heads(tokens, heads, kv):
    _run(tokens, heads, kv, 128, 128)
    _run(tokens, heads, kv, 64, 32, norm=(False, False))


def test_norm_alone():
    _run(70, 4, 2, 128, 0)
    _run(33, 2, 2, 24, 0, interleaved=True)


@pytest.mark.parametrize("start", [131071, (1 << 20) - 5, (1 << 31) - 9, -40])
def test_far_and_negative_positions(start):
    """Frequencies from one radian a position down; fp32 angles would be off by 2^-24 of the angle itself."""
    _run(9, 2, 1, 128, 128, start=start, base=500000.0, norm=(False, False))
    _run(9, 2, 1, 64, 64, True, start=start)


def test_positions_in_any_order():
    _run(8, 4, 4, 64, 64, positions=[5, 5, 0, 99, 3, 100000, 2, 1])


@pytest.mark.parametrize("layout", ["heads", "fused"])
def test_strides(layout):
    _run(40, 4, 2, 80, 80, layout=layout)
    _run(40, 4, 2, 128, 128, True, layout=layout, norm=(False, False))


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(interleaved):
    _run(50, 6, 2, 128, 128, interleaved, inplace=True)
    _run(50, 3, 3, 72, 16, interleaved, norm=(False, False), inplace=True)


def test_stretched_and_scaled():
    _run(30, 2, 2, 128, 128, start=40000, stretch=8.0, trained=8192, factor=1.2, base=500000.0)
    _run(30, 2, 2, 128, 128, start=40000, stretch=4.0)


@pytest.mark.parametrize("std", [1e-15, 1e-3, 1e15])
def test_magnitudes(std):
    _run(9, 2, 2, 64, 64, norm=(False, False), std=std)
    _run(9, 2, 2, 64, 64, std=std, eps=0.0)


def test_more_tokens_than_workgroups_start_with():
    """Groups go on to further tokens: past 2048 workgroups of 16 rows of four heads."""
    import bit_nf4_quantised_amd as nf4
    t = 40000
    g = torch.Generator(device="cuda:0").manual_seed(5)
    x = torch.randn(t, 1, 128, generator=g, device="cuda:0").to(torch.bfloat16)
    pos = torch.arange(t, device="cuda:0")
    rope, y, one = nf4.Rope(128), torch.empty_like(x), torch.empty(50, 1, 128, dtype=x.dtype, device=x.device)
    nf4.qlora_rope_fwd(rope, pos, x, None, y, None)
    dx, w, dw = torch.empty_like(x), torch.ones(128, dtype=torch.bfloat16, device=x.device), torch.empty(128, device=x.device)
    nf4.qlora_rope_bwd(rope, pos, x, None, dx, None, q=x, q_weight=w, dq_weight=dw)
    for a in (0, 32740, t - 50):        # parts give the same bits
        nf4.qlora_rope_fwd(rope, pos[a:a + 50], x[a:a + 50], None, one, None)
        assert torch.equal(one, y[a:a + 50])
        nf4.qlora_rope_bwd(rope, pos[a:a + 50], x[a:a + 50], None, one, None, q=x[a:a + 50], q_weight=w)
        assert torch.equal(one, dx[a:a + 50])
    h = host(x)
    rows = 1 + np.arange(0, t, 1)       # the weight's gradient of all tokens
    want, _, dwo, dwt = oracle.rope_bwd(h, rows - 1, rope.inv_freq, False, h, np.ones(128), 1e-6)
    # each of the 512 workgroups' lanes adds 20 values or fewer, then 16 and 512 / 16 + 16 sums: within 1e-5
    within("dw", dw, dwo, 1e-5 * dwt)
    again = torch.empty_like(dw)
    nf4.qlora_rope_bwd(rope, pos, x, None, dx, None, q=x, q_weight=w, dq_weight=again)
    assert torch.equal(dw, again)


def test_more_groups_than_the_largest_grid():
    """65536 workgroups of 32 groups take 2097152 items at a time (4 heads of a token, d <= 64), with sums of dw 4096 workgroups.
    dw: 64 values a lane, then 32 groups, 128 workgroups a slice and 32 slices, 256 * 2^-24 = 1.6e-5 of the terms, and the
    terms' own 2e-6."""
    import bit_nf4_quantised_amd as nf4
    t, h = 133000, 64
    g = torch.Generator(device="cuda:0").manual_seed(6)
    x, k = (torch.randn(t, n, 8, generator=g, device="cuda:0").to(torch.bfloat16) for n in (h, 1))
    w = torch.randn(8, generator=g, device="cuda:0").to(torch.bfloat16)
    pos, rope = torch.arange(t, device="cuda:0"), nf4.Rope(8)
    y, yk, dx, dk, dx2, dk2 = (torch.full_like(a, 3.0) for a in (x, k, x, k, x, k))
    dw, dwk = torch.zeros(8, device="cuda:0"), torch.zeros(8, device="cuda:0")
    nf4.qlora_rope_fwd(rope, pos, x, k, y, yk, q_weight=w, k_weight=w)
    nf4.qlora_rope_bwd(rope, pos, y, yk, dx, dk, q=x, k=k, q_weight=w, k_weight=w)
    nf4.qlora_rope_bwd(rope, pos, y, yk, dx2, dk2, q=x, k=k, q_weight=w, k_weight=w, dq_weight=dw, dk_weight=dwk)
    assert torch.equal(dx, dx2) and torch.equal(dk, dk2)
    for a in (0, 65500, 131060, t - 50):
        s = slice(a, a + 50)
        one, onek = torch.empty_like(x[s]), torch.empty_like(k[s])
        nf4.qlora_rope_fwd(rope, pos[s], x[s], k[s], one, onek, q_weight=w, k_weight=w)
        assert torch.equal(one, y[s]) and torch.equal(onek, yk[s])
        nf4.qlora_rope_bwd(rope, pos[s], y[s], yk[s], one, onek, q=x[s], k=k[s], q_weight=w, k_weight=w)
        assert torch.equal(one, dx[s]) and torch.equal(onek, dk[s])
    # without a rotation the weight's gradient is a plain sum
    nf4.qlora_rope_bwd(nf4.Rope(0), None, y, yk, dx, dk, q=x, k=k, q_weight=w, k_weight=w, dq_weight=dw, dk_weight=dwk)
    for d, i, got in ((y, x, dw), (yk, k, dwk)):
        i = i.double()
        terms = d.double() * i * torch.rsqrt(i.square().mean(-1, keepdim=True) + 1e-6)
        assert torch.all((got.double() - terms.sum((0, 1))).abs() <= 1.8e-5 * terms.abs().sum((0, 1)))


def test_gradient_against_differences():
    """Central differences of the framework's own forward in the direction of a perturbation: fp32-like accuracy is out of
    reach in bf16, so the loss is taken over many values: its rounding error is U times the root of the sum of squares."""
    import bit_nf4_quantised_amd as nf4
    g = torch.Generator(device="cuda:0").manual_seed(1)
    t, h, d = 64, 8, 128
    r = lambda *s: torch.randn(*s, generator=g, device="cuda:0")  # noqa: E731
    x, dy, w = r(t, h, d).bfloat16(), r(t, h, d).bfloat16(), (1 + 0.2 * r(d)).bfloat16()
    v = 0.125 * torch.sign(r(t, h, d))
    pos, rope = torch.arange(t, device="cuda:0") * 7, nf4.Rope(64)

    def loss(x):
        y = torch.empty_like(x)
        nf4.qlora_rope_fwd(rope, pos, x, None, y, None, q_weight=w)
        return (y.double() * dy.double())
    up, down = (x.float() + v).bfloat16(), (x.float() - v).bfloat16()
    step = up.double() - down.double()
    dx = torch.empty_like(x)
    nf4.qlora_rope_bwd(rope, pos, dy, None, dx, None, q=x, q_weight=w)
    lu, ld = loss(up), loss(down)
    got, want = (lu - ld).sum().item(), (dx.double() * step).sum().item()
    noise = U / 3 ** 0.5 * ((lu.square().sum() + ld.square().sum()).sqrt() + (dx.double() * step).square().sum().sqrt()).item()
    # third-order terms: x changes by 1/8, the norm's curvature is of the order of (step / |x|)^3 a value, random in sign
    assert abs(got - want) < 6 * noise + 0.125 ** 3 * (dy.double() * step).square().sum().sqrt().item()
