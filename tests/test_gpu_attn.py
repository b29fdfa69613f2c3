"""Attention, forward and backward, against the float64 oracle.

Bounds (element by element, from the roundings the kernels make; U = 2^-8 is bf16's unit roundoff):
o rounds every probability once (relative U) and the result once: U |o| + (U + E) sum_j P |v|, and dv
likewise. dS is rounded once and its delta is formed from the rounded o, so dq and dk lie within
U |dq| + (2 U + E) times the sum of the absolute terms P (|do.v| + sum |do o|) |k|. E = 1e-4 covers
fp32 scores, sums and the hardware exponential (arguments below 50 in magnitude: 50 * 2^-24 * 8).
lse is fp32: 2e-5 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import log
from layer_helpers import U, bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu
E = 1e-4


def _run(name, seqs, heads, kv, d, causal=True, window=0, tq=None, tk=None, backward=True, scale=None, std=1.5,
         layout="tokens", poison=False):
    import bit_nf4_quantised_amd as nf4
    log(f"[attn] {name}: seqs={seqs[:8]}{'...' if len(seqs) > 8 else ''} heads={heads}/{kv} d={d} causal={causal} window={window} {layout}")
    tq = max([s[0] + s[1] for s in seqs], default=0) if tq is None else tq
    tk = max([s[2] + s[3] for s in seqs], default=0) if tk is None else tk
    g = rng(len(seqs), heads, kv, d, int(causal), window, tq, tk)
    q, do = bf16(std * g.standard_normal((tq, heads, d))), bf16(g.standard_normal((tq, heads, d)))
    k, v = bf16(g.standard_normal((tk, kv, d))), bf16(g.standard_normal((tk, kv, d)))
    scale = d ** -0.5 if scale is None else scale
    want = oracle.attention(q, k, v, seqs, scale, causal, window, do=do if backward else None)
    if poison:   # rows outside every sequence are never read
        inq, ink = np.zeros(tq, bool), np.zeros(tk, bool)
        for q0, nq, k0, nk in seqs:
            inq[q0:q0 + nq] = True
            ink[k0:k0 + nk] = True
        for x, inside in ((q, inq), (do, inq), (k, ink), (v, ink)):
            x[~inside] = np.nan

    def place(a):
        t = dev(a)
        if layout == "heads":      # [heads][tokens][d]
            return t.permute(1, 0, 2).contiguous().permute(1, 0, 2)
        if layout == "fused":      # a slice of a wider row
            wide = torch.full((a.shape[0], a.shape[1] + 3, d + 8), 7.0, dtype=t.dtype, device=t.device)
            wide[:, 1:1 + a.shape[1], :d] = t
            return wide[:, 1:1 + a.shape[1], :d]
        return t
    Q, K, V, DO = place(q), place(k), place(v), place(do)
    O = place(np.full(q.shape, 3.0))
    lse = torch.full((heads, tq), 5.0, dtype=torch.float32, device="cuda:0")
    batch = nf4.AttnSeqs(seqs, causal=causal, window=window)
    nf4.qlora_attn_fwd(batch, Q, K, V, O, lse, scale=scale)
    torch.cuda.synchronize()
    rows = np.zeros(tq, bool)
    for q0, nq, _, _ in seqs:
        rows[q0:q0 + nq] = True
    assert np.all(host(O)[~rows] == 3.0) and np.all(host(lse)[:, ~rows] == 5.0), "a row outside the sequences was written"
    within("o", host(O)[rows], want["o"][rows], (U * np.abs(want["o"]) + (U + E) * want["o_terms"])[rows])
    within("lse", host(lse)[:, rows], want["lse"][:, rows], 2e-5 * (1 + np.abs(np.where(np.isfinite(want["lse"]), want["lse"], 0)))[:, rows])
    if not backward:
        return
    DQ, DK, DV = place(np.full(q.shape, 3.0)), place(np.full(k.shape, 3.0)), place(np.full(k.shape, 3.0))
    nf4.qlora_attn_bwd(batch, Q, K, V, O, lse, DO, DQ, DK, DV, scale=scale)
    torch.cuda.synchronize()
    keys = np.zeros(tk, bool)
    for _, _, k0, nk in seqs:
        keys[k0:k0 + nk] = True
    assert np.all(host(DQ)[~rows] == 3.0) and np.all(host(DK)[~keys] == 3.0) and np.all(host(DV)[~keys] == 3.0)
    for name_, t, inside, f in (("dq", DQ, rows, 2), ("dk", DK, keys, 2), ("dv", DV, keys, 1)):
        b = U * np.abs(want[name_]) + (f * U + E) * want[name_ + "_terms"]
        within(name_, host(t)[inside], want[name_][inside], b[inside])


def _packed(*lens):
    out, at = [], 0
    for n in lens:
        out.append((at, n, at, n))
        at += n
    return out


@pytest.mark.parametrize("lens", [(1,), (2, 1), (31, 32, 33), (64,), (127, 1, 129), (300, 5), (513,)])
@pytest.mark.parametrize("d", [64, 128])
def test_packed_causal(lens, d):
    _run("packed", _packed(*lens), 4, 2, d)


@pytest.mark.parametrize("d", [8, 24, 72, 80, 96, 120])
def test_head_sizes(d):
    _run("head size", _packed(70, 3), 2, 1, d)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (6, 2), (8, 8), (16, 8), (12, 1), (40, 8)])
def test_shared_heads(heads, kv):
    _run("heads", _packed(97, 40), heads, kv, 64)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 64, 65, 200, 1 << 40])
def test_window(window):
    _run("window", _packed(260, 33), 2, 2, 64, window=window)
    _run("window, whole sequence ahead", _packed(150), 2, 1, 128, causal=False, window=window)


@pytest.mark.parametrize("d,heads,kv,causal,window", [(128, 64, 8, True, 0), (128, 33, 11, True, 70), (64, 96, 2, True, 0),
                                                      (96, 64, 64, False, 0), (80, 48, 16, False, 130)])
def test_enough_rows_to_fill_the_gpu(d, heads, kv, causal, window):
    _run("many workgroups", _packed(300, 1, 130, 64) + [(495, 150, 495, 40), (645, 20, 535, 333)], heads, kv, d, causal=causal,
         window=window)
    _run("many workgroups, strided", _packed(257, 200), 128, 8, d, causal=causal, window=window, layout="heads")


@pytest.mark.parametrize("d", [80, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 40)])
def test_many_equal_sequences(d, causal, window):
    # enough equal work for the backward's form of two waves a SIMD
    _run("equal sequences", _packed(*([100, 64, 129, 33] * 4)), 64, 64, d, causal=causal, window=window)
    _run("equal sequences, shared heads", _packed(*([130] * 20)), 16, 4, d, causal=causal, window=window)


def test_not_causal():
    _run("not causal", _packed(129, 64, 1), 4, 4, 64, causal=False)
    _run("cross", [(0, 70, 0, 33), (70, 3, 33, 200)], 4, 2, 128, causal=False)


def test_rows_that_see_nothing():
    # more queries than keys: the first rows have no key; lengths of zero on either side
    _run("empty rows", [(0, 200, 0, 60), (200, 40, 60, 0), (240, 0, 60, 50), (240, 70, 110, 1)], 4, 2, 64)
    _run("empty rows, split", [(0, 5, 0, 2), (5, 1, 2, 0)], 4, 1, 128)
    _run("nothing at all", [], 2, 1, 64, tq=4, tk=4)


def test_rows_outside_the_sequences_stay_untouched_and_unread():
    _run("gaps", [(3, 20, 5, 20), (30, 100, 40, 140)], 4, 2, 64, tq=140, tk=200, poison=True)
    _run("gaps", [(1, 1, 7, 300), (3, 1, 400, 33)], 8, 2, 128, tq=6, tk=500, poison=True, backward=False)


@pytest.mark.parametrize("layout", ["heads", "fused"])
def test_strides(layout):
    _run("strides", _packed(150, 20), 4, 2, 64, layout=layout)
    _run("strides", _packed(40), 3, 3, 40, layout=layout)
    _run("strides, one token", [(0, 1, 0, 700)], 8, 2, 128, layout=layout)


@pytest.mark.parametrize("nk", [1, 2, 31, 33, 127, 128, 129, 1000, 2049])
@pytest.mark.parametrize("heads,kv,d", [(8, 2, 128), (4, 4, 64), (40, 1, 80)])
def test_one_token_over_a_cache(nk, heads, kv, d):
    _run("decode", [(0, 1, 0, nk), (1, 1, 0, max(1, nk // 2)), (2, 1, nk, 5)], heads, kv, d, backward=False)


@pytest.mark.parametrize("nq", [2, 7, 17, 40])
@pytest.mark.parametrize("window", [0, 50])
def test_few_tokens_over_a_cache(nq, window):
    _run("few tokens", [(0, nq, 0, 900), (nq, nq, 900, 1), (2 * nq, nq, 901, nq + 300)], 8, 2, 128, window=window,
         backward=False)


def test_prompt_on_top_of_a_cache():
    _run("chunk", [(0, 260, 0, 900), (260, 130, 900, 131)], 16, 8, 64)


def test_large_and_peaked_scores():
    # scores up to about 60: the running maximum is raised many times
    _run("peaked", _packed(300), 2, 1, 64, std=20.0, backward=False)
    _run("scale", _packed(100), 2, 1, 64, scale=0.01)


def test_more_sequences_than_a_launch_takes():
    g = rng(99)
    _run("many", _packed(*[int(n) for n in g.integers(1, 9, 150)]), 2, 1, 64)
    _run("many, split", [(i, 1, 9 * i, int(n)) for i, n in enumerate(g.integers(0, 9, 130))], 4, 1, 64, tk=1300,
         backward=False)


def test_results_repeat_bit_for_bit():
    import bit_nf4_quantised_amd as nf4
    g = torch.Generator(device="cuda:0").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    q, k, v, do = r(700, 8, 128), r(700, 2, 128), r(700, 2, 128), r(700, 8, 128)
    seqs = nf4.AttnSeqs.packed([500, 200])
    first = None
    for _ in range(3):
        o, lse = torch.empty_like(q), torch.empty(8, 700, device="cuda:0")
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        nf4.qlora_attn_fwd(seqs, q, k, v, o, lse)
        nf4.qlora_attn_bwd(seqs, q, k, v, o, lse, do, dq, dk, dv)
        torch.cuda.synchronize()
        now = [t.clone() for t in (o, lse, dq, dk, dv)]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_gradient_against_differences_of_the_forward():
    """dq, dk, dv of f = sum(o * do) against central differences along random directions, the steps
    representable in bf16. Each f carries the forward's rounding error, at most its bound summed over
    the elements (as a root of squares: the roundings are independent), and the difference of third
    order in the step is below 1e-2 of the result for these steps of 2^-3."""
    import bit_nf4_quantised_amd as nf4
    log("[attn] differences")
    g = rng(123)
    seqs = nf4.AttnSeqs.packed([40, 24])
    x = [bf16(np.round(g.standard_normal(s) * 4) / 4) for s in ((64, 4, 64), (64, 2, 64), (64, 2, 64))]
    do = bf16(g.standard_normal((64, 4, 64)))

    def f(q, k, v):
        o = torch.empty(64, 4, 64, dtype=torch.bfloat16, device="cuda:0")
        nf4.qlora_attn_fwd(seqs, dev(q), dev(k), dev(v), o, lse)
        return (host(o) * do).sum(), o
    lse = torch.empty(4, 64, device="cuda:0")
    _, o = f(*x)
    grads = [torch.empty(a.shape, dtype=torch.bfloat16, device="cuda:0") for a in x]
    nf4.qlora_attn_bwd(seqs, *[dev(a) for a in x], o, lse, dev(do), *grads)
    noise = 2 * np.sqrt(((U * np.abs(do) * (np.abs(host(o)) + 1.0)) ** 2).sum())
    for at, name in enumerate(("dq", "dk", "dv")):
        direction = np.sign(host(grads[at])) * 2.0 ** -3   # along the gradient: the largest difference
        hi, lo = list(x), list(x)
        hi[at], lo[at] = x[at] + direction, x[at] - direction
        diff = (f(*hi)[0] - f(*lo)[0]) / 2
        want = (host(grads[at]) * direction).sum()
        third = {"dq": 0.05, "dk": 0.05, "dv": 0.0}[name] * abs(want)
        assert abs(diff - want) <= noise + third + 2 * U * abs(want), (name, diff, want, noise)


@pytest.mark.parametrize("d,window,causal", [(128, 0, True), (80, 0, True), (64, 0, True), (128, 40, True), (128, 0, False),
                                             (64, 150, False)])
def test_rows_shared_by_two_groups_of_waves(d, window, causal):
    # a few hundred rows a sequence: too few workgroups to fill the GPU, too many rows for the key split
    _run("two groups", _packed(300, 257, 311, 290), 8, 2, d, causal=causal, window=window)
    _run("two groups, caches and short sequences", [(0, 500, 0, 700), (500, 130, 700, 131), (630, 1, 831, 90), (631, 7, 921, 7),
                                                    (638, 33, 928, 20)], 16, 8, d, causal=causal, window=window)


@pytest.mark.parametrize("seqs", [[(0, 40, 0, 40)], [(0, 1, 0, 700)], [(0, 300, 0, 300), (300, 300, 300, 300), (600, 300, 600, 300)]])
def test_vanishing_scale(seqs):
    # every score rounds to zero: o is the mean of the values that a row sees. Forward only: dq and dk carry the
    # factor 1e-39, below bf16's normal numbers (2^-126), where its rounding is not relative and the bounds above
    # do not hold
    _run("vanishing scale", seqs, 8, 2, 128, scale=1e-39, backward=False)
