"""How callers use the rotation, the 4-bit cache and the attention over it: after one another in training and in serving, from
a HIP graph, on another stream, from two threads, over a cache past 32-bit offsets."""
import os
import sys
import threading

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import gpu_dequant, log
from layer_helpers import U, bf16, dev, host, rng, within

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def test_training_chain_against_the_oracle():
    """Heads normed and rotated, attention, and all of it backward. A tensor's rounding to bf16 puts 1.7e-3 of its norm on it
    (error up to 2^-8 of a value, uniform in the logarithm); attention's probabilities as much again. q and k pass two roundings to
    the output (4e-3 with the probabilities'), the gradients up to five and the ill-conditioned difference in dS: 5e-3 sqrt(5)."""
    import bit_nf4_quantised_amd as nf4
    heads, kv, d, lens = 8, 2, 128, [150, 1, 77]
    M, g = sum(lens), rng(41)
    x = {n: bf16(1.5 * g.standard_normal((M, h, d))) for n, h in (("q", heads), ("k", kv), ("v", kv))}
    w = {n: bf16(1 + 0.2 * g.standard_normal(d)) for n in ("q", "k")}
    do = bf16(g.standard_normal((M, heads, d)))
    pos = np.concatenate([np.arange(n) for n in lens])
    rope, P = nf4.Rope(d), torch.from_numpy(pos).to("cuda:0")
    X, W = {n: dev(a) for n, a in x.items()}, {n: dev(a) for n, a in w.items()}
    q, k = torch.empty_like(X["q"]), torch.empty_like(X["k"])
    nf4.qlora_rope_fwd(rope, P, X["q"], X["k"], q, k, q_weight=W["q"], k_weight=W["k"])
    seqs = nf4.AttnSeqs.packed(lens)
    o, lse = torch.empty_like(q), torch.empty(heads, M, device="cuda:0")
    nf4.qlora_attn_fwd(seqs, q, k, X["v"], o, lse)
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, X["v"]))
    nf4.qlora_attn_bwd(seqs, q, k, X["v"], o, lse, dev(do), dq, dk, dv)
    dw = {n: torch.empty(d, device="cuda:0") for n in ("q", "k")}
    nf4.qlora_rope_bwd(rope, P, dq, dk, dq, dk, q=X["q"], k=X["k"], q_weight=W["q"], k_weight=W["k"], dq_weight=dw["q"], dk_weight=dw["k"])
    r = {n: oracle.rope_fwd(x[n], pos, rope.inv_freq, False, w[n], 1e-6)[0] for n in ("q", "k")}
    at = np.cumsum([0] + lens)
    t = oracle.attention(r["q"], r["k"], x["v"], [(a, n, a, n) for a, n in zip(at, lens)], d ** -0.5, True, 0, do=do)
    assert _rel(host(o), t["o"]) < 5e-3 * 2 ** 0.5 and _rel(host(dv), t["dv"]) < 5e-3 * 5 ** 0.5
    for n, got in (("q", dq), ("k", dk)):
        dx, _, dwn, _ = oracle.rope_bwd(t["d" + n], pos, rope.inv_freq, False, x[n], w[n], 1e-6)
        assert _rel(host(got), dx) < 5e-3 * 5 ** 0.5 and _rel(host(dw[n]), dwn) < 5e-3 * 5 ** 0.5, n


@pytest.mark.parametrize("book", ["nf4", "fp4", "int4"])
def test_serving_chain_against_the_oracle(book):
    """A prompt in chunks, then single tokens: rotated, written, attended to. The cache has to hold exactly what the rotated keys
    and the values quantise to, and the attention is over that."""
    import bit_nf4_quantised_amd as nf4
    heads, kv, d, room = 6, 2, 80, 128
    g, rope = rng(42), nf4.Rope(32, interleaved=True)
    k4, v4 = (nf4.empty_kv4(2 * room, kv, d, codebook=book) for _ in range(2))
    held = {n: np.zeros((2 * room, kv, d)) for n in ("k", "v")}
    have = [0, 0]
    for nq in (40, 33, 1, 1, 7):
        x = {n: bf16(g.standard_normal((2 * nq, h, d))) for n, h in (("q", heads), ("k", kv), ("v", kv))}
        pos = np.concatenate([np.arange(n, n + nq) for n in have])
        seqs = [(i * nq, nq, i * room, have[i] + nq) for i in range(2)]
        batch = nf4.AttnSeqs(seqs)
        q, k, v = (dev(x[n]) for n in ("q", "k", "v"))
        nf4.qlora_rope_fwd(rope, torch.from_numpy(pos).to("cuda:0"), q, k, q, k)
        nf4.qlora_kv4_write(batch, k, v, k4, v4)
        o, lse = torch.empty_like(q), torch.empty(heads, 2 * nq, device="cuda:0")
        nf4.qlora_attn_kv4_fwd(batch, q, k4, v4, o, lse)
        have = [n + nq for n in have]
        qr, kr = host(q), host(k)     # the rotation's own rounding is checked elsewhere
        for i in range(2):
            to = slice(i * room + have[i] - nq, i * room + have[i])
            for n, new in (("k", kr), ("v", x["v"])):
                held[n][to] = oracle.kv4_values(*oracle.kv4(new[i * nq:(i + 1) * nq], book), d, book)
        want = oracle.attention(qr, held["k"], held["v"], seqs, d ** -0.5, True, 0)
        within("o", o, want["o"], U * np.abs(want["o"]) + (U + 1e-4) * want["o_terms"])
        within("lse", lse, want["lse"], 2e-5 * (1 + np.abs(want["lse"])))
    every = nf4.AttnSeqs([(sum(have[:i]), have[i], i * room, have[i]) for i in range(2)])
    kb, vb = (torch.empty(sum(have), kv, d, dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
    nf4.qlora_kv4_read(every, k4, v4, kb, vb)
    keep = np.concatenate([np.arange(i * room, i * room + have[i]) for i in range(2)])
    assert np.array_equal(host(kb), held["k"][keep]) and np.array_equal(host(vb), held["v"][keep])


def _step(batch=3, room=700, heads=8, kv=2, d=128, lengths=(5, 333, 650), seed=9):
    """A decoding step: rotate, write, attend; and the backward of the rotation with its weights' gradients. Returns the step, its
    outputs and its inputs."""
    import bit_nf4_quantised_amd as nf4
    gen = torch.Generator(device="cuda:0").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    rope = nf4.Rope(d)
    k4, v4 = nf4.empty_kv4(batch * room, kv, d), nf4.empty_kv4(batch * room, kv, d)
    whole = nf4.AttnSeqs([(0, batch * room, 0, batch * room)])
    nf4.qlora_kv4_write(whole, r(batch * room, kv, d), r(batch * room, kv, d), k4, v4)
    seqs = nf4.AttnSeqs([(i, 1, i * room, n) for i, n in enumerate(lengths)])
    q, k, v, pos = r(batch, heads, d), r(batch, kv, d), r(batch, kv, d), torch.tensor([n - 1 for n in lengths], device="cuda:0")
    w = 1 + 0.1 * r(d)
    new = lambda t, *s: torch.zeros(*(s or t.shape), dtype=t.dtype, device="cuda:0")  # noqa: E731
    qr, kr, o, lse = new(q), new(k), new(q), torch.zeros(heads, batch, device="cuda:0")
    dq, dk, dw = new(q), new(k), torch.zeros(d, device="cuda:0")
    kb, vb = new(k), new(v)

    def step():
        nf4.qlora_rope_fwd(rope, pos, q, k, qr, kr, q_weight=w, k_weight=w)
        nf4.qlora_kv4_write(seqs, kr, v, k4, v4)
        nf4.qlora_attn_kv4_fwd(seqs, qr, k4, v4, o, lse)
        nf4.qlora_kv4_read(seqs, k4, v4, kb, vb)
        nf4.qlora_rope_bwd(rope, pos, o, kb, dq, dk, q=q, k=k, q_weight=w, k_weight=w, dq_weight=dw)
    return step, [qr, kr, o, lse, kb, vb, dq, dk, dw, k4.codes, v4.absmax], [q, k, v, pos]


def _renew(ins, seed):
    gen = torch.Generator(device="cuda:0").manual_seed(seed)
    for t in ins[:3]:
        t.copy_(torch.randn(t.shape, generator=gen, device="cuda:0"))
    ins[3].add_(seed)


@pytest.mark.parametrize("lengths,room", [((5, 333, 650), 700), ((9, 2, 40), 64)])
def test_a_step_replays_from_a_graph(lengths, room):
    log(f"[heads use] graph {lengths}")
    step, outs, ins = _step(lengths=lengths, room=room)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2, 3):
        _renew(ins, seed)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs[:9]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (seed, i)


def test_two_graphs_share_a_workspace():
    """Graphs of attention over long caches, whose ranges go through one workspace, replayed in turn."""
    import bit_nf4_quantised_amd as nf4
    gen = torch.Generator(device="cuda:0").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    n, kv, d = 3000, 2, 64
    k4, v4 = nf4.empty_kv4(n, kv, d, codebook="fp4"), nf4.empty_kv4(n, kv, d, codebook="fp4")
    nf4.qlora_kv4_write(nf4.AttnSeqs([(0, n, 0, n)]), r(n, kv, d), r(n, kv, d), k4, v4)
    ws = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda:0")
    calls = []
    for nk, nq in ((3000, 1), (1500, 4)):
        q, seqs = r(nq, 4, d), nf4.AttnSeqs([(0, nq, 0, nk)])
        o, want = torch.zeros_like(q), torch.zeros_like(q)
        nf4.qlora_attn_kv4_fwd(seqs, q, k4, v4, want)
        assert seqs.workspace_bytes(q, k4) > 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nf4.qlora_attn_kv4_fwd(seqs, q, k4, v4, o, ws=ws)
        calls.append((graph, o, want, q))      # the graph reads q again
    for _ in range(3):
        for graph, o, want, _ in calls:
            o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want)


def test_on_another_stream():
    import bit_nf4_quantised_amd as nf4
    step, outs, ins = _step()
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs[:9]:
        t.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # a stream that is named: the workspace comes from its pool
    q, k4, v4 = outs[0], nf4.empty_kv4(4000, 2, 128), nf4.empty_kv4(4000, 2, 128)
    for c in (k4, v4):
        c.codes.random_(0, 256)
        c.absmax.fill_(1.0)
    seqs = nf4.AttnSeqs([(0, 3, 0, 4000)])
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    nf4.qlora_attn_kv4_fwd(seqs, q, k4, v4, a)
    torch.cuda.synchronize()
    nf4.qlora_attn_kv4_fwd(seqs, q, k4, v4, b, stream=side)
    side.synchronize()
    assert torch.equal(a, b)


def test_two_threads_share_a_rope_and_a_batch():
    import bit_nf4_quantised_amd as nf4
    rope, seqs = nf4.Rope(64), nf4.AttnSeqs([(0, 2, 0, 900)])
    pos = torch.tensor([898, 899], device="cuda:0")
    wrong = []

    def work(heads, book, seed):
        gen = torch.Generator(device="cuda:0").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda:0").to(torch.bfloat16)  # noqa: E731
        with torch.cuda.stream(torch.cuda.Stream()):
            q, k, v = r(2, heads, 64), r(900, 2, 64), r(900, 2, 64)
            k4, v4 = nf4.empty_kv4(900, 2, 64, codebook=book), nf4.empty_kv4(900, 2, 64, codebook=book)
            nf4.qlora_kv4_write(nf4.AttnSeqs([(0, 900, 0, 900)]), k, v, k4, v4)
            first = None
            for i in range(60):
                t, o = torch.empty_like(q), torch.empty_like(q)
                nf4.qlora_rope_fwd(rope, pos, q, None, t, None)
                nf4.qlora_attn_kv4_fwd(seqs, t, k4, v4, o)
                torch.cuda.current_stream().synchronize()
                first = o if first is None else first
                if not torch.equal(o, first):
                    wrong.append((heads, i))
                    return
    threads = [threading.Thread(target=work, args=a) for a in ((4, "nf4", 1), (16, "fp4", 2))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_cache_past_32_bit_offsets():
    """Sequences at the end of a cache of 4.5 GiB of codes, heads first and tokens first: as over a small cache."""
    import bit_nf4_quantised_amd as nf4
    gen = torch.Generator(device="cuda:0").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    kv, d, n, tokens = 9, 128, 700, 8 << 20
    q, k, v = r(3, 18, d), r(n, kv, d), r(n, kv, d)
    small = nf4.empty_kv4(n, kv, d), nf4.empty_kv4(n, kv, d)
    nf4.qlora_kv4_write(nf4.AttnSeqs([(0, n, 0, n)]), k, v, *small)
    want, o = torch.empty_like(q), torch.empty_like(q)
    nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs([(0, 3, 0, n)]), q, *small, want)
    for heads_first in (True, False):
        if heads_first:
            big = [nf4.empty_kv4(tokens, kv, d) for _ in range(2)]
        else:
            big = [nf4.Kv4(torch.empty(tokens, kv, 4, 16, dtype=torch.uint8, device="cuda:0"),
                           torch.empty(tokens, kv, 4, dtype=torch.bfloat16, device="cuda:0"), d) for _ in range(2)]
        nf4.qlora_kv4_write(nf4.AttnSeqs([(0, n, tokens - n, n)]), k, v, *big)
        nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs([(0, 3, tokens - n, n)]), q, *big, o)
        assert torch.equal(o, want)
        del big


@pytest.mark.parametrize("nq", [1, 4, 9, 40, 70])
@pytest.mark.parametrize("d", [64, 128])
def test_every_form_agrees_with_the_attention_over_bf16(nq, d):
    """Row counts for each of the kernels, long ranges and short: against qlora_attn_fwd over the cache read back. Both round
    probabilities and outputs once: their difference is within twice each one's bound."""
    import bit_nf4_quantised_amd as nf4
    heads, kv = 16, 4
    for nks in ([2500, 130, 700], [16000], [200] * 20):
        gen = torch.Generator(device="cuda:0").manual_seed(nq + d)
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda:0").to(torch.bfloat16)  # noqa: E731
        total, B = sum(nks), len(nks)
        k4, v4 = nf4.empty_kv4(total, kv, d, codebook="int4"), nf4.empty_kv4(total, kv, d, codebook="int4")
        kb, vb = r(total, kv, d), r(total, kv, d)
        every = nf4.AttnSeqs([(0, total, 0, total)])
        nf4.qlora_kv4_write(every, kb, vb, k4, v4)
        nf4.qlora_kv4_read(every, k4, v4, kb, vb)
        q = r(B * nq, heads, d)
        seqs = nf4.AttnSeqs([(i * nq, nq, sum(nks[:i]), n) for i, n in enumerate(nks)])
        o4, ob, terms = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
        l4, lb = (torch.empty(heads, B * nq, device="cuda:0") for _ in range(2))
        nf4.qlora_attn_kv4_fwd(seqs, q, k4, v4, o4, l4)
        nf4.qlora_attn_fwd(seqs, q, kb, vb, ob, lb)
        nf4.qlora_attn_fwd(seqs, q, kb, vb.abs(), terms)
        t, a = host(terms), host(ob)
        assert np.all(np.abs(host(o4) - a) <= 2 * (U * np.abs(a) + (U + 1e-4) * t) * (1 + U))
        assert np.all(np.abs(host(l4) - host(lb)) <= 4e-5 * (1 + np.abs(host(lb))))
        again = torch.empty_like(q)
        nf4.qlora_attn_kv4_fwd(seqs, q, k4, v4, again)
        assert torch.equal(o4, again)


def test_example_block_with_positions_against_the_oracle():
    """The example with head norms and a rotation, forward and backward. The bounds are those of the block without them with one
    rounding more forward and two more backward: 5e-3 sqrt(6), and 5e-3 sqrt(11) + 6e-3 for the 8-bit checkpoints."""
    import bit_nf4_quantised_amd as nf4
    from attention_block import EPS, AttentionBlock
    log("[heads use] example block")
    rope = nf4.Rope(48, interleaved=True)
    blk = AttentionBlock(hidden=256, heads=4, kv_heads=2, d=64, rope=rope)
    lens, d, s = [40, 1, 23], 64, blk.scale
    M, g = sum(lens), rng(77)
    x, res, dout, dh = (bf16(g.standard_normal((M, 256))) for _ in range(4))
    pos = np.concatenate([np.arange(n) for n in lens])
    out, h = blk.forward(dev(x), dev(res), nf4.AttnSeqs.packed(lens), torch.from_numpy(pos).to("cuda:0"))
    dx = blk.backward(dev(dout), dev(dh))
    torch.cuda.synchronize()
    W = [oracle.f32_from_bf16_bits(gpu_dequant(w)).astype(np.float64).reshape(w.N, w.K) for w in blk.weights]
    A, B = [host(t) for t in blk.A], [host(t) for t in blk.B]
    w, wq, wk = host(blk.norm_weight), host(blk.q_weight), host(blk.k_weight)
    hh, n, rstd = oracle.rmsnorm(x, res, w, EPS)
    q, k, v = (n @ W[i].T + s * (n @ A[i].T) @ B[i].T for i in range(3))
    q, k, v = q.reshape(M, 4, d), k.reshape(M, 2, d), v.reshape(M, 2, d)
    qr, kr = (oracle.rope_fwd(t, pos, rope.inv_freq, True, wt, EPS)[0] for t, wt in ((q, wq), (k, wk)))
    seqs = [(sum(lens[:i]), m, sum(lens[:i]), m) for i, m in enumerate(lens)]
    a = oracle.attention(qr, kr, v, seqs, d ** -0.5, True, 0)["o"].reshape(M, -1)
    want = a @ W[3].T + s * (a @ A[3].T) @ B[3].T
    assert _rel(host(out), want) < 5e-3 * 6 ** 0.5
    bwd = lambda i, y, inp: (y @ W[i] + s * (y @ B[i]) @ A[i], s * (y @ B[i]).T @ inp, s * y.T @ (inp @ A[i].T))  # noqa: E731
    da = bwd(3, dout, a)[0]
    t = oracle.attention(qr, kr, v, seqs, d ** -0.5, True, 0, do=da.reshape(M, 4, d))
    grads = [oracle.rope_bwd(t["d" + m], pos, rope.inv_freq, True, y, wt, EPS)[0] for m, y, wt in (("q", q, wq), ("k", k, wk))] + [t["dv"]]
    parts = [bwd(i, y.reshape(M, -1), n) for i, y in enumerate(grads)]
    bound = 5e-3 * 11 ** 0.5 + 6e-3
    assert _rel(host(dx), oracle.rmsnorm_bwd(sum(p[0] for p in parts), dh, hh, w, rstd)[0]) < bound
    for i, (_, dA, dB) in enumerate(parts):
        assert _rel(host(blk.grads[2 * i]), dA) < bound and _rel(host(blk.grads[2 * i + 1]), dB) < bound, i


def test_example_decodes_over_both_caches():
    """Token by token over a bf16 cache as the packed forward; over a 4-bit cache as the same attention over what the cache
    holds: the block's own bf16 decoding with its cache replaced by the values read back."""
    import bit_nf4_quantised_amd as nf4
    from attention_block import AttentionBlock
    log("[heads use] example decoding")
    blk = AttentionBlock(rope=nf4.Rope(64))
    g, n, room = rng(78), 20, 32
    x, res = dev(bf16(g.standard_normal((n, 512)))), dev(bf16(g.standard_normal((n, 512))))
    out, _ = blk.forward(x, res, nf4.AttnSeqs.packed([n]), torch.arange(n, device="cuda:0"))
    kc = torch.zeros(1, room, blk.kv_heads, blk.d, dtype=torch.bfloat16, device="cuda:0")
    vc = torch.zeros_like(kc)
    one = torch.cat([blk.decode(x[i:i + 1], res[i:i + 1], kc, vc, [i]) for i in range(n)])
    assert _rel(host(one), host(out)) < 1.2e-2
    k4, v4 = nf4.empty_kv4(room, blk.kv_heads, blk.d), nf4.empty_kv4(room, blk.kv_heads, blk.d)
    four, like = [], []
    for i in range(n):
        four.append(blk.decode(x[i:i + 1], res[i:i + 1], k4, v4, [i]))
        kb, vb = torch.zeros(i + 1, blk.kv_heads, blk.d, dtype=torch.bfloat16, device="cuda:0"), torch.zeros(i + 1, blk.kv_heads, blk.d, dtype=torch.bfloat16, device="cuda:0")
        nf4.qlora_kv4_read(nf4.AttnSeqs([(0, i + 1, 0, i + 1)]), k4, v4, kb, vb)
        seen = {}
        real = nf4.qlora_attn_fwd
        try:      # the same step, with the attention over the values read back
            nf4.qlora_attn_fwd = lambda seqs, q, k, v, o, **kw: (seen.update(q=q), real(nf4.AttnSeqs([(0, 1, 0, i + 1)]), q, kb, vb, o))[1]
            like.append(blk.decode(x[i:i + 1], res[i:i + 1], kc, vc, [i]))
        finally:
            nf4.qlora_attn_fwd = real
    four, like = host(torch.cat(four)), host(torch.cat(like))
    assert _rel(four, like) < 5e-3 * 2 ** 0.5      # the probabilities' and the output's roundings differ


def test_calls_with_nothing_to_do():
    """No tokens, no sequences, sequences without new tokens, an empty cache: nothing is written and nothing fails."""
    import bit_nf4_quantised_amd as nf4
    e, ek, some = (torch.empty(*s, dtype=torch.bfloat16, device="cuda:0") for s in ((0, 4, 64), (0, 2, 64), (3, 4, 64)))
    some.fill_(3.0)
    pos, rope = torch.empty(0, dtype=torch.int64, device="cuda:0"), nf4.Rope(64)
    w, dw = torch.ones(64, dtype=torch.bfloat16, device="cuda:0"), torch.full((64,), 2.0, device="cuda:0")
    nf4.qlora_rope_fwd(rope, pos, e, ek, e, ek)
    nf4.qlora_rope_bwd(rope, pos, e, ek, e, ek, q=e, q_weight=w, dq_weight=dw, accumulate=True)
    none, full = [nf4.empty_kv4(0, 2, 64) for _ in range(2)], [nf4.empty_kv4(9, 2, 64) for _ in range(2)]
    for t in full:
        t.codes.fill_(7)
        t.absmax.fill_(1.0)
    nf4.qlora_kv4_write(nf4.AttnSeqs([]), ek, ek, *none)
    nf4.qlora_kv4_write(nf4.AttnSeqs([(0, 0, 0, 9), (0, 0, 4, 0)]), ek, ek, *full)
    nf4.qlora_kv4_read(nf4.AttnSeqs([(0, 0, 0, 9)]), *full, ek, ek)
    o, lse = torch.full_like(some, 5.0), torch.full((4, 3), 5.0, device="cuda:0")
    nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs([]), some, *full, o, lse)
    nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs([(0, 0, 0, 9)]), some, *full, o, lse)
    nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs([]), e, *none, torch.empty_like(e))
    torch.cuda.synchronize()
    assert torch.all(o == 5) and torch.all(lse == 5) and torch.all(full[0].codes == 7) and torch.all(full[1].absmax == 1) and torch.all(dw == 2)
    nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs([(1, 2, 0, 0)]), some, *none, o, lse)      # rows, but no keys
    assert torch.all(o[0] == 5) and torch.all(o[1:] == 0) and torch.all(torch.isneginf(lse[:, 1:])) and torch.all(lse[:, 0] == 5)


def test_heads_that_are_one_in_memory():
    """Inputs whose heads are broadcast (head stride 0), and a query that is every head's: as their copies."""
    import bit_nf4_quantised_amd as nf4
    gen = torch.Generator(device="cuda:0").manual_seed(3)
    one = torch.randn(40, 1, 96, generator=gen, device="cuda:0").to(torch.bfloat16)
    q, k = one.expand(-1, 8, -1), one.expand(-1, 4, -1)
    qc, kc = q.contiguous(), k.contiguous()
    pos, rope = torch.arange(40, device="cuda:0") * 3, nf4.Rope(96)
    w = torch.randn(96, generator=gen, device="cuda:0").to(torch.bfloat16)
    got, want = [[torch.empty_like(t) for t in (qc, kc, qc, kc)] + [torch.empty(96, device="cuda:0") for _ in range(2)] for _ in range(2)]
    for (a, b), o in (((q, k), got), ((qc, kc), want)):
        nf4.qlora_rope_fwd(rope, pos, a, b, o[0], o[1], q_weight=w)
        nf4.qlora_rope_bwd(rope, pos, a, b, o[2], o[3], q=a, k=b, q_weight=w, k_weight=w, dq_weight=o[4], dk_weight=o[5])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    seqs, caches = nf4.AttnSeqs([(0, 40, 0, 40)]), [[nf4.empty_kv4(40, 4, 96) for _ in range(2)] for _ in range(2)]
    outs = [torch.empty_like(qc) for _ in range(2)]
    for (a, b), c, o in (((q, k), caches[0], outs[0]), ((qc, kc), caches[1], outs[1])):
        nf4.qlora_kv4_write(seqs, b, b, *c)
        nf4.qlora_attn_kv4_fwd(seqs, a, *c, o)
    assert torch.equal(outs[0], outs[1])
    assert all(torch.equal(x.codes, y.codes) and torch.equal(x.absmax, y.absmax) for x, y in zip(*caches))


def test_sequences_that_share_keys():
    """Several continuations of one prompt: ranges that start together, lie in one another, and are the same twice. Against each
    alone, whose ranges may be others: both round probabilities (the terms) and outputs once, so they differ by twice that."""
    import bit_nf4_quantised_amd as nf4
    gen = torch.Generator(device="cuda:0").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    k4, v4 = nf4.empty_kv4(3000, 2, 128), nf4.empty_kv4(3000, 2, 128)
    nf4.qlora_kv4_write(nf4.AttnSeqs([(0, 3000, 0, 3000)]), r(3000, 2, 128), r(3000, 2, 128), k4, v4)
    keys = [(0, 3000), (0, 3000), (0, 2000), (500, 1700), (2999, 1)]
    q = r(5, 16, 128)
    q[1] = q[0]
    o, terms, alone = torch.empty_like(q), torch.empty_like(q), torch.empty(1, 16, 128, dtype=q.dtype, device=q.device)
    seqs = nf4.AttnSeqs([(i, 1, k0, n) for i, (k0, n) in enumerate(keys)])
    nf4.qlora_attn_kv4_fwd(seqs, q, k4, v4, o)
    kb, vb = r(3000, 2, 128), r(3000, 2, 128)
    nf4.qlora_kv4_read(nf4.AttnSeqs([(0, 3000, 0, 3000)]), k4, v4, kb, vb)
    nf4.qlora_attn_fwd(seqs, q, kb, vb.abs(), terms)
    assert torch.equal(o[0], o[1])
    for i, (k0, n) in enumerate(keys):
        nf4.qlora_attn_kv4_fwd(nf4.AttnSeqs([(0, 1, k0, n)]), q[i:i + 1], k4, v4, alone)
        a, b, t = alone[0].float(), o[i].float(), terms[i].float()
        assert torch.all((a - b).abs() <= 2 * (U * b.abs() + (U + 1e-4) * t) * (1 + U))


def test_a_training_step_replays_from_a_graph():
    """Forward and backward of normed and rotated heads with attention between them, the weights' gradients added to: three
    replays against three eager steps, bit for bit."""
    import bit_nf4_quantised_amd as nf4
    gen = torch.Generator(device="cuda:0").manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    lens, heads, kv, d = [300, 1, 99], 8, 2, 80
    M = sum(lens)
    q, k, v, do, wq, wk = r(M, heads, d), r(M, kv, d), r(M, kv, d), r(M, heads, d), r(d), r(d)
    pos, rope, seqs = torch.cat([torch.arange(n) for n in lens]).to("cuda:0"), nf4.Rope(32, interleaved=True), nf4.AttnSeqs.packed(lens)
    acc = torch.zeros(2, d, device="cuda:0")
    outs = [torch.empty_like(t) for t in (q, k, q, q, k, k, q, k)] + [acc]

    def step():
        y, yk, o, dy, dyk, dv, dx, dxk, _ = outs
        lse = torch.empty(heads, M, device="cuda:0")
        nf4.qlora_rope_fwd(rope, pos, q, k, y, yk, q_weight=wq, k_weight=wk)
        nf4.qlora_attn_fwd(seqs, y, yk, v, o, lse)
        nf4.qlora_attn_bwd(seqs, y, yk, v, o, lse, do, dy, dyk, dv)
        nf4.qlora_rope_bwd(rope, pos, dy, dyk, dx, dxk, q=q, k=k, q_weight=wq, k_weight=wk, dq_weight=acc[0], dk_weight=acc[1], accumulate=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2, 3):
        gen.manual_seed(seed)
        for t in (q, k, v, do):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda:0"))
        start = acc.clone()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs[:8]:
            t.zero_()
        acc.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (seed, i)


def test_tensors_of_another_device_than_the_current_one_are_refused(monkeypatch):
    """Before anything is launched; the current device is made to look like another one."""
    import bit_nf4_quantised_amd as nf4
    q, k = (torch.zeros(4, h, 64, dtype=torch.bfloat16, device="cuda:0") for h in (4, 2))
    k4, v4 = (nf4.empty_kv4(8, 2, 64, device="cuda:0") for _ in range(2))
    pos, rope, seqs = torch.zeros(4, dtype=torch.int64, device="cuda:0"), nf4.Rope(64), nf4.AttnSeqs([(0, 4, 0, 4)])
    calls = [lambda: nf4.qlora_rope_fwd(rope, pos, q, k, q, k), lambda: nf4.qlora_rope_bwd(rope, pos, q, k, q, k),
             lambda: nf4.qlora_kv4_write(seqs, k, k, k4, v4), lambda: nf4.qlora_kv4_read(seqs, k4, v4, k, torch.empty_like(k)),
             lambda: nf4.qlora_attn_kv4_fwd(seqs, q, k4, v4, torch.empty_like(q), torch.empty(4, 4, device="cuda:0"))]
    for f in calls:
        f()
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for f in calls:
        with pytest.raises(ValueError, match="current device"):
            f()
