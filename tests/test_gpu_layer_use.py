"""How callers use attention, the norm and the 8-bit checkpoints: from a HIP graph, on another stream, over
a cache past 32-bit offsets, behind a window. Results are compared bit for bit with the same call in its
plainest use, which the other tests compare with the oracle."""
import pytest
import torch

from gpu_helpers import log

pytestmark = pytest.mark.gpu


def _rand(seed):
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda:0").to(torch.bfloat16)


def _layer(M, K, lens, seed=1):
    """A step of every call over M rows; returns (step, its outputs, its inputs)."""
    import bit_nf4_quantised_amd as nf4
    r = _rand(seed)
    heads, kv, d = 8, 2, 64
    x, res, dy, w = r(M, K), r(M, K), r(M, K), r(K)
    q, k, v, do = r(M, heads, d), r(M, kv, d), r(M, kv, d), r(M, heads, d)
    W = nf4.quantize_weight(r(64, K).float())
    A, B, dl = r(16, K), r(64, 16), r(M, 64)
    new = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda:0")  # noqa: E731
    h, y, rstd, y8, back = new(M, K), new(M, K), new(M, dtype=torch.float32), nf4.empty_act8(M, K, "cuda:0"), new(M, K)
    dxn, dw = new(M, K), new(K, dtype=torch.float32)
    o, lse = new(M, heads, d), new(heads, M, dtype=torch.float32)
    dq, dk, dv = new(M, heads, d), new(M, kv, d), new(M, kv, d)
    o1 = new(1, heads, d)
    yl, u, dxl = new(M, 64), new(M, 16, dtype=torch.float32), new(M, K)
    dA, dB = new(16, K, dtype=torch.float32), new(64, 16, dtype=torch.float32)
    seqs, one = nf4.AttnSeqs.packed(lens), nf4.AttnSeqs([(0, 1, 0, M)])

    def step():
        nf4.qlora_rmsnorm_fwd(x, w, 1e-5, y, residual=res, h=h, rstd=rstd, act8=y8)
        nf4.qlora_act8_unpack(y8, back)
        nf4.qlora_linear_fwd(W, y, A, B, 2.0, yl, u)
        nf4.qlora_attn_fwd(seqs, q, k, v, o, lse)
        nf4.qlora_attn_fwd(one, q[:1], k, v, o1)
        nf4.qlora_attn_bwd(seqs, q, k, v, o, lse, do, dq, dk, dv)
        nf4.qlora_linear_bwd_act8([W], y8, [dl], [A], [B], 2.0, [u], [dxl], [dA], [dB])
        nf4.qlora_rmsnorm_bwd(dy, h, w, rstd, dxn, dw=dw)
    return step, [h, y, rstd, y8.codes, y8.absmax, back, yl, u, o, lse, o1, dq, dk, dv, dxl, dA, dB, dxn, dw], [x, q, v, do, dl]


@pytest.mark.parametrize("M,lens", [(900, [500, 300, 100]), (40, [40])])
def test_a_step_replays_from_a_graph(M, lens):
    log(f"[layer use] graph of {M} rows")
    step, outs, ins = _layer(M, 512, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for t in ins:   # other values every time
            t.copy_(torch.roll(t, 1, 0))
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        step()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(replayed, outs)):
            assert torch.equal(a, b), (i, j)


def test_on_another_stream():
    """The calls run on the current stream: what is queued there before them is what they read."""
    log("[layer use] another stream")
    step, outs, ins = _layer(900, 512, [500, 300, 100], seed=2)
    step()
    torch.cuda.synchronize()
    want, right = [t.clone() for t in outs], [t.clone() for t in ins]
    for t in ins + outs:
        t.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        busy = torch.randn(4096, 4096, device="cuda:0")
        for _ in range(8):
            busy = busy @ busy * 1e-2   # the copies below wait behind this
        for t, v in zip(ins, right):
            t.copy_(v)
        step()
    side.synchronize()
    for j, (a, b) in enumerate(zip(want, outs)):
        assert torch.equal(a, b), j


@pytest.mark.parametrize("nq", [1, 300])
def test_cache_past_32_bit_offsets(nq):
    """Sequences at the end of a cache of 5.4 GB a tensor (2.7 G elements) against the same in a small one."""
    import bit_nf4_quantised_amd as nf4
    log(f"[layer use] large cache, {nq} queries")
    kv, d, heads, n = 8, 128, 16, 700
    total = (1 << 31) // (kv * d) + (1 << 19)
    r = _rand(3)
    k, v, q, do = r(n, kv, d), r(n, kv, d), r(nq, heads, d), r(nq, heads, d)
    big = [torch.empty(total, kv, d, dtype=torch.bfloat16, device="cuda:0") for _ in range(2)]
    big[0][total - n:].copy_(k)
    big[1][total - n:].copy_(v)
    grads = [torch.empty(total, kv, d, dtype=torch.bfloat16, device="cuda:0") for _ in range(2)]
    got = []
    for kk, vv, dk, dv, at in ((k, v, torch.empty_like(k), torch.empty_like(v), 0), (*big, *grads, total - n)):
        seqs = nf4.AttnSeqs([(0, nq, at, n)])
        o, lse, dq = torch.empty_like(q), torch.empty(heads, nq, device="cuda:0"), torch.empty_like(q)
        nf4.qlora_attn_fwd(seqs, q, kk, vv, o, lse)
        nf4.qlora_attn_bwd(seqs, q, kk, vv, o, lse, do, dq, dk, dv)
        torch.cuda.synchronize()
        got.append([o, lse, dq, dk[at:].clone(), dv[at:].clone()])
    for j, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), j


def test_tokens_past_32_bit_offsets():
    """[heads][tokens][d] tensors whose head stride puts the last head past 2^32 bytes."""
    import bit_nf4_quantised_amd as nf4
    log("[layer use] large head stride")
    heads, d, n, room = 4, 64, 150, 12 << 20
    r = _rand(4)
    small = [r(n, heads, d) for _ in range(4)]
    far = []
    for t in small:
        w = torch.empty(heads, room, d, dtype=torch.bfloat16, device="cuda:0")
        w[:, :n].copy_(t.permute(1, 0, 2))
        far.append(w.permute(1, 0, 2)[:n])
    got = []
    for q, k, v, do in (small, far):
        seqs = nf4.AttnSeqs.packed([100, 50])
        o, lse = torch.empty_like(small[0]), torch.empty(heads, n, device="cuda:0")
        dq, dk, dv = (torch.empty_like(small[0]) for _ in range(3))
        nf4.qlora_attn_fwd(seqs, q, k, v, o, lse)
        nf4.qlora_attn_bwd(seqs, q, k, v, o, lse, do, dq, dk, dv)
        torch.cuda.synchronize()
        got.append([o, lse, dq, dk, dv])
    for j, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), j


@pytest.mark.parametrize("nq", [1, 9, 700])
def test_keys_behind_the_window_may_hold_anything(nq):
    """With a window the keys that no query of the call sees are given up (a rolling cache); NaN there
    changes nothing, and their gradients are zero."""
    import bit_nf4_quantised_amd as nf4
    log(f"[layer use] {nq} queries behind a window")
    heads, kv, d, n, window = 64, 8, 128, 1500, 100
    r = _rand(5)
    q, k, v, do = r(nq, heads, d), r(n, kv, d), r(n, kv, d), r(nq, heads, d)
    gone = n - nq - window + 1
    k2, v2 = k.clone(), v.clone()
    k2[:gone] = float("nan")
    v2[:gone] = float("nan")
    got = []
    for kk, vv in ((k, v), (k2, v2)):
        seqs = nf4.AttnSeqs([(0, nq, 0, n)], window=window)
        o, lse, dq = torch.empty_like(q), torch.empty(heads, nq, device="cuda:0"), torch.empty_like(q)
        dk, dv = torch.full_like(k, 3.0), torch.full_like(v, 3.0)
        nf4.qlora_attn_fwd(seqs, q, kk, vv, o, lse)
        nf4.qlora_attn_bwd(seqs, q, kk, vv, o, lse, do, dq, dk, dv)
        torch.cuda.synchronize()
        assert not dk[:gone].any() and not dv[:gone].any()
        got.append([o, lse, dq, dk, dv])
    for j, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), j
