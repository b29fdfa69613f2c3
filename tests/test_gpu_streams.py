"""Calls that are given a stream, without a workspace of the caller's, while the current stream allocates and
writes memory: results equal, bit for bit, those of the same calls with nothing beside them."""
import pytest
import torch

from gpu_helpers import log

pytestmark = pytest.mark.gpu


def _calls():
    """(name, call(stream), its outputs, workspace bytes) of every call that takes a workspace."""
    import bit_nf4_quantised_amd as nf4
    g = torch.Generator(device="cuda:0").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    new = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda:0")  # noqa: E731
    M, N, K, R, f32 = 900, 128, 512, 16, torch.float32
    W = nf4.quantize_weight(r(N, K).float())
    x, dy, A, B, u = r(M, K), r(M, N), r(R, K), r(N, R), r(M, R).float()
    x8 = nf4.empty_act8(M, K)
    nf4.qlora_act8_pack(x, x8)
    y, y2, u2, dx, dA, dB = new(M, N), new(M, N), new(M, R, dtype=f32), new(M, K), new(R, K, dtype=f32), new(N, R, dtype=f32)
    dx8, dA8, dB8 = new(M, K), new(R, K, dtype=f32), new(N, R, dtype=f32)
    w, rstd, dn, dw = r(K), r(M).float().abs(), new(M, K), new(K, dtype=f32)
    q, k, v, do = r(M, 16, 128), r(M, 4, 128), r(M, 4, 128), r(M, 16, 128)
    seqs, one = nf4.AttnSeqs.packed([500, 400]), nf4.AttnSeqs([(0, 1, 0, 9000)])
    o, lse, dq, dk, dv = new(M, 16, 128), new(16, M, dtype=f32), new(M, 16, 128), new(M, 4, 128), new(M, 4, 128)
    nf4.qlora_attn_fwd(seqs, q, k, v, o, lse)
    kc, vc, o1 = r(9000, 2, 128), r(9000, 2, 128), new(1, 16, 128)
    wide = r(1024, 1024).float()
    qw = []
    torch.cuda.synchronize()

    def quantise(s):
        qw[:] = [nf4.quantize_weight(wide, stream=s)]
    sizes = nf4.qlora_workspace_bytes(M, N, K, R), nf4.qlora_workspace_bytes_act8(M, [N], K, R)
    return [
        ("linear_fwd", lambda s: nf4.qlora_linear_fwd(W, x, A, B, 2.0, y, u2, stream=s), lambda: [y, u2], sizes[0]),
        ("linear_fwd_group", lambda s: nf4.qlora_linear_fwd_group([W], x, [A], [B], 2.0, [y2], stream=s), lambda: [y2], sizes[0]),
        ("linear_bwd", lambda s: nf4.qlora_linear_bwd(W, x, dy, A, B, 2.0, u, dx, dA, dB, stream=s),
         lambda: [dx, dA, dB], sizes[0]),
        ("linear_bwd_act8", lambda s: nf4.qlora_linear_bwd_act8([W], x8, [dy], [A], [B], 2.0, [u], [dx8], [dA8], [dB8], stream=s),
         lambda: [dx8, dA8, dB8], sizes[1]),
        ("rmsnorm_bwd", lambda s: nf4.qlora_rmsnorm_bwd(x, x, w, rstd, dn, dw=dw, stream=s), lambda: [dn, dw],
         int(nf4.lib.qlora_rmsnorm_workspace_bytes(M, K))),
        ("attn_fwd", lambda s: nf4.qlora_attn_fwd(one, q[:1], kc, vc, o1, stream=s), lambda: [o1],
         one.workspace_bytes(q[:1], kc)),
        ("attn_bwd", lambda s: nf4.qlora_attn_bwd(seqs, q, k, v, o, lse, do, dq, dk, dv, stream=s), lambda: [dq, dk, dv],
         seqs.workspace_bytes(q, k, True)),
        ("quantize_weight", quantise, lambda: [qw[0].packed, qw[0].scale_q, qw[0].scale_c2], 4 * wide.numel() // 64),
    ]


def _busy():
    a = torch.randn(4096, 4096, device="cuda:0")
    for _ in range(8):
        a = a @ a * 1e-2
    return a


def test_current_stream_writes_beside_a_call():
    """The call's kernels wait on the side stream while the current one allocates blocks of the workspace's size and
    fills them."""
    side = torch.cuda.Stream()
    for name, call, outs, nbytes in _calls():
        log(f"[streams] {name}, workspace of {nbytes} bytes")
        assert nbytes > 0
        call(None)
        torch.cuda.synchronize()
        want = [t.clone() for t in outs()]
        for t in outs():
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            _busy()
        call(side)
        junk = [torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda:0") for _ in range(3)]
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(want, outs())):
            assert torch.equal(a, b), (name, j)
        del junk


def test_a_call_beside_what_the_current_stream_reads():
    """The current stream's kernels wait, their input already freed there; a call on the side stream must not get
    that memory."""
    side = torch.cuda.Stream()
    for name, call, _, nbytes in _calls():
        log(f"[streams] {name} beside a reader")
        torch.cuda.synchronize()
        read = torch.zeros(3, dtype=torch.int64, device="cuda:0")
        held = [torch.full((nbytes,), 5, dtype=torch.uint8, device="cuda:0") for _ in range(3)]
        _busy()
        for i, t in enumerate(held):
            read[i] = (t == 5).all()
        del held, t
        call(side)
        torch.cuda.synchronize()
        assert read.tolist() == [1, 1, 1], name
