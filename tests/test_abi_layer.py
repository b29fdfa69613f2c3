"""Refusals of the attention, norm and 8-bit checkpoint calls: the documented status, before any GPU
work. No kernel runs here."""
import ctypes

import pytest

q = pytest.importorskip("bit_nf4_quantised_amd")
lib = q.lib
FAKE, ODD = 0x100000, 0x100004
OK, NULL, SHAPE, ALIGN, RANK, WS = q.NF4_OK, q.NF4_ERR_NULL, q.NF4_ERR_SHAPE, q.NF4_ERR_ALIGN, q.NF4_ERR_RANK, q.NF4_ERR_WORKSPACE


def test_act8_refusals():
    for call, args in ((lib.qlora_act8_pack, lambda n, a, b, c: (a, n, b, c, None)),
                       (lib.qlora_act8_unpack, lambda n, a, b, c: (a, b, n, c, None))):
        assert call(*args(0, None, None, None)) == OK
        assert call(*args(-64, FAKE, FAKE, FAKE)) == SHAPE and call(*args(65, FAKE, FAKE, FAKE)) == SHAPE
        assert call(*args(1 << 43, FAKE, FAKE, FAKE)) == SHAPE
        for k in range(3):
            ptrs = [FAKE] * 3
            ptrs[k] = None
            assert call(*args(64, *ptrs)) == NULL
            ptrs[k] = ODD
            assert call(*args(64, *ptrs)) == ALIGN


def _norm(M=4, K=64, eps=1e-5, x=FAKE, res=None, w=FAKE, h=None, y=FAKE, rstd=None, y8=None):
    return lib.qlora_rmsnorm_fwd(x, res, w, M, K, eps, h, y, rstd, y8, None)


def test_norm_refusals():
    assert _norm(M=0, x=None) == OK
    for bad in (dict(M=-1), dict(K=0), dict(K=12), dict(K=16392), dict(M=1 << 31), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf"))):
        assert _norm(**bad) == SHAPE, bad
    c8 = q.CAct8(FAKE, FAKE)
    assert _norm(K=72, y8=ctypes.byref(c8)) == SHAPE       # a checkpoint needs whole blocks
    assert _norm(y8=ctypes.byref(q.CAct8(None, FAKE))) == NULL
    assert _norm(y8=ctypes.byref(q.CAct8(FAKE, ODD))) == ALIGN
    for k in ("x", "w", "y"):
        assert _norm(**{k: None}) == NULL
    for k in ("x", "res", "w", "h", "y", "rstd"):
        assert _norm(**{k: ODD}) == ALIGN


def _norm_bwd(M=4, K=64, dy=FAKE, dh=None, h=FAKE, w=FAKE, rstd=FAKE, dx=FAKE, dw=None, ws=None, ws_bytes=0):
    return lib.qlora_rmsnorm_bwd(dy, dh, h, w, rstd, M, K, dx, dw, 0, ws, ws_bytes, None)


def test_norm_backward_refusals():
    need = lib.qlora_rmsnorm_workspace_bytes(4, 64)
    assert need >= 64 * 4 and lib.qlora_rmsnorm_workspace_bytes(4, 65) == 0
    assert _norm_bwd(M=0, dy=None) == OK
    assert _norm_bwd(K=9) == SHAPE
    for k in ("dy", "h", "w", "rstd", "dx"):
        assert _norm_bwd(**{k: None}) == NULL
    for k in ("dy", "dh", "h", "w", "rstd", "dx", "dw", "ws"):
        assert _norm_bwd(**{k: ODD}) == ALIGN
    assert _norm_bwd(dw=FAKE) == WS and _norm_bwd(dw=FAKE, ws=FAKE, ws_bytes=need - 1) == WS


def _arr(*v):
    return (ctypes.c_void_p * 4)(*v)


def test_backward_from_a_checkpoint_refusals():
    W = q.CNF4Weight(FAKE, FAKE, FAKE, 64, 128)
    wp = _arr(ctypes.addressof(W))
    c8 = q.CAct8(FAKE, FAKE)
    n = (ctypes.c_int64 * 1)(64)
    need = lib.qlora_workspace_bytes_act8(1, n, 8, 128, 16)
    assert need > 0 and lib.qlora_workspace_bytes_act8(1, n, 8, 100, 16) == 0
    assert lib.qlora_workspace_bytes_act8(5, n, 8, 128, 16) == 0

    def call(count=1, x8=c8, M=8, r=16, dy=_arr(FAKE), dA=_arr(FAKE), ws=FAKE, ws_bytes=need):
        return lib.qlora_linear_bwd_act8(count, wp, None if x8 is None else ctypes.byref(x8), dy, M, _arr(FAKE), _arr(FAKE),
                                         r, 1.0, _arr(FAKE), None, dA, _arr(FAKE), 0, ws, ws_bytes, None)
    assert call(M=0) == OK
    assert call(count=0) == SHAPE and call(count=5) == SHAPE and call(M=-1) == SHAPE
    assert call(r=8) == RANK
    assert call(x8=None) == NULL and call(x8=q.CAct8(None, FAKE)) == NULL and call(x8=q.CAct8(FAKE, None)) == NULL
    assert call(x8=q.CAct8(ODD, FAKE)) == ALIGN and call(x8=q.CAct8(FAKE, ODD)) == ALIGN
    assert call(dy=_arr(None)) == NULL and call(dA=_arr(ODD)) == ALIGN
    assert call(ws=None) == WS and call(ws_bytes=need - 1) == WS


def _cfg(heads=4, kv=2, d=64, causal=1, window=0, scale=0.125, tq=100, tk=100):
    return q.CAttnConfig(heads, kv, d, causal, window, scale, tq, tk)


def _seqs(*s):
    flat = [v for one in s for v in one]
    return (ctypes.c_int64 * max(4, len(flat)))(*flat)


def _t(data=FAKE, token=256, head=64):
    return q.CAttnTensor(data, token, head)


def _fwd(cfg=None, seqs=((0, 10, 0, 10),), lse=None, ws=FAKE, ws_bytes=1 << 30, **t):
    cfg = _cfg() if cfg is None else cfg
    a = {k: t.get(k, _t()) for k in ("q", "k", "v", "o")}
    return lib.qlora_attn_fwd(ctypes.byref(cfg), len(seqs), _seqs(*seqs), *[ctypes.byref(a[k]) for k in ("q", "k", "v", "o")],
                              lse, ws, ws_bytes, None)


def _bwd(cfg=None, seqs=((0, 10, 0, 10),), lse=FAKE, ws=FAKE, ws_bytes=1 << 30, **t):
    cfg = _cfg() if cfg is None else cfg
    a = {k: t.get(k, _t()) for k in ("q", "k", "v", "o", "do", "dq", "dk", "dv")}
    r = {k: ctypes.byref(v) for k, v in a.items()}
    return lib.qlora_attn_bwd(ctypes.byref(cfg), len(seqs), _seqs(*seqs), r["q"], r["k"], r["v"], r["o"], lse, r["do"],
                              r["dq"], r["dk"], r["dv"], ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_attention_refusals(call):
    assert call(seqs=()) == OK
    for bad in (dict(kv=0), dict(heads=3), dict(heads=0, kv=1), dict(d=12), dict(d=0), dict(d=136), dict(window=-1),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(tq=-1),
                dict(tk=1 << 41)):
        assert call(cfg=_cfg(**bad)) == SHAPE, bad
    for bad in (((0, -1, 0, 5),), ((0, 101, 0, 5),), ((91, 10, 0, 5),), ((0, 5, 96, 5),), ((-1, 5, 0, 5),), ((0, 5, -1, 5),),
                ((0, 10, 0, 10), (9, 5, 10, 5)), ((20, 5, 0, 5), (0, 5, 5, 5))):   # query ranges overlap, or out of order
        assert call(seqs=bad) == SHAPE, bad
    for name in ("q", "k", "v", "o"):
        for bad in (_t(token=60), _t(token=252), _t(head=60), _t(token=1 << 22), _t(head=-64)):
            assert call(**{name: bad}) == SHAPE, (name, bad)
        assert call(**{name: _t(data=None)}) == NULL and call(**{name: _t(data=ODD)}) == ALIGN
    out = "o" if call is _fwd else "dk"
    assert call(**{out: _t(token=64, head=64)}) == SHAPE         # rows of an output overlap
    assert call(lse=ODD) == ALIGN and call(ws=ODD) == ALIGN
    assert lib.qlora_attn_fwd(None, 0, None, None, None, None, None, None, None, 0, None) == NULL


def test_attention_workspace():
    cfg = _cfg(heads=8, kv=2, d=128, tq=1, tk=9000)
    s = _seqs((0, 1, 0, 9000))
    need = lib.qlora_attn_workspace_bytes(ctypes.byref(cfg), 1, s, 0)
    assert need > 0
    t = _t(token=1024, head=128)
    one = dict(cfg=cfg, seqs=((0, 1, 0, 9000),), q=t, k=t, v=t, o=t)
    assert _fwd(ws=None, ws_bytes=0, **one) == WS and _fwd(ws_bytes=need // 2, **one) == WS
    assert lib.qlora_attn_workspace_bytes(ctypes.byref(_cfg(d=7)), 1, s, 0) == 0
    # key ranges may be shared by the forward's sequences, not by the backward's
    shared = _seqs((0, 10, 0, 10), (10, 10, 0, 10))
    assert lib.qlora_attn_workspace_bytes(ctypes.byref(_cfg()), 2, shared, 1) == 0
    assert _bwd(seqs=((0, 10, 0, 10), (10, 10, 0, 10))) == SHAPE
    assert _bwd(ws=None, ws_bytes=0) == WS
    assert _bwd(lse=None) == NULL


def test_binding_refusals():
    import torch
    with pytest.raises(ValueError):
        q.AttnSeqs([(0, 1, 2)])
    a = torch.zeros(4, 2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.qlora_attn_fwd(q.AttnSeqs.packed([4]), a, a, a, a)          # not on the GPU
    with pytest.raises(TypeError):
        q.qlora_rmsnorm_fwd(a[0].float(), a[0, 0], 1e-5, a[0])        # float32 activations
    with pytest.raises(ValueError):
        q.qlora_rmsnorm_fwd(a[0], a[0, 0, :4], 1e-5, a[0])            # weight of another size
    with pytest.raises(ValueError):
        q.Act8(torch.zeros(2, 64, dtype=torch.int8), torch.zeros(1, 1, dtype=torch.bfloat16), 2, 64).c_struct()
