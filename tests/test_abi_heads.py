"""Refusals of the rotation, the 4-bit cache and the attention over it: the documented status, before any GPU work; and what
the binding refuses or marshals. No kernel runs here."""
import ctypes
import math

import pytest
import torch

q = pytest.importorskip("bit_nf4_quantised_amd")
lib = q.lib
FAKE, ODD = 0x100000, 0x100004
OK, NULL, SHAPE, ALIGN, WS = q.NF4_OK, q.NF4_ERR_NULL, q.NF4_ERR_SHAPE, q.NF4_ERR_ALIGN, q.NF4_ERR_WORKSPACE


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _t(data=FAKE, token=4096, head=128):
    return q.CAttnTensor(data, token, head)


FREQ = (ctypes.c_double * 64)(*[10000.0 ** (-i / 64) for i in range(64)])


def _rope(heads=8, kv=2, d=128, rot=128, eps=1e-6, factor=1.0, tokens=4, freq=FREQ, pos=FAKE, tq=_t(), tk=_t(), qw=None, kw=None,
          qo=_t(), ko=_t()):
    cfg = q.CRopeConfig(heads, kv, d, rot, 0, eps, factor, tokens)
    return lib.qlora_rope_fwd(ctypes.byref(cfg), freq, pos, _ref(tq), _ref(tk), qw, kw, _ref(qo), _ref(ko), None)


def test_rope_refusals():
    assert _rope(tokens=0, tq=_t(None), tk=_t(None), qo=_t(None), ko=_t(None), pos=None, freq=None) == OK
    nan, inf = float("nan"), float("inf")
    for bad in (dict(heads=0), dict(heads=65536), dict(kv=-1), dict(kv=65536), dict(d=0), dict(d=136), dict(d=12), dict(rot=-8),
                dict(rot=12), dict(rot=136), dict(d=64, rot=72), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(factor=nan),
                dict(factor=inf), dict(tokens=-1), dict(tokens=(1 << 40) + 1), dict(tq=_t(token=64)), dict(tq=_t(token=4100)),
                dict(qo=_t(token=128, head=64)), dict(ko=_t(head=0))):
        assert _rope(**bad) == SHAPE, bad
    for bad in ([inf] + [0.0] * 63, [0.0] * 63 + [nan]):
        assert _rope(freq=(ctypes.c_double * 64)(*bad)) == SHAPE
    for bad in (dict(freq=None), dict(pos=None), dict(tq=None), dict(tk=None), dict(qo=None), dict(ko=None), dict(tq=_t(None)),
                dict(ko=_t(None))):
        assert _rope(**bad) == NULL, bad
    for bad in (dict(tq=_t(ODD)), dict(tk=_t(ODD)), dict(qo=_t(ODD)), dict(qw=ODD), dict(kw=ODD), dict(pos=ODD)):
        assert _rope(**bad) == ALIGN, bad
    cfg = q.CRopeConfig(8, 2, 128, 128, 0, 1e-6, 1.0, 4)
    assert lib.qlora_rope_fwd(None, FREQ, FAKE, _ref(_t()), None, None, None, _ref(_t()), None, None) == NULL
    assert lib.qlora_rope_workspace_bytes(ctypes.byref(cfg)) >= 128 * 4
    assert lib.qlora_rope_workspace_bytes(ctypes.byref(q.CRopeConfig(8, 2, 12, 8, 0, 1e-6, 1.0, 4))) == 0


def _rope_bwd(tokens=4, kv=2, tq=_t(), tk=_t(), qw=FAKE, kw=FAKE, go=_t(), gk=_t(), dq=_t(), dk=_t(), dqw=None, dkw=None, ws=None,
              ws_bytes=0):
    cfg = q.CRopeConfig(8, kv, 128, 64, 1, 1e-6, 1.0, tokens)
    return lib.qlora_rope_bwd(ctypes.byref(cfg), FREQ, FAKE, _ref(tq), _ref(tk), qw, kw, _ref(go), _ref(gk), _ref(dq), _ref(dk), dqw,
                              dkw, 0, ws, ws_bytes, None)


def test_rope_backward_refusals():
    assert _rope_bwd(tokens=0) == OK
    need = lib.qlora_rope_workspace_bytes(ctypes.byref(q.CRopeConfig(8, 2, 128, 64, 1, 1e-6, 1.0, 4)))
    for bad in (dict(tq=None), dict(tk=None), dict(go=None), dict(gk=None), dict(dq=None), dict(dk=None), dict(tq=_t(None)),
                dict(qw=None, dqw=FAKE), dict(kw=None, dkw=FAKE), dict(kv=0, dkw=FAKE)):
        assert _rope_bwd(**bad) == NULL, bad
    assert _rope_bwd(dq=_t(head=0)) == SHAPE and _rope_bwd(tk=_t(token=4)) == SHAPE
    for bad in (dict(go=_t(ODD)), dict(tq=_t(ODD)), dict(dqw=ODD), dict(dkw=ODD, ws=FAKE, ws_bytes=need), dict(qw=ODD),
                dict(dqw=FAKE, ws=ODD, ws_bytes=need)):
        assert _rope_bwd(**bad) == ALIGN, bad
    assert _rope_bwd(dqw=FAKE) == WS and _rope_bwd(dqw=FAKE, ws=FAKE, ws_bytes=need - 1) == WS


def test_rope_outputs_that_meet_are_refused():
    """One memory for two outputs, an output in the other's input, and one in its own input with other strides."""
    a, b, c, e = (_t(FAKE * i) for i in (1, 2, 3, 4))
    for bad in (dict(tq=a, tk=b, qo=c, ko=c), dict(tq=a, tk=b, qo=b, ko=c), dict(tq=a, tk=b, qo=c, ko=a), dict(tq=a, tk=b, qo=_t(token=8192), ko=b),
                dict(tq=a, tk=b, qo=a, ko=_t(2 * FAKE, head=256))):
        assert _rope(**bad) == SHAPE, bad
    for bad in (dict(go=a, gk=b, dq=c, dk=c), dict(go=a, gk=b, dq=b, dk=c), dict(go=a, gk=b, dq=_t(token=8192), dk=b),
                dict(go=a, gk=b, tq=c, tk=e, dq=e, dk=b), dict(go=a, gk=b, tq=c, tk=e, dq=a, dk=_t(4 * FAKE, head=256)),
                dict(go=a, gk=b, tq=c, tk=e, dq=a, dk=b, dqw=FAKE, dkw=FAKE, ws=FAKE, ws_bytes=1 << 20)):
        assert _rope_bwd(**bad) == SHAPE, bad


def test_values_read_over_keys_are_refused():
    assert _write(read=True) == SHAPE and _write(read=True, k=_t(), v=_t(token=8192)) == SHAPE
    assert _write(read=True, seqs=((0, 0, 0, 10),)) == OK


def _c4(codes=FAKE, absmax=FAKE + 2, token=4, head=4096, book=0):
    return q.CKv4(codes, absmax, token, head, book)


def _seqs(*s):
    flat = [v for x in s for v in x]
    return (ctypes.c_int64 * max(len(flat), 4))(*flat)


K4, V4 = _c4(), _c4(0x900000, 0xA00000)


def _write(seqs=((0, 4, 0, 10),), kv=2, d=128, tq=100, tk=1024, k=_t(), v=_t(), k4=K4, v4=V4, read=False):
    cfg = q.CAttnConfig(kv, kv, d, 1, 0, 0.1, tq, tk)
    n, s = len(seqs), _seqs(*seqs)
    if read:
        return lib.qlora_kv4_read(ctypes.byref(cfg), n, s, _ref(k4), _ref(v4), _ref(k), _ref(v), None)
    return lib.qlora_kv4_write(ctypes.byref(cfg), n, s, _ref(k), _ref(v), _ref(k4), _ref(v4), None)


@pytest.mark.parametrize("read", [False, True])
def test_cache_refusals(read):
    w = lambda **a: _write(read=read, **a)  # noqa: E731
    assert w(seqs=()) == OK and w(seqs=((0, 0, 0, 10), (5, 0, 3, 3))) == OK
    for bad in (dict(seqs=((0, 4, 0, 3),)), dict(seqs=((0, 4, 1020, 5),)), dict(seqs=((98, 4, 0, 9),)), dict(seqs=((0, 4, 0, 9), (3, 4, 20, 9))),
                dict(seqs=((0, -1, 0, 4),)), dict(kv=0), dict(d=4), dict(d=136), dict(d=12), dict(k4=_c4(token=3)), dict(k4=_c4(token=1 << 20)),
                dict(k4=_c4(head=-1)), dict(k4=_c4(head=(1 << 40) + 1)), dict(k4=_c4(book=3)), dict(v4=_c4(book=-1)),
                dict(v4=_c4(0x900000, 0xA00000, book=1))):
        assert w(**bad) == SHAPE, bad
    for bad in (dict(k=None), dict(v=None), dict(k4=None), dict(v4=None), dict(k=_t(None)), dict(k4=_c4(None)), dict(v4=_c4(0x900000, None))):
        assert w(**bad) == NULL, bad
    for bad in (dict(k=_t(ODD)), dict(k4=_c4(ODD)), dict(v4=_c4(0x900000, 0xA00001))):
        assert w(**bad) == ALIGN, bad
    big = 1 << 24    # of one sequence, nq * kv * blocks / 64 workgroups and more
    assert w(seqs=((0, big, 0, big),), kv=8, tq=big, tk=big, k=_t(), v=_t(), k4=_c4(head=1 << 30), v4=_c4(0x900000, 0xA00000, head=1 << 30)) == SHAPE


def test_writes_that_would_meet_are_refused():
    assert _write(seqs=((0, 4, 0, 10), (4, 4, 2, 10))) == SHAPE            # tokens 6..9 and 8..11
    assert _write(seqs=((0, 4, 0, 10), (4, 4, 0, 10))) == SHAPE            # the same
    assert _write(seqs=((0, 1, 20, 5), (4, 10, 10, 20))) == SHAPE          # in any order
    assert _write(v4=_c4(FAKE, 0xA00000)) == SHAPE and _write(v4=_c4(0x900000, FAKE + 2)) == SHAPE     # one memory for both
    for rows in (dict(token=4, head=0), dict(token=7, head=4), dict(token=4, head=4095)):
        assert _write(k4=_c4(**rows)) == SHAPE, rows                        # rows over one another
    assert _write(seqs=(), k4=_c4(token=8, head=4)) == OK


def _attend(seqs=((0, 1, 0, 1000),), heads=8, kv=2, d=128, tq=100, tk=1024, tq_=_t(), o=_t(), k4=K4, v4=V4, lse=None, ws=None, ws_bytes=0,
            scale=0.1, window=0):
    cfg = q.CAttnConfig(heads, kv, d, 1, window, scale, tq, tk)
    return lib.qlora_attn_kv4_fwd(ctypes.byref(cfg), len(seqs), _seqs(*seqs), _ref(tq_), _ref(k4), _ref(v4), _ref(o), lse, ws, ws_bytes, None)


def test_attention_refusals():
    assert _attend(seqs=()) == OK and _attend(seqs=((0, 0, 0, 10),)) == OK
    for bad in (dict(heads=7), dict(d=132), dict(scale=0.0), dict(scale=float("nan")), dict(window=-1), dict(seqs=((0, 1, 1000, 25),)),
                dict(seqs=((5, 1, 0, 9), (5, 1, 0, 9))), dict(k4=_c4(token=2)), dict(v4=_c4(0x900000, 0xA00000, book=2)), dict(o=_t(head=0))):
        assert _attend(**bad) == SHAPE, bad
    for bad in (dict(tq_=None), dict(o=None), dict(k4=None), dict(v4=_c4(None))):
        assert _attend(**bad) == NULL, bad
    for bad in (dict(lse=ODD), dict(ws=ODD), dict(tq_=_t(ODD)), dict(k4=_c4(ODD))):
        assert _attend(**bad) == ALIGN, bad
    assert _attend(seqs=((0, 100, 0, 1000),), heads=1 << 15, kv=1, tq=1 << 20) != OK
    cfg = q.CAttnConfig(8, 2, 128, 1, 0, 0.1, 100, 1024)
    need = lambda book, c=cfg: lib.qlora_attn_kv4_workspace_bytes(ctypes.byref(c), 1, _seqs((0, 1, 0, 1000)), book)  # noqa: E731
    assert need(0) > 0 and need(1) > 0 and need(3) == 0 and need(-1) == 0
    assert _attend() == WS and _attend(ws=FAKE, ws_bytes=need(0) - 256) == WS
    cfg.window = 100     # one range
    assert need(0) == 0


def test_attention_workspace_of_large_calls_stays_small():
    """Where the rows fill the GPU many times over, keys are not split: nothing to join, whatever their number."""
    cfg = q.CAttnConfig(64, 8, 128, 1, 0, 0.1, 1 << 20, 1 << 20)
    assert lib.qlora_attn_kv4_workspace_bytes(ctypes.byref(cfg), 1, _seqs((0, 1 << 20, 0, 1 << 20)), 0) == 0
    cfg = q.CAttnConfig(64, 8, 128, 1, 0, 0.1, 4096, 1 << 20)
    assert lib.qlora_attn_kv4_workspace_bytes(ctypes.byref(cfg), 64, _seqs(*[(64 * i, 64, 0, 1 << 20) for i in range(64)]), 0) < 1 << 31


def test_rope_frequencies():
    r = q.Rope(64, base=500.0)
    assert r.inv_freq == tuple(500.0 ** (-2.0 * i / 64) for i in range(32)) and r.rot == 64 and not r.interleaved and r.factor == 1.0
    s = q.Rope(64, base=500.0, stretch=4.0)
    assert all(math.isclose(a * 4, b) for a, b in zip(s.inv_freq, r.inv_freq))
    t = q.Rope(128, base=500000.0, stretch=8.0, trained=8192, factor=1.3, interleaved=True)
    plain = q.Rope(128, base=500000.0).inv_freq
    turns = [8192 * f / (2 * math.pi) for f in plain]
    for f, p, n in zip(t.inv_freq, plain, turns):
        assert math.isclose(f, p if n >= 4 else p / 8 if n <= 1 else p * ((n - 1) / 3 + (4 - n) / 3 / 8), rel_tol=1e-12)
    assert min(turns) < 1 < 4 < max(turns) and t.interleaved and t.factor == 1.3
    for bad in (dict(rot=64, inv_freq=[1.0] * 31), dict(rot=64, base=0.0), dict(rot=64, stretch=0.0), dict(rot=64, stretch=2.0, trained=9, low=4.0)):
        with pytest.raises(ValueError):
            q.Rope(**bad)
    for name in ("rot", "factor", "interleaved", "inv_freq"):      # calls keep what they marshalled
        with pytest.raises(AttributeError):
            setattr(r, name, 1)


def test_binding_sizes_workspaces():
    x, y = torch.empty(3, 4, 64), torch.empty(3, 2, 64)
    assert q.Rope(64).workspace_bytes(x, y) >= q.Rope(64).workspace_bytes(x) >= 512
    assert q.Rope(72).workspace_bytes(x, y) == 0      # refused: more features than the head has


def test_binding_refuses_before_the_library():
    x, y = torch.empty(3, 4, 64, dtype=torch.bfloat16), torch.empty(3, 2, 64, dtype=torch.bfloat16)
    r, pos = q.Rope(64), torch.zeros(3, dtype=torch.int64)
    for args in ((x, y, x[:2], y), (x, y[:2], x, y[:2]), (x, y, x, None), (x, None, x, y), (x, y[..., :32], x, y[..., :32]), (x[0], None, x[0], None),
                 (x, y, x, x)):
        with pytest.raises(ValueError):
            q.qlora_rope_fwd(r, pos, *args)
    with pytest.raises(ValueError):      # on the CPU
        q.qlora_rope_fwd(r, pos, x, y, x, y)
    with pytest.raises(ValueError):
        q.qlora_rope_bwd(r, pos, x, y, x, y, q_weight=x[0, 0])       # normed heads without their inputs
    with pytest.raises(ValueError):
        q.Kv4(torch.empty(4, 2, 4, 16, dtype=torch.uint8), torch.empty(4, 2, 4, dtype=torch.bfloat16), 128)
    with pytest.raises(ValueError):
        q.empty_kv4(4, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        q.Kv4(torch.empty(4, 2, 3, 16, dtype=torch.uint8), torch.empty(4, 2, 3, dtype=torch.bfloat16), 128)
    with pytest.raises(TypeError):
        q.Kv4(torch.empty(4, 2, 4, 16, dtype=torch.int8), torch.empty(4, 2, 4, dtype=torch.bfloat16), 128)
