"""Attention calls whose sequences' workgroups do not fit a launch are refused, those that do are accepted. No kernel
runs here."""
import ctypes

import pytest

q = pytest.importorskip("bit_nf4_quantised_amd")
FAKE = 0x100000


def _accepted(heads, kv, nq, nk):
    """Whether the backward takes one sequence of these sizes (its workspace is never empty then)."""
    cfg = q.CAttnConfig(heads, kv, 8, 1, 0, 0.5, nq, nk)
    return q.lib.qlora_attn_workspace_bytes(ctypes.byref(cfg), 1, (ctypes.c_int64 * 4)(0, nq, 0, nk), 1) > 0


def _forward(heads, kv, nq, nk):
    cfg = q.CAttnConfig(heads, kv, 8, 1, 0, 0.5, nq, nk)
    t = q.CAttnTensor(FAKE, 8 * 65536, 8)
    r = ctypes.byref(t)
    return q.lib.qlora_attn_fwd(ctypes.byref(cfg), 1, (ctypes.c_int64 * 4)(0, nq, 0, nk), r, r, r, r, None, None, 0, None)


def test_tiles_of_queries_over_heads():
    assert _accepted(4096, 1, 4095 * 128, 64)
    assert not _accepted(4096, 1, 4095 * 128 + 1, 64)
    assert _forward(4096, 1, 4095 * 128 + 1, 64) == q.NF4_ERR_SHAPE
    assert _accepted(65535, 1, 256 * 128, 64) and not _accepted(65535, 1, 257 * 128, 64)


def test_tiles_of_keys_over_key_heads_in_the_backward():
    assert _accepted(4096, 4096, 1, 4095 * 128)
    assert not _accepted(4096, 4096, 1, 4095 * 128 + 1)
    assert _accepted(4096, 1, 1, 4095 * 128 + 1)        # one key head: few workgroups


def test_parts_never_ask_for_more_than_a_launch_holds():
    """A prime number of heads splits into one part or all; by time alone all of them, 2e7 workgroups, would be chosen
    here, where a window leaves most of 300 key tiles without work. The workspace holds 2 floats a query and head and,
    for every key tile and part, 2 * 128 rows of 64 floats."""
    heads, nq, nk = 65521, 6400, 300 * 128
    cfg = q.CAttnConfig(heads, 1, 8, 1, 6400, 0.5, nq, nk)
    nbytes = q.lib.qlora_attn_workspace_bytes(ctypes.byref(cfg), 1, (ctypes.c_int64 * 4)(0, nq, 0, nk), 1)
    rows = 2 * 4 * heads * nq
    assert rows <= nbytes < rows + 300 * 2 * 128 * 64 * 4
