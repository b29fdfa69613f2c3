"""A rotation's backward without tokens still has its weights' gradients checked. No kernel runs here."""
import ctypes

import pytest

q = pytest.importorskip("bit_nf4_quantised_amd")
FAKE, ODD = 0x100000, 0x100004


def _bwd(dqw, dkw, accumulate=0, kv=2):
    cfg, none = q.CRopeConfig(8, kv, 128, 64, 1, 1e-6, 1.0, 0), q.CAttnTensor(None, 4096, 128)
    r = ctypes.byref(none)
    return q.lib.qlora_rope_bwd(ctypes.byref(cfg), None, None, r, r, FAKE, FAKE, r, r, r, r, dqw, dkw, accumulate, None, 0, None)


def test_gradients_without_tokens_are_checked():
    assert _bwd(None, None) == q.NF4_OK and _bwd(FAKE, 2 * FAKE, accumulate=1) == q.NF4_OK
    assert _bwd(ODD, None) == q.NF4_ERR_ALIGN and _bwd(None, ODD) == q.NF4_ERR_ALIGN
    assert _bwd(FAKE, FAKE) == q.NF4_ERR_SHAPE and _bwd(None, FAKE, kv=0) == q.NF4_ERR_NULL
