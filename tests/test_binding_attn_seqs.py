"""AttnSeqs on the host: the configuration that a call gets is that of its own tensors and of the mask as it
stands, whatever calls came before or run beside it. No kernel runs here."""
import pytest
import torch

q = pytest.importorskip("bit_nf4_quantised_amd")


def _qk(tokens, heads, kv, d, keys=None):
    return (torch.empty(tokens, heads, d, dtype=torch.bfloat16),
            torch.empty(tokens if keys is None else keys, kv, d, dtype=torch.bfloat16))


def _read(cfg):
    c = cfg._obj
    return c.heads, c.kv_heads, c.d, c.causal, c.window, c.q_tokens, c.k_tokens


def test_changed_mask_is_taken():
    s = q.AttnSeqs([(0, 1, 0, 9000)])
    Q, K = _qk(1, 8, 2, 128, 9000)
    whole = s.workspace_bytes(Q, K)
    assert whole == q.AttnSeqs([(0, 1, 0, 9000)]).workspace_bytes(Q, K) > 0
    s.window = 100      # 100 keys are one range: no workspace
    assert s.workspace_bytes(Q, K) == q.AttnSeqs([(0, 1, 0, 9000)], window=100).workspace_bytes(Q, K) == 0
    assert _read(s._config(Q, K, None))[3:5] == (1, 100)
    s.causal, s.window = False, 0
    assert _read(s._config(Q, K, None))[3:5] == (0, 0)
    assert s.workspace_bytes(Q, K) == whole


def test_layers_of_different_sizes_share_one():
    s = q.AttnSeqs.packed([40, 24])
    sizes = [(64, 8, 2, 128), (64, 4, 4, 64), (64, 8, 2, 128), (64, 8, 8, 128)]
    held = [(z, s._config(*_qk(*z), None)) for z in sizes]
    for (tokens, heads, kv, d), cfg in held:      # earlier ones keep what they were made with
        assert _read(cfg) == (heads, kv, d, 1, 0, tokens, tokens)
