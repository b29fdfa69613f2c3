"""AttnSeqs on the host: the configuration that a call gets is that of its own tensors and of the mask as it
stands, whatever calls came before or run beside it. No kernel runs here."""
import threading

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


class _Interrupted(float):
    """A scale during whose comparison another call for other sizes runs to its end, as a thread may."""
    def __new__(cls, value, other):
        self = super().__new__(cls, value)
        self.other = other
        return self

    def __eq__(self, x):
        self.other()
        return float(self) == float(x)

    def __ne__(self, x):
        return not self == x

    __hash__ = float.__hash__


def test_a_call_in_between_changes_nothing():
    s = q.AttnSeqs.packed([40, 24])
    a, b = _qk(64, 8, 2, 128), _qk(64, 4, 4, 64)
    other = lambda: s._config(*b, 0.5)  # noqa: E731
    s._config(*a, _Interrupted(0.125, other))
    got = s._config(*a, _Interrupted(0.125, other))
    assert _read(got) == (8, 2, 128, 1, 0, 64, 64) and got._obj.scale == 0.125
    assert _read(s._config(*b, 0.5)) == (4, 4, 64, 1, 0, 64, 64)
    assert _read(s._config(*a, 0.125)) == (8, 2, 128, 1, 0, 64, 64)


def test_threads_share_one():
    s = q.AttnSeqs.packed([40, 24])
    wrong = []

    def work(heads, kv, d):
        Q, K = _qk(64, heads, kv, d)
        for _ in range(2000):
            got = _read(s._config(Q, K, None))
            if got != (heads, kv, d, 1, 0, 64, 64):
                wrong.append((heads, got))
                return
    threads = [threading.Thread(target=work, args=z) for z in ((8, 2, 128), (4, 4, 64), (16, 1, 80))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_entries_from_an_iterator_are_checked():
    good = q.AttnSeqs((i, 1, 10 * i, 10) for i in range(3))
    assert good.count == 3 and list(good._seqs) == [0, 1, 0, 10, 1, 1, 10, 10, 2, 1, 20, 10]
    with pytest.raises(ValueError):
        q.AttnSeqs((i, 1, 10 * i) for i in range(4))     # twelve values: no three sequences
