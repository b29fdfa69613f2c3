"""A call that is given a stream takes its workspace from that stream's memory pool: a block of the current
stream's pool would go back there when the call returns, while the kernels on the given stream still use it.
No kernel runs here: the library's launches and torch's streams are stand-ins that record."""
import contextlib

import pytest
import torch

q = pytest.importorskip("bit_nf4_quantised_amd")


class _Stream:
    cuda_stream = 0x5EED


class _Library:
    """The built library with every call that would launch replaced by one that records its name and arguments."""
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if "bytes" in name or name == "nf4_status_string":
            return getattr(q_lib, name)
        return lambda *a: self.calls.append((name, a)) or 0


q_lib = q.lib


@pytest.fixture
def seen(monkeypatch):
    """Names of the streams whose pool torch.empty was called for, and the recording library."""
    pools, at = [], ["current"]
    empty = torch.empty

    @contextlib.contextmanager
    def on(stream):
        at.append(stream)
        yield
        at.pop()

    def record(*size, **kw):
        pools.append(at[-1])
        return empty(*size, **kw)
    lib = _Library()
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(q, "lib", lib)
    monkeypatch.setattr(torch, "empty", record)
    return pools, lib


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


M, N, K, R = 300, 64, 128, 16


def _weight():
    return q.NF4Weight(torch.zeros(N * K // 2, dtype=torch.uint8), torch.zeros(N * K // 64, dtype=torch.uint8),
                       torch.zeros(1), N, K)


def _calls():
    w, x, y, A, B, u = _weight(), _bf(M, K), _bf(M, N), _bf(R, K), _bf(N, R), torch.zeros(M, R)
    dx, dA, dB = _bf(M, K), torch.zeros(R, K), torch.zeros(N, R)
    x8 = q.Act8(torch.zeros(M, K, dtype=torch.int8), _bf(M, K // 64), M, K)
    a, seqs = [_bf(M, 4, 64) for _ in range(8)], q.AttnSeqs.packed([200, 100])
    lse, one, long = torch.zeros(4, M), q.AttnSeqs([(0, 1, 0, 9000)]), [_bf(1, 8, 128), _bf(9000, 2, 128)]
    return {
        "qlora_linear_fwd": lambda s: q.qlora_linear_fwd(w, x, A, B, 1.0, y, u, stream=s),
        "qlora_linear_fwd_group": lambda s: q.qlora_linear_fwd_group([w], x, [A], [B], 1.0, [y], stream=s),
        "qlora_linear_fwd_recompute": lambda s: q.qlora_linear_fwd_recompute(w, x, A, B, 1.0, u, y, stream=s),
        "qlora_linear_fwd_recompute_group": lambda s: q.qlora_linear_fwd_recompute_group([w], x, [A], [B], 1.0, [u], [y],
                                                                                        stream=s),
        "qlora_linear_bwd": lambda s: q.qlora_linear_bwd(w, x, y, A, B, 1.0, u, dx, dA, dB, stream=s),
        "qlora_linear_bwd_group": lambda s: q.qlora_linear_bwd_group([w], x, [y], [A], [B], 1.0, [u], [dx], [dA], [dB],
                                                                    stream=s),
        "qlora_linear_bwd_act8": lambda s: q.qlora_linear_bwd_act8([w], x8, [y], [A], [B], 1.0, [u], [dx], [dA], [dB],
                                                                  stream=s),
        "qlora_rmsnorm_bwd": lambda s: q.qlora_rmsnorm_bwd(x, x, _bf(K), torch.zeros(M), dx, dw=torch.zeros(K), stream=s),
        "qlora_attn_fwd": lambda s: q.qlora_attn_fwd(one, long[0], long[1], long[1], long[0], stream=s),
        "qlora_attn_bwd": lambda s: q.qlora_attn_bwd(seqs, *a[:4], lse, *a[4:], stream=s),
        "nf4_double_quant": lambda s: q.quantize_weight(torch.zeros(N, K), stream=s),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_workspace_is_of_the_stream_that_the_call_is_given(seen, name):
    pools, lib = seen
    call, stream = _calls()[name], _Stream()
    pools.clear()
    call(stream)
    assert pools and all(p is stream for p in pools), (name, pools)
    launched, args = lib.calls[-1]
    assert launched == name and args[-1] == stream.cuda_stream


def test_any_object_with_a_handle_is_a_stream(seen, monkeypatch):
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: made.append((handle, device)) or "external",
                        raising=False)

    class Handle:
        cuda_stream = 77
    pools, lib = seen
    call = _calls()["qlora_attn_bwd"]
    pools.clear()
    call(Handle())
    assert made == [(77, torch.device("cpu"))] and pools == ["external"] and lib.calls[-1][1][-1] == 77
