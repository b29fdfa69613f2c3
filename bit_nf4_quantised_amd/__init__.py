"""NF4-quantised QLoRA linear layer on AMD Instinct MI355X (gfx950): Python binding.

A thin ctypes layer over ``libqlora_nf4.so`` (the C ABI in ``include/qlora_nf4.h``). Every function
only checks tensor placement and marshals device pointers, sizes and the current HIP stream; all
computation runs in the library's HIP kernels. PyTorch supplies device memory and streams.

The library must have been built (``python bit_nf4_quantised_amd/build.py``); importing this
package without it raises ImportError, and there is no CPU fallback.

Operations ("QLoRA, explained", pofe.ai): blockwise absmax NF4 quantisation with two indices per
byte, double quantisation of the scales to E4M3, two-level dequantisation to bf16, and the adapted
linear's forward y = x W~^T + s x A^T B^T and backward (dX, dA, dB; no gradient for W), the
adapter merged into the base for serving, and the adapter update of a training step (global
gradient-norm clipping, then AdamW over A and B). Around the linears: root-mean-square norm with the
residual's addition, rotary positions with norms of the query and key heads, attention over packed
sequences or a key/value cache, all with their backward passes, 8-bit activation checkpoints that the
linears' backward reads, and a key/value cache in 4 bits with the attention over it.
"""
from __future__ import annotations

import ctypes
import math
import os
from array import array
from contextlib import nullcontext
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# NF4_LIBRARY names another build of the same library (the host-sanitised one the CPU tests use)
LIB_PATH = os.environ.get("NF4_LIBRARY") or os.path.join(_HERE, "libqlora_nf4.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first with "
        "`python bit_nf4_quantised_amd/build.py` (hipcc, gfx950). There is no CPU fallback.")

lib = ctypes.CDLL(LIB_PATH)

NF4_OK, NF4_ERR_NULL, NF4_ERR_SHAPE, NF4_ERR_ALIGN, NF4_ERR_RANK, NF4_ERR_WORKSPACE, NF4_ERR_HIP = range(7)


class CNF4Weight(ctypes.Structure):
    """Mirror of ``nf4_weight`` in include/qlora_nf4.h."""
    _fields_ = [("packed", ctypes.c_void_p), ("scale_q", ctypes.c_void_p),
                ("scale_c2", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("absmax", ctypes.c_void_p), ("codebook", ctypes.c_int32)]


class CAdamWConfig(ctypes.Structure):
    """Mirror of ``qlora_adamw_config`` in include/qlora_nf4.h."""
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("max_grad_norm", ctypes.c_float)]


class CAct8(ctypes.Structure):
    """Mirror of ``qlora_act8`` in include/qlora_nf4.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("absmax", ctypes.c_void_p)]


class CAttnConfig(ctypes.Structure):
    """Mirror of ``qlora_attn_config`` in include/qlora_nf4.h."""
    _fields_ = [("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("d", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("window", ctypes.c_int64), ("scale", ctypes.c_float),
                ("q_tokens", ctypes.c_int64), ("k_tokens", ctypes.c_int64)]


class CAttnTensor(ctypes.Structure):
    """Mirror of ``qlora_attn_tensor`` in include/qlora_nf4.h."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class CRopeConfig(ctypes.Structure):
    """Mirror of ``qlora_rope_config`` in include/qlora_nf4.h."""
    _fields_ = [("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("d", ctypes.c_int32),
                ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("factor", ctypes.c_float), ("tokens", ctypes.c_int64)]


class CKv4(ctypes.Structure):
    """Mirror of ``qlora_kv4`` in include/qlora_nf4.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("absmax", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("codebook", ctypes.c_int32)]


_p, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_W = ctypes.POINTER(CNF4Weight)
_SIGS = {
    "nf4_quantize": (ctypes.c_int, [_p, _i64, _p, _p, _p]),
    "nf4_quantize_bf16": (ctypes.c_int, [_p, _i64, _p, _p, _p]),
    "nf4_double_quant": (ctypes.c_int, [_p, _i64, _p, _p, _p]),
    "nf4_double_quant_many": (ctypes.c_int, [_i64, _p, _p, _p, _p, _p]),
    "nf4_dequant": (ctypes.c_int, [_W, _p, _p]),
    "qlora_linear_fwd": (ctypes.c_int, [_W, _p, _i64, _p, _p, _i32, _f32, _p, _p, _p, _sz, _p]),
    "qlora_linear_fwd_noalloc": (ctypes.c_int, [_W, _p, _i64, _p, _p, _i32, _f32, _p, _p, _p]),
    "qlora_linear_fwd_group": (ctypes.c_int, [_i32, _p, _p, _i64, _p, _p, _i32, _f32, _p, _p, _p, _sz, _p]),
    "qlora_linear_fwd_recompute_group": (ctypes.c_int, [_i32, _p, _p, _i64, _p, _p, _i32, _f32, _p, _p, _p, _sz,
                                                        _p]),
    "qlora_linear_bwd": (ctypes.c_int, [_W, _p, _p, _i64, _p, _p, _i32, _f32, _p, _p, _p, _p,
                                        ctypes.c_int, _p, _sz, _p]),
    "qlora_linear_fwd_recompute": (ctypes.c_int, [_W, _p, _i64, _p, _p, _i32, _f32, _p, _p, _p, _sz,
                                                  _p]),
    "qlora_merge": (ctypes.c_int, [_W, _p, _p, _i32, _f32, _p, _p]),
    "q4_codebook_values": (ctypes.c_int, [_i32, ctypes.POINTER(ctypes.c_float)]),
    "q4_quantize": (ctypes.c_int, [_p, _i64, _i32, _i32, _p, _p, _p]),
    "q4_dequant": (ctypes.c_int, [_p, _i64, _i32, _i32, _p, _p, _p, _p, _p]),
    "qlora_adamw_plan_create": (ctypes.c_int, [_i64, _p, _p, _p, _p, _p, _p,
                                               ctypes.POINTER(ctypes.c_void_p)]),
    "qlora_adamw_plan_step": (ctypes.c_int, [_p, ctypes.POINTER(CAdamWConfig), _i64, _p, _p]),
    "qlora_adamw_plan_destroy": (ctypes.c_int, [_p]),
    "qlora_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32]),
    "qlora_workspace_bytes_group": (_sz, [_i32, _p, _i64, _i64, _i32]),
    "qlora_linear_bwd_group": (ctypes.c_int, [_i32, _p, _p, _p, _i64, _p, _p, _i32, _f32, _p, _p, _p, _p,
                                              ctypes.c_int, _p, _sz, _p]),
    "qlora_act8_pack": (ctypes.c_int, [_p, _i64, _p, _p, _p]),
    "qlora_act8_unpack": (ctypes.c_int, [_p, _p, _i64, _p, _p]),
    "qlora_linear_bwd_act8": (ctypes.c_int, [_i32, _p, _p, _p, _i64, _p, _p, _i32, _f32, _p, _p, _p, _p,
                                             ctypes.c_int, _p, _sz, _p]),
    "qlora_workspace_bytes_act8": (_sz, [_i32, _p, _i64, _i64, _i32]),
    "qlora_rmsnorm_fwd": (ctypes.c_int, [_p, _p, _p, _i64, _i64, _f32, _p, _p, _p, _p, _p]),
    "qlora_rmsnorm_bwd": (ctypes.c_int, [_p, _p, _p, _p, _p, _i64, _i64, _p, _p, ctypes.c_int, _p, _sz, _p]),
    "qlora_rmsnorm_workspace_bytes": (_sz, [_i64, _i64]),
    "qlora_attn_fwd": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "qlora_attn_bwd": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "qlora_attn_workspace_bytes": (_sz, [_p, _i64, _p, ctypes.c_int]),
    "qlora_rope_fwd": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p]),
    "qlora_rope_bwd": (ctypes.c_int, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, ctypes.c_int, _p, _sz, _p]),
    "qlora_rope_workspace_bytes": (_sz, [_p]),
    "qlora_kv4_write": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _p, _p]),
    "qlora_kv4_read": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _p, _p]),
    "qlora_attn_kv4_fwd": (ctypes.c_int, [_p, _i64, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "qlora_attn_kv4_workspace_bytes": (_sz, [_p, _i64, _p, _i32]),
    "nf4_storage_bytes": (_i64, [_i64]),
    "nf4_codebook": (None, [ctypes.POINTER(ctypes.c_float)]),
    "nf4_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


class NF4Error(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {lib.nf4_status_string(status).decode()} (status {status})")


def _check(status: int, call: str) -> None:
    if status != NF4_OK:
        raise NF4Error(status, call)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


# the current stream's handle without building a torch.cuda.Stream (0.2 us against 2.9 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _stream_on(stream, gpu, *tensors):
    """_stream, for a call with tensors of device `gpu` and these (None: not there): all must live on the current device, on
    whose streams the kernels run. A kernel that is given another GPU's memory faults where the two are not peers."""
    current = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != current:
            gpu = t.get_device()
    if gpu != current:
        raise ValueError(f"a tensor lives on GPU {gpu} and the current device is GPU {current}")
    if stream is None and _raw_stream is not None:
        return _raw_stream(current)
    return _stream(stream)


def _pool_of(stream, device):
    """The context in which torch allocates from the memory pool of the stream that a call is given. A block of
    another pool may be handed out again, or still be read, by that other stream's work while the call's kernels
    use it."""
    if stream is None:
        return nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    return torch.cuda.stream(stream)


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace for one call on `stream` (None: the current one), to be dropped when the call returns."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with _pool_of(stream, device):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _dtype(t, *allowed):
    if t is not None and t.dtype not in allowed:
        raise TypeError(f"dtype {t.dtype} not in {allowed}")


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_F32 = (torch.float32,)


def _dptr(t, dtypes):
    """_dtype and _ptr in one."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _dtype(t, *dtypes)
    return _ptr(t)


def _mptrs(kind, tensors, dtypes, shapes):
    """_dptr of every tensor, which must have the shape at its place, as an array of the ctypes type."""
    out = kind()
    for i, t in enumerate(tensors):
        if t.shape != shapes[i]:
            raise ValueError("shape mismatch")
        if t.dtype not in dtypes or not t.is_cuda or not t.is_contiguous():
            _dtype(t, *dtypes)
            _ptr(t)
        out[i] = t.data_ptr()
    return out


@dataclass
class NF4Weight:
    """A quantised N x K weight in device tensors: double-quantised scales (scale_q, scale_c2) or,
    without double quantisation, the fp32 absmax (scale_q and scale_c2 None). codebook: the values
    the indices select (0 NF4, 1 FP4, 2 INT4; see Q4_CODEBOOKS)."""
    packed: torch.Tensor           # uint8 [N*K/2]
    scale_q: torch.Tensor | None   # uint8 [N*K/64]
    scale_c2: torch.Tensor | None  # float32 [ceil(N*K/16384)]
    N: int
    K: int
    absmax: torch.Tensor | None = None   # float32 [N*K/64]
    codebook: int = 0

    def c_struct(self) -> CNF4Weight:
        return CNF4Weight(_ptr(self.packed), _ptr(self.scale_q), _ptr(self.scale_c2), self.N, self.K,
                          _ptr(self.absmax), _book(self.codebook))


# ------------------------------------------------------------------------- the five calls
def nf4_quantize(w, packed, absmax, stream=None) -> None:
    _dtype(w, torch.float32); _dtype(packed, torch.uint8); _dtype(absmax, torch.float32)
    n = w.numel()
    if packed.numel() * 2 != n or absmax.numel() * 64 != n:
        raise ValueError("output sizes must be numel/2 and numel/64")
    _check(lib.nf4_quantize(_ptr(w), n, _ptr(packed), _ptr(absmax), _stream(stream)), "nf4_quantize")


def nf4_quantize_bf16(w, packed, absmax, stream=None) -> None:
    """nf4_quantize of a bf16 array (a merged weight quantised again)."""
    _dtype(w, *_BF16); _dtype(packed, torch.uint8); _dtype(absmax, torch.float32)
    n = w.numel()
    if packed.numel() * 2 != n or absmax.numel() * 64 != n:
        raise ValueError("output sizes must be numel/2 and numel/64")
    _check(lib.nf4_quantize_bf16(_ptr(w), n, _ptr(packed), _ptr(absmax), _stream(stream)),
           "nf4_quantize_bf16")


def nf4_double_quant(absmax, scale_q, scale_c2, stream=None) -> None:
    _dtype(absmax, torch.float32); _dtype(scale_q, torch.uint8); _dtype(scale_c2, torch.float32)
    nb = absmax.numel()
    if scale_q.numel() != nb or scale_c2.numel() != (nb + 255) // 256:
        raise ValueError("output sizes must be nblocks and ceil(nblocks/256)")
    _check(lib.nf4_double_quant(_ptr(absmax), nb, _ptr(scale_q), _ptr(scale_c2), _stream(stream)),
           "nf4_double_quant")


class DoubleQuantMany:
    """nf4_double_quant_many over fixed lists of tensors, with the argument arrays marshalled once
    (a model's weights at load time); calling it enqueues the launches on the stream."""

    def __init__(self, absmax: list, scale_q: list, scale_c2: list):
        n = len(absmax)
        if len(scale_q) != n or len(scale_c2) != n:
            raise ValueError("one scale_q and scale_c2 per absmax")
        for a, c, g in zip(absmax, scale_q, scale_c2):
            _dtype(a, torch.float32); _dtype(c, torch.uint8); _dtype(g, torch.float32)
            if c.numel() != a.numel() or g.numel() != (a.numel() + 255) // 256:
                raise ValueError("output sizes must be nblocks and ceil(nblocks/256)")
        P = ctypes.c_void_p * max(n, 1)
        self._keep = (list(absmax), list(scale_q), list(scale_c2))   # the tensors stay alive
        self._args = (n, P(*[_ptr(a) for a in absmax]), (ctypes.c_int64 * max(n, 1))(*[a.numel() for a in absmax]),
                      P(*[_ptr(c) for c in scale_q]), P(*[_ptr(g) for g in scale_c2]))

    def __call__(self, stream=None) -> None:
        _check(lib.nf4_double_quant_many(*self._args, _stream(stream)), "nf4_double_quant_many")


def nf4_double_quant_many(absmax: list, scale_q: list, scale_c2: list, stream=None) -> None:
    """nf4_double_quant over several weights' scales (up to 64 per kernel launch)."""
    DoubleQuantMany(absmax, scale_q, scale_c2)(stream)


def nf4_dequant(weight: NF4Weight, out, stream=None) -> None:
    _dtype(out, *_BF16)
    if out.numel() != weight.N * weight.K:
        raise ValueError("out must hold N*K values")
    cw = weight.c_struct()
    _check(lib.nf4_dequant(ctypes.byref(cw), _ptr(out), _stream(stream)), "nf4_dequant")


def qlora_linear_fwd(weight: NF4Weight, x, A, B, scale: float, y, u_out=None, ws=None,
                     stream=None) -> None:
    for t in (x, A, B, y):
        _dtype(t, *_BF16)
    _dtype(u_out, torch.float32)
    M = x.shape[0]
    r = A.shape[0]
    if x.shape != (M, weight.K) or A.shape != (r, weight.K) or B.shape != (weight.N, r) \
            or y.shape != (M, weight.N) or (u_out is not None and u_out.numel() != M * r):
        raise ValueError("shape mismatch")
    if ws is None:
        ws = _scratch(max(qlora_workspace_bytes(M, weight.N, weight.K, r), 256), x.device, stream)
    cw = weight.c_struct()
    _check(lib.qlora_linear_fwd(ctypes.byref(cw), _ptr(x), M, _ptr(A), _ptr(B), r, scale, _ptr(y),
                                _ptr(u_out), _ptr(ws), ws.numel() * ws.element_size(),
                                _stream(stream)), "qlora_linear_fwd")


def qlora_workspace_bytes_group(M: int, N: list, K: int, r: int) -> int:
    n = (ctypes.c_int64 * max(len(N), 1))(*[int(v) for v in N])
    return int(lib.qlora_workspace_bytes_group(len(N), n, M, K, r))


def workspace_group(M: int, N: list, K: int, r: int, device="cuda") -> torch.Tensor:
    """A device workspace large enough for qlora_linear_fwd_group over weights of N rows."""
    nbytes = max(qlora_workspace_bytes_group(M, N, K, r), 256)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def qlora_linear_fwd_group(weights: list, x, As: list, Bs: list, scale: float, ys: list, us=None, ws=None,
                           stream=None) -> None:
    """Forward of several linears that share x (e.g. q/k/v or gate/up): ys[i] = x W~_i^T +
    s (x A_i^T) B_i^T, as one fused launch where the shapes allow (see qlora_linear_fwd_group in
    include/qlora_nf4.h); us[i] (optional) receives u_i = x A_i^T."""
    n = len(weights)
    if not (len(As) == len(Bs) == len(ys) == n) or (us is not None and len(us) != n):
        raise ValueError("one A, B and y (and u) per weight")
    _dtype(x, *_BF16)
    M = x.shape[0]
    r = As[0].shape[0]
    for w, A, B, y in zip(weights, As, Bs, ys):
        for t in (A, B, y):
            _dtype(t, *_BF16)
        if x.shape != (M, w.K) or A.shape != (r, w.K) or B.shape != (w.N, r) or y.shape != (M, w.N):
            raise ValueError("shape mismatch")
    if us is not None:
        for u in us:
            _dtype(u, torch.float32)
            if u is not None and u.numel() != M * r:
                raise ValueError("shape mismatch")
    if ws is None:
        nbytes = qlora_workspace_bytes_group(M, [w.N for w in weights], weights[0].K, r)
        ws = _scratch(max(nbytes, 256), x.device, stream)
    cws = [w.c_struct() for w in weights]
    P = ctypes.c_void_p
    wp = (P * n)(*[ctypes.addressof(c) for c in cws])
    ap = (P * n)(*[_ptr(A) for A in As])
    bp = (P * n)(*[_ptr(B) for B in Bs])
    yp = (P * n)(*[_ptr(y) for y in ys])
    up = (P * n)(*[_ptr(u) for u in us]) if us is not None else None
    _check(lib.qlora_linear_fwd_group(n, wp, _ptr(x), M, ap, bp, r, scale, yp, up, _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)), "qlora_linear_fwd_group")


def qlora_linear_fwd_recompute_group(weights: list, x, As: list, Bs: list, scale: float, us: list, ys: list,
                                     ws=None, stream=None) -> None:
    """qlora_linear_fwd_group with every u_i = x A_i^T known: the fused GEMMs only."""
    n = len(weights)
    if not (len(As) == len(Bs) == len(ys) == len(us) == n):
        raise ValueError("one A, B, u and y per weight")
    _dtype(x, *_BF16)
    M = x.shape[0]
    r = As[0].shape[0]
    for w, A, B, y, u in zip(weights, As, Bs, ys, us):
        for t in (A, B, y):
            _dtype(t, *_BF16)
        _dtype(u, torch.float32)
        if x.shape != (M, w.K) or A.shape != (r, w.K) or B.shape != (w.N, r) or y.shape != (M, w.N) \
                or u.numel() != M * r:
            raise ValueError("shape mismatch")
    if ws is None:
        nbytes = qlora_workspace_bytes_group(M, [w.N for w in weights], weights[0].K, r)
        ws = _scratch(max(nbytes, 256), x.device, stream)
    cws = [w.c_struct() for w in weights]
    P = ctypes.c_void_p
    wp = (P * n)(*[ctypes.addressof(c) for c in cws])
    _check(lib.qlora_linear_fwd_recompute_group(n, wp, _ptr(x), M, (P * n)(*[_ptr(A) for A in As]),
                                                (P * n)(*[_ptr(B) for B in Bs]), r, scale,
                                                (P * n)(*[_ptr(u) for u in us]), (P * n)(*[_ptr(y) for y in ys]),
                                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "qlora_linear_fwd_recompute_group")


def qlora_linear_bwd_group(weights: list, x, dys: list, As: list, Bs: list, scale: float, us: list, dxs,
                           dAs: list, dBs: list, accumulate: bool = False, ws=None, stream=None) -> None:
    """Backward of several linears that share x: for each i as qlora_linear_bwd (dxs[i], dAs[i],
    dBs[i]), the dX GEMMs as one launch where the shapes allow; dxs None skips the input gradients."""
    n = len(weights)
    if not (len(dys) == len(As) == len(Bs) == len(us) == len(dAs) == len(dBs) == n) or \
            (dxs is not None and len(dxs) != n):
        raise ValueError("one dY, A, B, u, dA and dB (and dX) per weight")
    _dtype(x, *_BF16)
    M = x.shape[0]
    r = As[0].shape[0]
    for i, w in enumerate(weights):
        for t in (dys[i], As[i], Bs[i]) + ((dxs[i],) if dxs is not None else ()):
            _dtype(t, *_BF16)
        for t in (us[i], dAs[i], dBs[i]):
            _dtype(t, torch.float32)
        if x.shape != (M, w.K) or dys[i].shape != (M, w.N) or As[i].shape != (r, w.K) or Bs[i].shape != (w.N, r) \
                or us[i].numel() != M * r or dAs[i].shape != (r, w.K) or dBs[i].shape != (w.N, r) \
                or (dxs is not None and dxs[i].shape != (M, w.K)):
            raise ValueError("shape mismatch")
    if ws is None:
        nbytes = qlora_workspace_bytes_group(M, [w.N for w in weights], weights[0].K, r)
        ws = _scratch(max(nbytes, 256), x.device, stream)
    cws = [w.c_struct() for w in weights]
    P = ctypes.c_void_p
    arr = lambda ts: (P * n)(*[_ptr(t) for t in ts])  # noqa: E731
    _check(lib.qlora_linear_bwd_group(n, (P * n)(*[ctypes.addressof(c) for c in cws]), _ptr(x), arr(dys), M,
                                      arr(As), arr(Bs), r, scale, arr(us), arr(dxs) if dxs is not None else None,
                                      arr(dAs), arr(dBs), int(bool(accumulate)), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)), "qlora_linear_bwd_group")


def qlora_linear_fwd_noalloc(weight: NF4Weight, x, A, B, scale: float, y, u_out=None,
                             stream=None) -> None:
    """qlora_linear_fwd with the library's own per-GPU workspace (no allocation anywhere)."""
    for t in (x, A, B, y):
        _dtype(t, *_BF16)
    _dtype(u_out, torch.float32)
    M = x.shape[0]
    r = A.shape[0]
    if x.shape != (M, weight.K) or A.shape != (r, weight.K) or B.shape != (weight.N, r) \
            or y.shape != (M, weight.N) or (u_out is not None and u_out.numel() != M * r):
        raise ValueError("shape mismatch")
    cw = weight.c_struct()
    _check(lib.qlora_linear_fwd_noalloc(ctypes.byref(cw), _ptr(x), M, _ptr(A), _ptr(B), r, scale, _ptr(y),
                                        _ptr(u_out), _stream(stream)), "qlora_linear_fwd_noalloc")


def qlora_merge(weight: NF4Weight, A, B, scale: float, out, stream=None) -> None:
    """Adapter merged into the dequantised base: out = bf16(W~ + s B A), [N x K]."""
    for t in (A, B, out):
        _dtype(t, *_BF16)
    r = A.shape[0]
    if A.shape != (r, weight.K) or B.shape != (weight.N, r) or out.numel() != weight.N * weight.K:
        raise ValueError("shape mismatch")
    cw = weight.c_struct()
    _check(lib.qlora_merge(ctypes.byref(cw), _ptr(A), _ptr(B), r, scale, _ptr(out), _stream(stream)),
           "qlora_merge")


def qlora_linear_fwd_recompute(weight: NF4Weight, x, A, B, scale: float, u, y, ws=None,
                               stream=None) -> None:
    """Forward with a known u = x A^T (gradient-checkpointing recompute): the forward's GEMM
    without the pass that forms u."""
    for t in (x, A, B, y):
        _dtype(t, *_BF16)
    _dtype(u, torch.float32)
    M = x.shape[0]
    r = A.shape[0]
    if x.shape != (M, weight.K) or A.shape != (r, weight.K) or B.shape != (weight.N, r) \
            or y.shape != (M, weight.N) or u.numel() != M * r:
        raise ValueError("shape mismatch")
    if ws is None:   # with the forward's workspace the launches (and y) are the forward's own
        ws = _scratch(max(qlora_workspace_bytes(M, weight.N, weight.K, r), 256), x.device, stream)
    cw = weight.c_struct()
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.qlora_linear_fwd_recompute(ctypes.byref(cw), _ptr(x), M, _ptr(A), _ptr(B), r, scale,
                                          _ptr(u), _ptr(y), _ptr(ws), nbytes, _stream(stream)),
           "qlora_linear_fwd_recompute")


def qlora_linear_bwd(weight: NF4Weight, x, dy, A, B, scale: float, u, dx, dA, dB,
                     accumulate: bool = False, ws=None, stream=None) -> None:
    for t in (x, dy, A, B, dx):
        _dtype(t, *_BF16)
    for t in (u, dA, dB):
        _dtype(t, torch.float32)
    M = x.shape[0]
    r = A.shape[0]
    if x.shape != (M, weight.K) or dy.shape != (M, weight.N) or A.shape != (r, weight.K) \
            or B.shape != (weight.N, r) or u.numel() != M * r or dA.shape != (r, weight.K) \
            or dB.shape != (weight.N, r) or (dx is not None and dx.shape != (M, weight.K)):
        raise ValueError("shape mismatch")
    if ws is None:
        ws = _scratch(max(qlora_workspace_bytes(M, weight.N, weight.K, r), 256), x.device, stream)
    cw = weight.c_struct()
    _check(lib.qlora_linear_bwd(ctypes.byref(cw), _ptr(x), _ptr(dy), M, _ptr(A), _ptr(B), r, scale,
                                _ptr(u), _ptr(dx), _ptr(dA), _ptr(dB), int(bool(accumulate)),
                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "qlora_linear_bwd")


# ------------------------------------------------------------------------- 8-bit activation checkpoints
@dataclass
class Act8:
    """An M x K activation in 8 bits: int8 codes and the bf16 absmax of every block of 64 along K; a
    code stands for code * absmax / 127 (format in include/qlora_nf4.h)."""
    codes: torch.Tensor    # int8 [M, K]
    absmax: torch.Tensor   # bf16 [M, K/64]
    M: int
    K: int

    def c_struct(self) -> CAct8:
        n = self.M * self.K
        if self.codes.numel() != n or self.absmax.numel() * 64 != n:
            raise ValueError("codes must hold M*K values and absmax M*K/64")
        return CAct8(_dptr(self.codes, (torch.int8,)), _dptr(self.absmax, _BF16))


def empty_act8(M: int, K: int, device="cuda") -> Act8:
    return Act8(torch.empty(M, K, dtype=torch.int8, device=device),
                torch.empty(M, K // 64, dtype=torch.bfloat16, device=device), M, K)


def qlora_act8_pack(x, act8: Act8, stream=None) -> None:
    """The 8-bit checkpoint of a bf16 activation."""
    _dtype(x, *_BF16)
    if x.numel() != act8.M * act8.K:
        raise ValueError("x must hold M*K values")
    c = act8.c_struct()
    _check(lib.qlora_act8_pack(_ptr(x), x.numel(), c.codes, c.absmax, _stream(stream)), "qlora_act8_pack")


def qlora_act8_unpack(act8: Act8, out, stream=None) -> None:
    """The values of an 8-bit checkpoint, in bf16."""
    _dtype(out, *_BF16)
    if out.numel() != act8.M * act8.K:
        raise ValueError("out must hold M*K values")
    c = act8.c_struct()
    _check(lib.qlora_act8_unpack(c.codes, c.absmax, out.numel(), _ptr(out), _stream(stream)), "qlora_act8_unpack")


def qlora_workspace_bytes_act8(M: int, N: list, K: int, r: int) -> int:
    n = (ctypes.c_int64 * max(len(N), 1))(*[int(v) for v in N])
    return int(lib.qlora_workspace_bytes_act8(len(N), n, M, K, r))


def workspace_act8(M: int, N: list, K: int, r: int, device="cuda") -> torch.Tensor:
    """A device workspace large enough for qlora_linear_bwd_act8 over weights of N rows."""
    return torch.empty(max(qlora_workspace_bytes_act8(M, N, K, r), 256), dtype=torch.uint8, device=device)


def qlora_linear_bwd_act8(weights: list, act8: Act8, dys: list, As: list, Bs: list, scale: float, us: list, dxs,
                          dAs: list, dBs: list, accumulate: bool = False, ws=None, stream=None) -> None:
    """Backward of the linears that share the input kept as act8: as qlora_linear_bwd_group, with dAs[i]
    formed from the 8-bit codes; dxs None skips the input gradients."""
    n = len(weights)
    if not (len(dys) == len(As) == len(Bs) == len(us) == len(dAs) == len(dBs) == n) or n == 0 or \
            (dxs is not None and len(dxs) != n):
        raise ValueError("one dY, A, B, u, dA and dB (and dX) per weight, one weight at least")
    M, K = act8.M, act8.K
    r = As[0].shape[0]
    P = ctypes.c_void_p * n
    if any(w.K != K for w in weights) or any(u.numel() != M * r for u in us):
        raise ValueError("shape mismatch")
    rows_r, r_cols = [(w.N, r) for w in weights], [(r, K)] * n
    pdy = _mptrs(P, dys, _BF16, [(M, w.N) for w in weights])
    pa, pb = _mptrs(P, As, _BF16, r_cols), _mptrs(P, Bs, _BF16, rows_r)
    pu = P(*[_dptr(t, _F32) for t in us])
    pdx = None if dxs is None else _mptrs(P, dxs, _BF16, [(M, K)] * n)
    pda, pdb = _mptrs(P, dAs, _F32, r_cols), _mptrs(P, dBs, _F32, rows_r)
    if ws is None:
        ws = _scratch(max(qlora_workspace_bytes_act8(M, [w.N for w in weights], K, r), 256), act8.codes.device, stream)
    cws = [w.c_struct() for w in weights]
    x8 = act8.c_struct()
    _check(lib.qlora_linear_bwd_act8(n, P(*[ctypes.addressof(c) for c in cws]), ctypes.byref(x8), pdy, M, pa, pb, r, scale,
                                     pu, pdx, pda, pdb, int(bool(accumulate)), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)), "qlora_linear_bwd_act8")


# ------------------------------------------------------------------------- norm
def qlora_rmsnorm_fwd(x, weight, eps: float, y, residual=None, h=None, rstd=None, act8: Act8 | None = None,
                      stream=None) -> None:
    """h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight over the last dimension (M x K); h, rstd
    and the 8-bit checkpoint of y (act8) are optional outputs."""
    px, pw, py = _dptr(x, _BF16), _dptr(weight, _BF16), _dptr(y, _BF16)
    pr, ph, ps = _dptr(residual, _BF16), _dptr(h, _BF16), _dptr(rstd, _F32)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be M x K")
    M, K = shape
    if weight.numel() != K or y.shape != shape or (residual is not None and residual.shape != shape) \
            or (h is not None and h.shape != shape) or (rstd is not None and rstd.numel() != M) \
            or (act8 is not None and (act8.M, act8.K) != (M, K)):
        raise ValueError("shape mismatch")
    c8 = None if act8 is None else ctypes.byref(act8.c_struct())
    _check(lib.qlora_rmsnorm_fwd(px, pr, pw, M, K, eps, ph, py, ps, c8, _stream(stream)), "qlora_rmsnorm_fwd")


def qlora_rmsnorm_bwd(dy, h, weight, rstd, dx, dw=None, dh=None, accumulate: bool = False, ws=None,
                      stream=None) -> None:
    """Backward of qlora_rmsnorm_fwd from its h and rstd: dx (of x and of the residual alike; dh is what
    flows into h itself) and, if given, dw (float32, added to with accumulate)."""
    pdy, ph, pw, pdx = _dptr(dy, _BF16), _dptr(h, _BF16), _dptr(weight, _BF16), _dptr(dx, _BF16)
    pdh, ps, pdw = _dptr(dh, _BF16), _dptr(rstd, _F32), _dptr(dw, _F32)
    shape = h.shape
    if len(shape) != 2:
        raise ValueError("h must be M x K")
    M, K = shape
    if dy.shape != shape or dx.shape != shape or weight.numel() != K or rstd.numel() != M \
            or (dh is not None and dh.shape != shape) or (dw is not None and dw.numel() != K):
        raise ValueError("shape mismatch")
    if ws is None and dw is not None:
        ws = _scratch(max(int(lib.qlora_rmsnorm_workspace_bytes(M, K)), 256), h.device, stream)
    _check(lib.qlora_rmsnorm_bwd(pdy, pdh, ph, pw, ps, M, K, pdx, pdw, int(bool(accumulate)), _ptr(ws),
                                 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "qlora_rmsnorm_bwd")


# ------------------------------------------------------------------------- attention
class AttnSeqs:
    """The sequences of a batch for qlora_attn_fwd and qlora_attn_bwd, marshalled once (for all layers
    of a step): entries (q0, nq, k0, nk), nq query tokens from q0 and nk key tokens from k0, with the
    queries standing at the last nq key positions. causal hides later keys; window > 0 hides keys more
    than window - 1 positions back; both may be changed between calls. Layers of different sizes, and
    threads, may share one."""

    def __init__(self, seqs, causal: bool = True, window: int = 0):
        flat = []
        for s in seqs:   # any iterable, read once
            if len(s) != 4:
                raise ValueError("a sequence is (q0, nq, k0, nk)")
            flat += [int(v) for v in s]
        self.count = len(flat) // 4
        self.causal, self.window = bool(causal), int(window)
        self._seqs = (ctypes.c_int64 * max(len(flat), 4))(*flat)
        self._last = (None, None)   # what the last configuration was made of, and it
        self._plans = {}            # of the calls over 4-bit caches (_planned)

    @staticmethod
    def packed(lengths, causal: bool = True, window: int = 0) -> "AttnSeqs":
        """A packed training batch: sequences of the given lengths one after another, each attending to
        itself."""
        seqs, at = [], 0
        for n in lengths:
            seqs.append((at, n, at, n))
            at += n
        return AttnSeqs(seqs, causal, window)

    def _config(self, q, k, scale):
        """The configuration for tensors of these sizes, marshalled when anything it holds changes. The pair in
        _last is replaced whole and a configuration is never written to again: another thread's call for other
        sizes changes nothing here."""
        (tq, heads, d), (tk, kv_heads, dk) = q.shape, k.shape
        if d != dk:
            raise ValueError("shape mismatch: q and k differ in head size")
        key = (tq, heads, d, tk, kv_heads, scale, self.causal, self.window)
        last, cfg = self._last
        if last != key:
            cfg = CAttnConfig(heads, kv_heads, d, int(bool(self.causal)), int(self.window),
                              d ** -0.5 if scale is None else scale, tq, tk)
            self._last = (key, cfg)
        return ctypes.byref(cfg)

    def workspace_bytes(self, q, k, backward: bool = False, scale: float | None = None) -> int:
        """Of a call with these queries and keys; of qlora_attn_kv4_fwd if k is a Kv4."""
        if isinstance(k, Kv4):
            return int(lib.qlora_attn_kv4_workspace_bytes(self._config(q, k, scale), self.count, self._seqs, k.codebook))
        return int(lib.qlora_attn_workspace_bytes(self._config(q, k, scale), self.count, self._seqs,
                                                  int(bool(backward))))


def _attn_tensors(*pairs):
    """The qlora_attn_tensor structures of (tensor, shape it must have) pairs: the array that holds them, to be
    kept until the library has read them, then the address of each. The tensors are [tokens, heads, d], tokens
    and heads may be strided, d is contiguous."""
    v = array("q")
    for t, shape in pairs:
        if t.dtype not in _BF16:
            _dtype(t, *_BF16)
        if not t.is_cuda:
            raise ValueError("tensor must live on the GPU")
        if t.shape != shape or len(shape) != 3:
            raise ValueError("shape mismatch: attention tensors are [tokens, heads, d] with d contiguous")
        token, head, one = t.stride()
        if one != 1:
            raise ValueError("shape mismatch: attention tensors are [tokens, heads, d] with d contiguous")
        tokens, heads, d = shape
        # the stride of a single head or token carries no meaning: give it a valid value
        if heads <= 1:
            head = d
        if tokens <= 1:
            token = max(d, head * (heads - 1) + d) if head * heads < 1 << 22 else d
        v.extend((t.data_ptr(), token, head))
    at = v.buffer_info()[0]
    return [v, *range(at, at + 24 * len(pairs), 24)]


def _planned(plans, head, tensors, make):
    """What make() marshals for tensors [tokens, heads, d] (None: not there), kept in `plans` by `head` and all of the tensors
    that it may depend on, which their memory is not; their qlora_attn_tensor structures as an array, to be kept until
    the library has read them, and the array's address, 24 bytes for each."""
    key = [*head]
    for t in tensors:
        key += (t.shape, t.stride(), t.dtype, t.get_device()) if t is not None else (None,)
    key = tuple(key)
    plan = plans.get(key)
    if plan is None:
        made, v = make(), array("q")
        for t in tensors:
            v.extend(_attn_tensors((t, t.shape))[0] if t is not None else (0, 0, 0))
            v[-3] = 0
            if t is not None and t.get_device() != tensors[0].get_device():
                raise ValueError("the tensors must live on one GPU")
        if len(plans) >= 256:   # a program of ever new shapes
            plans.clear()
        plans[key] = plan = v, made
    v, i = plan[0][:], 0
    for t in tensors:
        if t is not None:
            v[i] = t.data_ptr()
        i += 3
    return plan[1], v, v.buffer_info()[0]


def _lse_ptr(lse, q):
    if lse is not None and lse.shape != (q.shape[1], q.shape[0]):
        raise ValueError("lse must be [heads, query tokens]")
    return _dptr(lse, _F32)


def _attn_ws(seqs, cfg, backward, ws, device, stream):
    if ws is None:
        need = int(lib.qlora_attn_workspace_bytes(cfg, seqs.count, seqs._seqs, backward))
        if not need:
            return None, None, 0
        ws = _scratch(need, device, stream)
    return ws, _ptr(ws), ws.numel() * ws.element_size()


def qlora_attn_fwd(seqs: AttnSeqs, q, k, v, o, lse=None, scale: float | None = None, ws=None, stream=None) -> None:
    """Attention of seqs: q, o [query tokens, heads, d], k, v [key tokens, kv heads, d] (bf16, tokens and
    heads may be strided); lse [heads, query tokens] float32 is needed by the backward. scale defaults
    to d ** -0.5."""
    keep, tq, tk, tv, to = _attn_tensors((q, q.shape), (k, k.shape), (v, k.shape), (o, q.shape))
    cfg = seqs._config(q, k, scale)
    plse = _lse_ptr(lse, q)
    ws, pws, nbytes = _attn_ws(seqs, cfg, 0, ws, q.device, stream)
    _check(lib.qlora_attn_fwd(cfg, seqs.count, seqs._seqs, tq, tk, tv, to, plse, pws, nbytes, _stream(stream)),
           "qlora_attn_fwd")


def qlora_attn_bwd(seqs: AttnSeqs, q, k, v, o, lse, dout, dq, dk, dv, scale: float | None = None, ws=None,
                   stream=None) -> None:
    """Backward of qlora_attn_fwd: dq, dk, dv from the gradient dout of o, recomputing the probabilities
    from lse."""
    if lse is None:
        raise ValueError("the backward needs lse")
    sq, sk = q.shape, k.shape
    keep, *ts = _attn_tensors((q, sq), (k, sk), (v, sk), (o, sq), (dout, sq), (dq, sq), (dk, sk), (dv, sk))
    cfg = seqs._config(q, k, scale)
    plse = _lse_ptr(lse, q)
    ws, pws, nbytes = _attn_ws(seqs, cfg, 1, ws, q.device, stream)
    _check(lib.qlora_attn_bwd(cfg, seqs.count, seqs._seqs, *ts[:4], plse, *ts[4:], pws, nbytes, _stream(stream)),
           "qlora_attn_bwd")


# ------------------------------------------------------------------------- rotary positions
class Rope:
    """Rotary positions, marshalled once (for all layers of a model; not changed afterwards): the first `rot`
    features of a head in pairs, (2i, 2i+1) if interleaved, else (i, i + rot/2), pair i turned by inv_freq[i] radians
    a position, by default base ** (-2 i / rot). `factor` multiplies the rotated features.

    For contexts longer than the model was trained on, `stretch` divides the frequencies: all of them when `trained`
    is 0 (positions are interpolated); else those that make less than `low` turns in `trained` positions, while
    those that make more than `high` stay, and in between the share that stays grows linearly with the turns."""

    def __init__(self, rot: int, base: float = 10000.0, interleaved: bool = False, stretch: float = 1.0, trained: int = 0,
                 low: float = 1.0, high: float = 4.0, factor: float = 1.0, inv_freq=None):
        self._made = int(rot), bool(interleaved), float(factor)
        if inv_freq is None:
            if not stretch > 0 or not base > 0 or (trained and not high > low):
                raise ValueError("base and stretch must be above 0, and high above low")
            inv_freq = []
            for i in range(self.rot // 2):
                f = float(base) ** (-2.0 * i / self.rot)
                keep = min(1.0, max(0.0, (trained * f / (2 * math.pi) - low) / (high - low))) if trained else 0.0
                inv_freq.append(f * (keep + (1.0 - keep) / stretch))
        self._inv_freq = tuple(float(f) for f in inv_freq)
        if len(self._inv_freq) * 2 != self.rot:
            raise ValueError("one frequency for each of the rot / 2 pairs")
        self._freq = (ctypes.c_double * max(len(self._inv_freq), 1))(*self._inv_freq)
        self._plans = {}

    # what the plans were made with: read only
    rot = property(lambda self: self._made[0])
    interleaved = property(lambda self: self._made[1])
    factor = property(lambda self: self._made[2])
    inv_freq = property(lambda self: self._inv_freq)

    def _planned(self, eps, qs, ks):
        """_planned for a call's query-like and key-like tensors, which must be alike: with the configuration, the tokens and the
        bytes of the backward's workspace."""
        def make():
            q, k = qs[0], ks[0]
            for ts, like in ((qs, q), (ks, k)):
                for t in ts:
                    if t is not None and (like is None or t.dim() != 3 or t.shape != like.shape):
                        raise ValueError("shape mismatch: heads are [tokens, heads, d], gradients and outputs like their inputs")
            if any((t is None) != (k is None) for t in ks[:2]) or (k is not None and (k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2])):
                raise ValueError("shape mismatch: keys go with keys, of the queries' tokens and head size")
            tokens, heads, d = q.shape
            cfg = CRopeConfig(heads, 0 if k is None else k.shape[1], d, self.rot, int(self.interleaved), eps, self.factor, tokens)
            return ctypes.byref(cfg), tokens, self.workspace_bytes(q, k)
        return _planned(self._plans, (eps,), qs + ks, make)

    def workspace_bytes(self, q, k=None) -> int:
        """Of qlora_rope_bwd for weights' gradients."""
        tokens, heads, d = q.shape
        cfg = CRopeConfig(heads, 0 if k is None else k.shape[1], d, self.rot, int(self.interleaved), 0.0, self.factor, tokens)
        return int(lib.qlora_rope_workspace_bytes(ctypes.byref(cfg)))


def _rope_positions(rope, positions, tokens):
    if positions is None:
        if rope.rot:
            raise ValueError("positions are needed to rotate")
        return None
    if positions.shape != (tokens,):
        raise ValueError("positions must hold one value a token")
    return _dptr(positions, (torch.int64,))


def _rope_weight(w, like):
    if w is None:
        return None
    if like is None or w.numel() != like.shape[2]:
        raise ValueError("a head weight must hold d values")
    return _dptr(w, _BF16)


def qlora_rope_fwd(rope: Rope, positions, q, k, q_out, k_out, q_weight=None, k_weight=None, eps: float = 1e-6,
                   stream=None) -> None:
    """Query and key heads [tokens, heads, d] (bf16, tokens and heads may be strided), normed over d where a weight
    [d] is given, then rotated by their tokens' positions (int64 [tokens]). k and k_out may be None; an output may
    be its input."""
    (cfg, tokens, _), keep, at = rope._planned(eps, (q, q_out), (k, k_out))
    tk, tko = (None, None) if k is None else (at + 48, at + 72)
    _check(lib.qlora_rope_fwd(cfg, rope._freq, _rope_positions(rope, positions, tokens), at, tk, _rope_weight(q_weight, q),
                              _rope_weight(k_weight, k), at + 24, tko,
                              _stream_on(stream, q.get_device(), positions, q_weight, k_weight)), "qlora_rope_fwd")


def qlora_rope_bwd(rope: Rope, positions, dq_out, dk_out, dq, dk, q=None, k=None, q_weight=None, k_weight=None,
                   dq_weight=None, dk_weight=None, eps: float = 1e-6, accumulate: bool = False, ws=None,
                   stream=None) -> None:
    """Backward of qlora_rope_fwd: dq, dk from the gradients dq_out, dk_out of its outputs, and, where asked for, the
    weights' (float32 [d], added to with accumulate). Normed heads need the forward's inputs q and k."""
    if (q_weight is not None and q is None) or (k_weight is not None and k is None):
        raise ValueError("the backward of normed heads needs their inputs")
    (cfg, tokens, need), keep, at = rope._planned(
        eps, (dq_out, dq, q if q_weight is not None else None), (dk_out, dk, k if k_weight is not None else None))
    tgk, tdk = (None, None) if dk_out is None else (at + 72, at + 96)
    tq, tk = None if q_weight is None else at + 48, None if k_weight is None else at + 120
    pdw = None, None
    nbytes = 0
    if dq_weight is not None or dk_weight is not None:
        for dw, w in ((dq_weight, q_weight), (dk_weight, k_weight)):
            if dw is not None and (w is None or dw.numel() != w.numel()):
                raise ValueError("a head weight's gradient goes with the weight and holds d values")
        pdw = _dptr(dq_weight, _F32), _dptr(dk_weight, _F32)
        if ws is None:
            ws = _scratch(max(need, 256), dq.device, stream)
        nbytes = ws.numel() * ws.element_size()
    _check(lib.qlora_rope_bwd(cfg, rope._freq, _rope_positions(rope, positions, tokens), tq, tk, _rope_weight(q_weight, dq_out),
                              _rope_weight(k_weight, dk_out), at, tgk, at + 24, tdk, *pdw, int(bool(accumulate)),
                              None if ws is None else _ptr(ws), nbytes,
                              _stream_on(stream, dq.get_device(), positions, q_weight, k_weight, dq_weight, dk_weight, ws)),
           "qlora_rope_bwd")


# ------------------------------------------------------------------------- a key/value cache in 4 bits
class Kv4:
    """The keys or the values of a cache in 4 bits: codes uint8 [tokens, kv_heads, blocks, 16] and absmax bf16
    [tokens, kv_heads, blocks] for blocks of 32 along the head (format in include/qlora_nf4.h). Tokens and heads
    may be strided, in the same way in both; empty_kv4 makes one whose heads come first in memory."""

    def __init__(self, codes, absmax, d: int, codebook="nf4"):
        nb = (int(d) + 31) // 32
        _dtype(codes, torch.uint8)
        _dtype(absmax, *_BF16)
        if codes.dim() != 4 or absmax.dim() != 3 or codes.shape[:3] != absmax.shape or codes.shape[2:] != (nb, 16):
            raise ValueError(f"codes must be [tokens, kv_heads, {nb}, 16] and absmax [tokens, kv_heads, {nb}]")
        if not codes.is_cuda or codes.device != absmax.device:
            raise ValueError("codes and absmax must live on one GPU")
        tokens, heads = codes.shape[:2]
        ts, hs, bs, one = codes.stride()
        at, ah, ab = absmax.stride()
        # the stride of a single head, token or block carries no meaning: give it a valid value
        if heads <= 1:
            hs, ah = 16 * nb, nb
        if tokens <= 1:
            ts = at = max(nb, ah * (heads - 1) + nb)
            ts, at = (16 * at, at) if at < 1 << 20 else (16 * nb, nb)
        if nb == 1:
            bs, ab = 16, 1
        if one != 1 or bs != 16 or ab != 1 or (ts, hs) != (16 * at, 16 * ah):
            raise ValueError("codes and absmax must have whole blocks and the same order of tokens and heads")
        self.codes, self.absmax, self.d, self.codebook = codes, absmax, int(d), _book(codebook)
        self.shape = (tokens, heads, self.d)
        self._c = CKv4(codes.data_ptr(), absmax.data_ptr(), at, ah, self.codebook)
        self._ptr = ctypes.byref(self._c)


def empty_kv4(tokens: int, kv_heads: int, d: int, device="cuda", codebook="nf4") -> Kv4:
    """An uninitialised 4-bit cache for `tokens` keys or values of kv_heads heads of size d."""
    nb = (d + 31) // 32
    return Kv4(torch.empty(kv_heads, tokens, nb, 16, dtype=torch.uint8, device=device).permute(1, 0, 2, 3),
               torch.empty(kv_heads, tokens, nb, dtype=torch.bfloat16, device=device).permute(1, 0, 2), d, codebook)


def _kv4_planned(seqs, tensors, heads, k4, v4, scale, need):
    """_planned for a call over a cache, whose k4 and v4 must be alike and go with the tensors: with the configuration and,
    if need, the bytes of the attention's workspace."""
    def make():
        t = tensors[0]
        if t.dim() != 3 or any(x.shape != t.shape for x in tensors):
            raise ValueError("shape mismatch: the tensors are [tokens, heads, d] and alike")
        if k4.shape != v4.shape or k4.codebook != v4.codebook:
            raise ValueError("k4 and v4 must be alike")
        if k4.d != t.shape[2] or (heads and k4.shape[1] != t.shape[1]):
            raise ValueError("shape mismatch between the cache and the tensors")
        cfg = seqs._config(t, k4, scale)
        return cfg, int(lib.qlora_attn_kv4_workspace_bytes(cfg, seqs.count, seqs._seqs, k4.codebook)) if need else 0
    return _planned(seqs._plans, (need, scale, seqs.causal, seqs.window, k4.shape, v4.shape, k4.codebook, v4.codebook), tensors, make)


def qlora_kv4_write(seqs: AttnSeqs, k, v, k4: Kv4, v4: Kv4, stream=None) -> None:
    """New keys and values k, v [tokens, kv heads, d] (bf16, strided) into a 4-bit cache: the nq tokens of every
    sequence (q0, nq, k0, nk) become its last nq keys, so the list that the attention then takes says where."""
    (cfg, _), keep, at = _kv4_planned(seqs, (k, v), True, k4, v4, None, False)
    _check(lib.qlora_kv4_write(cfg, seqs.count, seqs._seqs, at, at + 24, k4._ptr, v4._ptr,
                               _stream_on(stream, k.get_device(), k4.codes, v4.codes)), "qlora_kv4_write")


def qlora_kv4_read(seqs: AttnSeqs, k4: Kv4, v4: Kv4, k, v, stream=None) -> None:
    """The last nq keys and values of every sequence out of a 4-bit cache, in bf16: into tokens q0 .. of k and v."""
    (cfg, _), keep, at = _kv4_planned(seqs, (k, v), True, k4, v4, None, False)
    _check(lib.qlora_kv4_read(cfg, seqs.count, seqs._seqs, k4._ptr, v4._ptr, at, at + 24,
                              _stream_on(stream, k.get_device(), k4.codes, v4.codes)), "qlora_kv4_read")


def qlora_attn_kv4_fwd(seqs: AttnSeqs, q, k4: Kv4, v4: Kv4, o, lse=None, scale: float | None = None, ws=None,
                       stream=None) -> None:
    """qlora_attn_fwd over a 4-bit cache: q, o [query tokens, heads, d] (bf16, strided)."""
    (cfg, need), keep, at = _kv4_planned(seqs, (q, o), False, k4, v4, scale, True)
    plse = None if lse is None else _lse_ptr(lse, q)
    pws, nbytes = None, 0
    if ws is None and need:
        ws = _scratch(need, q.device, stream)
    if ws is not None:
        pws, nbytes = _ptr(ws), ws.numel() * ws.element_size()
    _check(lib.qlora_attn_kv4_fwd(cfg, seqs.count, seqs._seqs, at, k4._ptr, v4._ptr, at + 24, plse, pws, nbytes,
                                  _stream_on(stream, q.get_device(), k4.codes, v4.codes, lse, ws)), "qlora_attn_kv4_fwd")


# ------------------------------------------------------------------------- format variants
Q4_CODEBOOKS = {"nf4": 0, "fp4": 1, "int4": 2}


def _book(codebook) -> int:
    if isinstance(codebook, str):
        if codebook not in Q4_CODEBOOKS:
            raise ValueError(f"codebook must be one of {sorted(Q4_CODEBOOKS)}")
        return Q4_CODEBOOKS[codebook]
    return int(codebook)


def q4_codebook_values(codebook) -> list:
    out = (ctypes.c_float * 16)()
    n = lib.q4_codebook_values(_book(codebook), out)
    if n < 0:
        raise NF4Error(-n, "q4_codebook_values")
    return list(out)[:n]


def q4_quantize(w, codebook, blocksize: int, packed, absmax, stream=None) -> None:
    """Blockwise absmax quantisation with the NF4, FP4 or INT4 codebook and blocksize 16..4096."""
    _dtype(w, torch.float32); _dtype(packed, torch.uint8); _dtype(absmax, torch.float32)
    n = w.numel()
    if packed.numel() * 2 != n or absmax.numel() * blocksize != n:
        raise ValueError("output sizes must be numel/2 and numel/blocksize")
    _check(lib.q4_quantize(_ptr(w), n, _book(codebook), blocksize, _ptr(packed), _ptr(absmax),
                           _stream(stream)), "q4_quantize")


def q4_dequant(packed, numel: int, codebook, blocksize: int, out, absmax=None, scale_q=None,
               scale_c2=None, stream=None) -> None:
    """bf16 weights from packed indices and either fp32 scales (absmax) or double-quantised ones
    (scale_q, scale_c2)."""
    _dtype(packed, torch.uint8); _dtype(out, *_BF16); _dtype(absmax, torch.float32)
    _dtype(scale_q, torch.uint8); _dtype(scale_c2, torch.float32)
    if packed.numel() * 2 != numel or out.numel() != numel:
        raise ValueError("packed must hold numel/2 bytes and out numel values")
    nb = numel // blocksize
    if (absmax is not None and absmax.numel() != nb) or (scale_q is not None and scale_q.numel() != nb) \
            or (scale_c2 is not None and scale_c2.numel() != (nb + 255) // 256):
        raise ValueError("scale sizes do not match numel / blocksize")
    _check(lib.q4_dequant(_ptr(packed), numel, _book(codebook), blocksize, _ptr(absmax), _ptr(scale_q),
                          _ptr(scale_c2), _ptr(out), _stream(stream)), "q4_dequant")


# ------------------------------------------------------------------------- the adapter update
@dataclass(frozen=True)
class AdamWConfig:
    """Hyper-parameters of the adapter update; lr and the clipping threshold are the ones "QLoRA,
    explained" gives (The algorithm, step by step; Minimal implementation), the rest torch's AdamW
    defaults."""
    lr: float = 2e-4
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.01
    max_grad_norm: float = 0.3   # <= 0: no clipping

    def c_struct(self) -> CAdamWConfig:
        return CAdamWConfig(self.lr, self.beta1, self.beta2, self.eps, self.weight_decay,
                            self.max_grad_norm)


def _ptr_array(tensors, dtypes, allow_none=False):
    arr = (ctypes.c_void_p * len(tensors))()
    for i, t in enumerate(tensors):
        if t is None and allow_none:
            arr[i] = None
            continue
        _dtype(t, *dtypes)
        arr[i] = _ptr(t)
    return arr


class AdamWPlan:
    """qlora_adamw_plan over a set of adapter tensors (fp32 master weights, gradients, first and
    second moments, optional bf16 copies): one call runs the clipped AdamW step over all of them
    in three kernel launches. The tensors must stay alive, at the same storage, while the plan is
    used; the plan keeps references to them."""

    def __init__(self, params, grads, exp_avg, exp_avg_sq, params_bf16=None,
                 cfg: AdamWConfig = AdamWConfig()):
        n = len(params)
        if not (len(grads) == len(exp_avg) == len(exp_avg_sq) == n) or n == 0 or \
                (params_bf16 is not None and len(params_bf16) != n):
            raise ValueError("tensor lists differ in length or are empty")
        for i in range(n):
            sizes = [grads[i].numel(), exp_avg[i].numel(), exp_avg_sq[i].numel()]
            if params_bf16 is not None and params_bf16[i] is not None:
                sizes.append(params_bf16[i].numel())
            if any(k != params[i].numel() for k in sizes):
                raise ValueError(f"tensor {i}: sizes differ")
        self._keep = (list(params), list(grads), list(exp_avg), list(exp_avg_sq),
                      None if params_bf16 is None else list(params_bf16))
        self.cfg = cfg
        self._ccfg = cfg.c_struct()
        f32 = (torch.float32,)
        pb = None if params_bf16 is None else _ptr_array(params_bf16, _BF16, allow_none=True)
        numel = (ctypes.c_int64 * n)(*[t.numel() for t in params])
        handle = ctypes.c_void_p()
        with torch.cuda.device(params[0].device):
            _check(lib.qlora_adamw_plan_create(n, _ptr_array(params, f32), _ptr_array(grads, f32),
                                               _ptr_array(exp_avg, f32), _ptr_array(exp_avg_sq, f32),
                                               pb, numel, ctypes.byref(handle)),
                   "qlora_adamw_plan_create")
        self._handle = handle
        self.values = sum(t.numel() for t in params)

    def step(self, step: int, grad_norm=None, stream=None) -> None:
        """AdamW step number `step` (from 1); grad_norm (one float64 on the device) receives the
        gradient norm before clipping."""
        _dtype(grad_norm, torch.float64)
        _check(lib.qlora_adamw_plan_step(self._handle, ctypes.byref(self._ccfg), int(step),
                                         _ptr(grad_norm), _stream(stream)), "qlora_adamw_plan_step")

    def close(self) -> None:
        if getattr(self, "_handle", None) is not None and self._handle.value:
            lib.qlora_adamw_plan_destroy(self._handle)
        self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # pragma: no cover - interpreter shutdown
            pass


# ------------------------------------------------------------------------- helpers
def qlora_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return int(lib.qlora_workspace_bytes(M, N, K, r))


def nf4_storage_bytes(numel: int) -> int:
    return int(lib.nf4_storage_bytes(numel))


def nf4_codebook() -> list:
    out = (ctypes.c_float * 16)()
    lib.nf4_codebook(out)
    return list(out)


def workspace(M: int, N: int, K: int, r: int, device="cuda") -> torch.Tensor:
    """A device workspace large enough for qlora_linear_fwd/bwd at these sizes."""
    nbytes = max(qlora_workspace_bytes(M, N, K, r), 256)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def empty_weight(N: int, K: int, device="cuda", codebook=0) -> NF4Weight:
    nb = N * K // 64
    return NF4Weight(torch.empty(N * K // 2, dtype=torch.uint8, device=device),
                     torch.empty(nb, dtype=torch.uint8, device=device),
                     torch.empty((nb + 255) // 256, dtype=torch.float32, device=device), N, K,
                     codebook=_book(codebook))


def quantize_weight(w: torch.Tensor, stream=None, absmax: torch.Tensor | None = None,
                    double_quant: bool = True, codebook=0) -> NF4Weight:
    """Quantise a float32 N x K device tensor: nf4_quantize (q4_quantize at blocksize 64 for the FP4
    or INT4 codebook) followed by nf4_double_quant, or with double_quant=False a weight that keeps
    the fp32 absmax as its scales. As under torch.cuda.stream(stream), the weight's memory comes from
    the pool of the stream it is written on."""
    N, K = w.shape
    book = _book(codebook)
    with _pool_of(stream, w.device):
        if absmax is None:
            absmax = torch.empty(N * K // 64, dtype=torch.float32, device=w.device)
        if not double_quant:
            qw = NF4Weight(torch.empty(N * K // 2, dtype=torch.uint8, device=w.device), None, None, N, K, absmax,
                           codebook=book)
        else:
            qw = empty_weight(N, K, w.device, book)
    if book == 0:
        nf4_quantize(w, qw.packed, absmax, stream)
    else:
        q4_quantize(w, book, 64, qw.packed, absmax, stream)
    if double_quant:
        nf4_double_quant(absmax, qw.scale_q, qw.scale_c2, stream)
    return qw


__all__ = ["lib", "LIB_PATH", "EXPORTED", "NF4Error", "NF4Weight", "CNF4Weight", "nf4_quantize",
           "nf4_quantize_bf16",
           "nf4_double_quant", "nf4_double_quant_many", "DoubleQuantMany", "nf4_dequant", "qlora_linear_fwd", "qlora_linear_fwd_noalloc",
           "qlora_linear_fwd_recompute", "qlora_linear_fwd_group", "qlora_linear_fwd_recompute_group",
           "qlora_workspace_bytes_group", "qlora_linear_bwd_group",
           "workspace_group",
           "qlora_linear_bwd", "qlora_merge", "AdamWConfig", "CAdamWConfig", "AdamWPlan",
           "Q4_CODEBOOKS", "q4_codebook_values", "q4_quantize", "q4_dequant",
           "Act8", "CAct8", "empty_act8", "qlora_act8_pack", "qlora_act8_unpack", "qlora_linear_bwd_act8",
           "qlora_workspace_bytes_act8", "workspace_act8", "qlora_rmsnorm_fwd", "qlora_rmsnorm_bwd",
           "AttnSeqs", "CAttnConfig", "CAttnTensor", "qlora_attn_fwd", "qlora_attn_bwd",
           "Rope", "CRopeConfig", "qlora_rope_fwd", "qlora_rope_bwd", "Kv4", "CKv4", "empty_kv4", "qlora_kv4_write",
           "qlora_kv4_read", "qlora_attn_kv4_fwd",
           "qlora_workspace_bytes", "nf4_storage_bytes", "nf4_codebook", "workspace",
           "empty_weight", "quantize_weight"]
