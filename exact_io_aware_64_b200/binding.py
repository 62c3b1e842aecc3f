"""ctypes binding for libfa.so (include/fa.h).

Argument marshalling only: it checks that tensors are CUDA, contiguous and of the right
shape and dtype, allocates outputs with torch when the caller does not pass them, and
hands raw pointers and the current CUDA stream to the C ABI.  Every step of the
computation runs in the library's kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_TIMEOUT = 4

_lib = None
_fns = {}  # the library's functions that _run has looked up

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_ll = ctypes.c_longlong

SIGNATURES = {
    "fa_abi_version": ([], _i),
    "fa_fwd": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_fwd_qk": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_fwd_varlen": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp],
                      _i),
    "fa_fwd_packed": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i,
                       _vp], _i),
    "fa_fwd_f32": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_fwd_f32_qk": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_fwd_f32_varlen": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i,
                           _vp], _i),
    "fa_fwd_f32_packed": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f,
                           _i, _vp], _i),
    "fa_bwd_workspace_bytes": ([_i, _i, _i, _i], _sz),
    "fa_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _sz,
                _vp], _i),
    "fa_bwd_qk": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp,
                   _sz, _vp], _i),
    "fa_bwd_varlen": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                       _i, _f, _i, _vp, _sz, _vp], _i),
    "fa_bwd_packed": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                       _i, _i, _i, _f, _i, _vp, _sz, _vp], _i),
    "fa_bwd_f32": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp,
                    _sz, _vp], _i),
    "fa_bwd_f32_qk": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i,
                       _vp, _sz, _vp], _i),
    "fa_bwd_f32_varlen": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i,
                           _i, _i, _f, _i, _vp, _sz, _vp], _i),
    "fa_bwd_f32_packed": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i,
                           _i, _i, _i, _i, _f, _i, _vp, _sz, _vp], _i),
    "fa_doc_ranges": ([_vp, _vp, _vp, _i, _i, _vp], _i),
    "fa_fwd_mod": ([_vp] * 9 + [_i] * 6 + [_f, _i, _f, _vp], _i),
    "fa_bwd_mod": ([_vp] * 13 + [_i] * 6 + [_f, _i, _f, _vp, _sz, _vp], _i),
    "fa_rotary": ([_vp] * 6 + [_ll] + [_i] * 8 + [_f, _vp, _vp, _vp], _i),
    "fa_rotary_f32": ([_vp] * 6 + [_ll] + [_i] * 8 + [_f, _vp, _vp, _vp], _i),
    "fa_fwd_tree_workspace_bytes": ([_i] * 5, _sz),
    "fa_fwd_tree": ([_vp] * 9 + [_i] * 8 + [_f, _f, _vp, _sz, _vp], _i),
    "fa_merge": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp], _i),
    "fa_accumulate": ([_vp, _vp, _vp, _sz, _vp], _i),
    "fa_selftest_timeout": ([ctypes.c_longlong, _vp], _i),
    "fa_bwd_noalloc": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i,
                        _vp], _i),
    "fa_bwd_noalloc_max_scratch_bytes": ([], _sz),
    "fa_trace_events": ([ctypes.POINTER(_vp), _i], _i),
    "fa_status_string": ([_i], ctypes.c_char_p),
    "fa_last_error_message": ([], ctypes.c_char_p),
    "fa_check_device_error": ([_vp], _i),
}


class FAError(RuntimeError):
    def __init__(self, call: str, status: int, message: str):
        super().__init__(f"{call} failed: {status_name(status)}: {message}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libfa.so (built in place by ``python -m exact_io_aware_64_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with python -m exact_io_aware_64_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def status_name(status: int) -> str:
    return lib().fa_status_string(status).decode()


def _check(call: str, status: int) -> None:
    if status != FA_OK:
        raise FAError(call, status, lib().fa_last_error_message().decode())


def _stream_handle(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _run(name: str, device: torch.device, stream: Optional[torch.cuda.Stream], *args) -> None:
    """Call ``name`` on ``stream`` (default: the current stream of ``device``) with
    ``device`` current.  The host's part of a small call takes longer than its kernel, so
    nothing is looked up twice: the raw handle of the current stream instead of a Stream
    object (0.2 us against 7 us), and no device change where the device is current."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    index = device.index
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device_index != index:
        raise ValueError(f"stream is on device {stream.device_index}, the tensors on {index}")
    else:
        handle = stream.cuda_stream
    if torch.cuda.current_device() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != FA_OK:
        _check(name, st)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_bhnd(name: str, t: torch.Tensor, shape, dtype) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fwd(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, scale: Optional[float] = None,
        causal: bool = False, O: Optional[torch.Tensor] = None,
        LSE: Optional[torch.Tensor] = None, want_lse: bool = True,
        stream: Optional[torch.cuda.Stream] = None):
    """Exact attention forward through ``fa_fwd`` / ``fa_fwd_qk`` (bf16; the latter when
    Nq != Nk) or ``fa_fwd_f32`` / ``fa_fwd_f32_qk`` (float32).

    Q: [B, H, Nq, d]; K, V: [B, H, Nk, d]; CUDA tensors, contiguous, all bf16 or all
    float32.  With Nq != Nk the queries are the last Nq of the Nk tokens (causal masking
    aligned at the bottom right).
    Returns (O, LSE); LSE is None when ``want_lse`` is False and none is passed.
    """
    B, H, Nq, d = Q.shape
    Nk = K.shape[2]
    dtype = Q.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("Q, K, V must be bfloat16 or float32")
    _check_bhnd("Q", Q, (B, H, Nq, d), dtype)
    for name, t in (("K", K), ("V", V)):
        _check_bhnd(name, t, (B, H, Nk, d), dtype)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    _check_bhnd("O", O, (B, H, Nq, d), dtype)
    if LSE is None and want_lse:
        LSE = torch.empty((B, H, Nq), device=Q.device, dtype=torch.float32)
    if LSE is not None:
        _check_bhnd("LSE", LSE, (B, H, Nq), torch.float32)
    with torch.cuda.device(Q.device):
        if dtype == torch.float32 and Nq == Nk:
            name = "fa_fwd_f32"
            st = lib().fa_fwd_f32(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, H, Nq, d,
                                  float(scale), int(bool(causal)), _stream_handle(stream))
        elif dtype == torch.float32:
            name = "fa_fwd_f32_qk"
            st = lib().fa_fwd_f32_qk(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, H, Nq,
                                     Nk, d, float(scale), int(bool(causal)),
                                     _stream_handle(stream))
        elif Nq == Nk:
            name = "fa_fwd"
            st = lib().fa_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, H, Nq, d,
                              float(scale), int(bool(causal)), _stream_handle(stream))
        else:
            name = "fa_fwd_qk"
            st = lib().fa_fwd_qk(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, H, Nq, Nk,
                                 d, float(scale), int(bool(causal)), _stream_handle(stream))
    _check(name, st)
    return O, LSE


def workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, H, N, d))


def bwd(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor,
        dO: torch.Tensor, LSE: torch.Tensor, scale: Optional[float] = None,
        causal: bool = False, dQ: Optional[torch.Tensor] = None,
        dK: Optional[torch.Tensor] = None, dV: Optional[torch.Tensor] = None,
        workspace: Optional[torch.Tensor] = None,
        stream: Optional[torch.cuda.Stream] = None):
    """Exact attention backward through ``fa_bwd`` / ``fa_bwd_qk`` (bf16; the latter when
    Nq != Nk) or ``fa_bwd_f32`` / ``fa_bwd_f32_qk`` (float32).

    Q, O, dO: [B, H, Nq, d]; K, V: [B, H, Nk, d]; CUDA tensors, contiguous, all bf16 or
    all float32; LSE: [B, H, Nq] float32.  Returns (dQ, dK, dV) in the inputs' dtype."""
    B, H, Nq, d = Q.shape
    Nk = K.shape[2]
    dtype = Q.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("Q, K, V, O, dO must be bfloat16 or float32")
    for name, t in (("Q", Q), ("O", O), ("dO", dO)):
        _check_bhnd(name, t, (B, H, Nq, d), dtype)
    for name, t in (("K", K), ("V", V)):
        _check_bhnd(name, t, (B, H, Nk, d), dtype)
    _check_bhnd("LSE", LSE, (B, H, Nq), torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    _check_bhnd("dQ", dQ, (B, H, Nq, d), dtype)
    for name, t in (("dK", dK), ("dV", dV)):
        _check_bhnd(name, t, (B, H, Nk, d), dtype)
    need = workspace_bytes(B, H, Nq, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=Q.device, dtype=torch.uint8)
    ws_bytes = workspace.numel() * workspace.element_size()
    ptrs = (_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(LSE), _ptr(dQ), _ptr(dK),
            _ptr(dV))
    tail = (float(scale), int(bool(causal)), _ptr(workspace), ws_bytes, _stream_handle(stream))
    with torch.cuda.device(Q.device):
        if dtype == torch.float32 and Nq == Nk:
            name = "fa_bwd_f32"
            st = lib().fa_bwd_f32(*ptrs, B, H, Nq, d, *tail)
        elif dtype == torch.float32:
            name = "fa_bwd_f32_qk"
            st = lib().fa_bwd_f32_qk(*ptrs, B, H, Nq, Nk, d, *tail)
        elif Nq == Nk:
            name = "fa_bwd"
            st = lib().fa_bwd(*ptrs, B, H, Nq, d, *tail)
        else:
            name = "fa_bwd_qk"
            st = lib().fa_bwd_qk(*ptrs, B, H, Nq, Nk, d, *tail)
    _check(name, st)
    return dQ, dK, dV


def bwd_noalloc(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor,
                dO: torch.Tensor, LSE: torch.Tensor, scale: Optional[float] = None,
                causal: bool = False, dQ: Optional[torch.Tensor] = None,
                dK: Optional[torch.Tensor] = None, dV: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """Backward through ``fa_bwd_noalloc``: the library's fixed scratch replaces the
    workspace, for callers that cannot allocate device memory.  Outputs may be passed in
    so that nothing is allocated here either.  Returns (dQ, dK, dV)."""
    B, H, N, d = Q.shape
    for name, t in (("Q", Q), ("K", K), ("V", V), ("O", O), ("dO", dO)):
        _check_bhnd(name, t, (B, H, N, d), torch.bfloat16)
    _check_bhnd("LSE", LSE, (B, H, N), torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    for name, t in (("dQ", dQ), ("dK", dK), ("dV", dV)):
        _check_bhnd(name, t, (B, H, N, d), torch.bfloat16)
    with torch.cuda.device(Q.device):
        st = lib().fa_bwd_noalloc(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(LSE),
                                  _ptr(dQ), _ptr(dK), _ptr(dV), B, H, N, d, float(scale),
                                  int(bool(causal)), _stream_handle(stream))
    _check("fa_bwd_noalloc", st)
    return dQ, dK, dV


def _layout_dtype(Q: torch.Tensor) -> torch.dtype:
    if Q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("Q, K, V must be bfloat16 or float32")
    return Q.dtype


def _check_seqlens(seqlens_q: torch.Tensor, seqlens_k: torch.Tensor, B: int, device) -> None:
    for name, t in (("seqlens_q", seqlens_q), ("seqlens_k", seqlens_k)):
        if not t.is_cuda or t.device != device:
            raise ValueError(f"{name} must be on the inputs' CUDA device")
        if t.dtype != torch.int32 or tuple(t.shape) != (B,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor of shape ({B},)")


def fwd_varlen(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, seqlens_q: torch.Tensor,
               seqlens_k: torch.Tensor, scale: Optional[float] = None, causal: bool = False,
               O: Optional[torch.Tensor] = None, LSE: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """Forward over a padded batch through ``fa_fwd_varlen`` (bf16) or
    ``fa_fwd_f32_varlen`` (float32): sequence b uses its first seqlens_q[b] query rows of
    Q [B, H, Nq, d] and seqlens_k[b] key rows of K, V [B, H, Nk, d].  Rows of O and LSE
    past a sequence's length are not written (outputs allocated here start as zeros and
    -inf).  Returns (O, LSE)."""
    B, H, Nq, d = Q.shape
    Nk = K.shape[2]
    dtype = _layout_dtype(Q)
    _check_bhnd("Q", Q, (B, H, Nq, d), dtype)
    for name, t in (("K", K), ("V", V)):
        _check_bhnd(name, t, (B, H, Nk, d), dtype)
    _check_seqlens(seqlens_q, seqlens_k, B, Q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.zeros_like(Q)
    if LSE is None:
        LSE = torch.full((B, H, Nq), float("-inf"), device=Q.device, dtype=torch.float32)
    _check_bhnd("O", O, (B, H, Nq, d), dtype)
    _check_bhnd("LSE", LSE, (B, H, Nq), torch.float32)
    name = "fa_fwd_varlen" if dtype == torch.bfloat16 else "fa_fwd_f32_varlen"
    with torch.cuda.device(Q.device):
        st = getattr(lib(), name)(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE),
                                  _ptr(seqlens_q), _ptr(seqlens_k), B, H, Nq, Nk, d,
                                  float(scale), int(bool(causal)), _stream_handle(stream))
    _check(name, st)
    return O, LSE


def bwd_varlen(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor,
               dO: torch.Tensor, LSE: torch.Tensor, seqlens_q: torch.Tensor,
               seqlens_k: torch.Tensor, scale: Optional[float] = None, causal: bool = False,
               dQ: Optional[torch.Tensor] = None, dK: Optional[torch.Tensor] = None,
               dV: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """Backward over a padded batch through ``fa_bwd_varlen`` (bf16) or
    ``fa_bwd_f32_varlen`` (float32), the gradient of ``fwd_varlen`` with the same lengths.
    Rows past a sequence's lengths are not written (gradients allocated here start as
    zeros).  Returns (dQ, dK, dV)."""
    B, H, Nq, d = Q.shape
    Nk = K.shape[2]
    dtype = _layout_dtype(Q)
    for name, t in (("Q", Q), ("O", O), ("dO", dO)):
        _check_bhnd(name, t, (B, H, Nq, d), dtype)
    for name, t in (("K", K), ("V", V)):
        _check_bhnd(name, t, (B, H, Nk, d), dtype)
    _check_bhnd("LSE", LSE, (B, H, Nq), torch.float32)
    _check_seqlens(seqlens_q, seqlens_k, B, Q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dQ = torch.zeros_like(Q) if dQ is None else dQ
    dK = torch.zeros_like(K) if dK is None else dK
    dV = torch.zeros_like(V) if dV is None else dV
    _check_bhnd("dQ", dQ, (B, H, Nq, d), dtype)
    for name, t in (("dK", dK), ("dV", dV)):
        _check_bhnd(name, t, (B, H, Nk, d), dtype)
    need = workspace_bytes(B, H, Nq, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=Q.device, dtype=torch.uint8)
    ws_bytes = workspace.numel() * workspace.element_size()
    name = "fa_bwd_varlen" if dtype == torch.bfloat16 else "fa_bwd_f32_varlen"
    with torch.cuda.device(Q.device):
        st = getattr(lib(), name)(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(LSE),
                                  _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(seqlens_q),
                                  _ptr(seqlens_k), B, H, Nq, Nk, d, float(scale),
                                  int(bool(causal)), _ptr(workspace), ws_bytes,
                                  _stream_handle(stream))
    _check(name, st)
    return dQ, dK, dV


def _check_packed(name: str, t: torch.Tensor, tokens: int, H: int, d: int,
                  dtype: torch.dtype = torch.bfloat16) -> None:
    _check_bhnd(name, t, (tokens, H, d), dtype)


def _check_cu(cu_q: torch.Tensor, cu_k: torch.Tensor, device) -> int:
    for name, t in (("cu_seqlens_q", cu_q), ("cu_seqlens_k", cu_k)):
        if not t.is_cuda or t.device != device or t.dtype != torch.int32 or t.dim() != 1 \
                or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA vector on the inputs' device")
    if cu_q.numel() != cu_k.numel() or cu_q.numel() < 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both have B+1 entries")
    return cu_q.numel() - 1


def fwd_packed(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu_seqlens_q: torch.Tensor,
               cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int,
               scale: Optional[float] = None, causal: bool = False,
               O: Optional[torch.Tensor] = None, LSE: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """Forward over a packed batch through ``fa_fwd_packed`` (bf16) or
    ``fa_fwd_f32_packed`` (float32): Q [total_q, H, d], K and V [total_k, H, d], sequences
    delimited by the int32 start arrays (B+1 entries).
    Returns (O [total_q, H, d], LSE [H, total_q])."""
    total_q, H, d = Q.shape
    total_k = K.shape[0]
    dtype = _layout_dtype(Q)
    _check_packed("Q", Q, total_q, H, d, dtype)
    for name, t in (("K", K), ("V", V)):
        _check_packed(name, t, total_k, H, d, dtype)
    B = _check_cu(cu_seqlens_q, cu_seqlens_k, Q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    O = torch.zeros_like(Q) if O is None else O
    LSE = torch.full((H, total_q), float("-inf"), device=Q.device) if LSE is None else LSE
    _check_packed("O", O, total_q, H, d, dtype)
    _check_bhnd("LSE", LSE, (H, total_q), torch.float32)
    name = "fa_fwd_packed" if dtype == torch.bfloat16 else "fa_fwd_f32_packed"
    with torch.cuda.device(Q.device):
        st = getattr(lib(), name)(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE),
                                  _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, H,
                                  int(max_seqlen_q), int(max_seqlen_k), total_q, total_k, d,
                                  float(scale), int(bool(causal)), _stream_handle(stream))
    _check(name, st)
    return O, LSE


def bwd_packed(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor,
               dO: torch.Tensor, LSE: torch.Tensor, cu_seqlens_q: torch.Tensor,
               cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int,
               scale: Optional[float] = None, causal: bool = False,
               dQ: Optional[torch.Tensor] = None, dK: Optional[torch.Tensor] = None,
               dV: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """Backward over a packed batch through ``fa_bwd_packed`` (bf16) or
    ``fa_bwd_f32_packed`` (float32), the gradient of ``fwd_packed`` with the same start
    arrays.  Returns (dQ, dK, dV)."""
    total_q, H, d = Q.shape
    total_k = K.shape[0]
    dtype = _layout_dtype(Q)
    for name, t in (("Q", Q), ("O", O), ("dO", dO)):
        _check_packed(name, t, total_q, H, d, dtype)
    for name, t in (("K", K), ("V", V)):
        _check_packed(name, t, total_k, H, d, dtype)
    _check_bhnd("LSE", LSE, (H, total_q), torch.float32)
    B = _check_cu(cu_seqlens_q, cu_seqlens_k, Q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dQ = torch.zeros_like(Q) if dQ is None else dQ
    dK = torch.zeros_like(K) if dK is None else dK
    dV = torch.zeros_like(V) if dV is None else dV
    _check_packed("dQ", dQ, total_q, H, d, dtype)
    for name, t in (("dK", dK), ("dV", dV)):
        _check_packed(name, t, total_k, H, d, dtype)
    need = workspace_bytes(B, H, int(max_seqlen_q), d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=Q.device, dtype=torch.uint8)
    ws_bytes = workspace.numel() * workspace.element_size()
    name = "fa_bwd_packed" if dtype == torch.bfloat16 else "fa_bwd_f32_packed"
    with torch.cuda.device(Q.device):
        st = getattr(lib(), name)(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(LSE),
                                  _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(cu_seqlens_q),
                                  _ptr(cu_seqlens_k), B, H, int(max_seqlen_q),
                                  int(max_seqlen_k), total_q, total_k, d, float(scale),
                                  int(bool(causal)), _ptr(workspace), ws_bytes,
                                  _stream_handle(stream))
    _check(name, st)
    return dQ, dK, dV


def _check_like(name: str, t: Optional[torch.Tensor], shape: tuple, dtype, device,
                optional: bool = False) -> None:
    """t is a contiguous tensor of this shape, dtype and device (or None when optional)."""
    if t is None and optional:
        return
    if t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous():
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on the inputs' device ({device}), not {t.device}")
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got "
                     f"{t.dtype} {tuple(t.shape)}")


def _check_workspace(t: torch.Tensor, device) -> int:
    if t.device != device or not t.is_contiguous():
        raise ValueError("workspace must be contiguous and on the inputs' device")
    return t.numel() * t.element_size()


def doc_ranges(doc_ids: torch.Tensor, starts: Optional[torch.Tensor] = None,
               ends: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """The documents of a batch as ``fwd_mod`` and ``bwd_mod`` take them, through
    ``fa_doc_ranges``: doc_ids [B, N] int32 (an id per key token, negative for padding)
    -> (starts, ends), [B, N] int32 each, the run of equal ids every token lies in.  One
    call serves every layer's forward and backward calls over the batch."""
    if doc_ids.dim() != 2:
        raise ValueError("doc_ids must have two dimensions [B, N]")
    B, N = doc_ids.shape
    device = doc_ids.device
    _check_bhnd("doc_ids", doc_ids, (B, N), torch.int32)
    starts = torch.empty_like(doc_ids) if starts is None else starts
    ends = torch.empty_like(doc_ids) if ends is None else ends
    _check_like("starts", starts, (B, N), torch.int32, device)
    _check_like("ends", ends, (B, N), torch.int32, device)
    _run("fa_doc_ranges", device, stream, _ptr(doc_ids), _ptr(starts), _ptr(ends), B, N)
    return starts, ends


def _mod_shapes(Q, K, V, slopes, prefix, docs):
    if Q.dim() != 4 or K.dim() != 4:
        raise ValueError("Q must be [B, H, Nq, d] and K, V [B, Hkv, Nk, d]")
    B, H, Nq, d = Q.shape
    Hkv, Nk = K.shape[1], K.shape[2]
    device = Q.device
    _check_bhnd("Q", Q, (B, H, Nq, d), torch.bfloat16)
    _check_like("K", K, (B, Hkv, Nk, d), torch.bfloat16, device)
    _check_like("V", V, (B, Hkv, Nk, d), torch.bfloat16, device)
    _check_like("slopes", slopes, (H,), torch.float32, device, optional=True)
    _check_like("prefix", prefix, (B,), torch.int32, device, optional=True)
    starts, ends = (None, None) if docs is None else docs
    if docs is not None:
        _check_like("docs[0]", starts, (B, Nk), torch.int32, device)
        _check_like("docs[1]", ends, (B, Nk), torch.int32, device)
    mods = (_ptr(slopes), _ptr(prefix), _ptr(starts), _ptr(ends))
    return B, H, Hkv, Nq, Nk, d, device, mods


def fwd_mod(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, scale: Optional[float] = None,
            causal: bool = False, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
            prefix: Optional[torch.Tensor] = None, docs=None, O: Optional[torch.Tensor] = None,
            LSE: Optional[torch.Tensor] = None, want_lse: bool = True,
            stream: Optional[torch.cuda.Stream] = None):
    """Forward with modified scores and shared key heads through ``fa_fwd_mod`` (bf16).

    Q [B, H, Nq, d]; K, V [B, Hkv, Nk, d], H a multiple of Hkv; the queries are the last
    Nq of the Nk tokens, row i at position p = i + Nk - Nq.  ``softcap`` c > 0 turns the
    scaled score z into c tanh(z / c); ``slopes`` [H] float32 subtracts slopes[h] |p - j|;
    ``causal`` hides keys past p except the first ``prefix`` [B] int32 of each sequence;
    ``docs`` = ``doc_ranges(ids)`` hides keys of other documents.  A row that sees no key
    gets O = 0 and LSE = -inf.  Returns (O, LSE); LSE is None when ``want_lse`` is False
    and none is passed."""
    B, H, Hkv, Nq, Nk, d, device, mods = _mod_shapes(Q, K, V, slopes, prefix, docs)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    else:
        _check_like("O", O, (B, H, Nq, d), torch.bfloat16, device)
    if LSE is not None:
        _check_like("LSE", LSE, (B, H, Nq), torch.float32, device)
    elif want_lse:
        LSE = torch.empty((B, H, Nq), device=device, dtype=torch.float32)
    _run("fa_fwd_mod", device, stream, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), *mods, B,
         H, Hkv, Nq, Nk, d, float(scale), int(bool(causal)), float(softcap))
    return O, LSE


def bwd_mod(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor,
            dO: torch.Tensor, LSE: torch.Tensor, scale: Optional[float] = None,
            causal: bool = False, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
            prefix: Optional[torch.Tensor] = None, docs=None,
            dQ: Optional[torch.Tensor] = None, dK: Optional[torch.Tensor] = None,
            dV: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None):
    """Backward of ``fwd_mod`` with the same modifications through ``fa_bwd_mod``.  dK and
    dV [B, Hkv, Nk, d] are summed over the query heads that share a key head; slopes are
    constants.  Every row of every gradient is written.  Returns (dQ, dK, dV)."""
    B, H, Hkv, Nq, Nk, d, device, mods = _mod_shapes(Q, K, V, slopes, prefix, docs)
    q_shape, k_shape = (B, H, Nq, d), (B, Hkv, Nk, d)
    _check_like("O", O, q_shape, torch.bfloat16, device)
    _check_like("dO", dO, q_shape, torch.bfloat16, device)
    _check_like("LSE", LSE, (B, H, Nq), torch.float32, device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    _check_like("dQ", dQ, q_shape, torch.bfloat16, device)
    _check_like("dK", dK, k_shape, torch.bfloat16, device)
    _check_like("dV", dV, k_shape, torch.bfloat16, device)
    if workspace is None:
        workspace = torch.empty(max(workspace_bytes(B, H, Nq, d), 16), device=device,
                                dtype=torch.uint8)
    ws_bytes = _check_workspace(workspace, device)
    _run("fa_bwd_mod", device, stream, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(LSE),
         _ptr(dQ), _ptr(dK), _ptr(dV), *mods, B, H, Hkv, Nq, Nk, d, float(scale),
         int(bool(causal)), float(softcap), _ptr(workspace), ws_bytes)
    return dQ, dK, dV


def rotary_frequencies(rot: int, base: float = 10000.0, factor: float = 1.0,
                       scaling: str = "linear", original_len: int = 8192,
                       device="cuda"):
    """Inverse frequencies [rot/2] float32 and the scale for ``rotary``: base^(-2k/rot),
    stretched ``factor`` times for contexts longer than the ``original_len`` tokens a model
    was trained on.

    "linear": every frequency divided by factor.  "base": the base raised to base *
    factor^(rot / (rot - 2)), which divides the slowest frequency by factor and leaves the
    fastest.  "parts": frequencies that turn at least 32 times within original_len are
    kept, those that turn less than once are divided by factor, those between are blended
    linearly in the number of turns' place between the two limits (in log space), and the
    scale is 0.1 ln(factor) + 1.  Returns (inv_freq, mscale)."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and positive")
    if not factor > 0 or not base > 0:
        raise ValueError("base and factor must be positive")
    k = torch.arange(rot // 2, dtype=torch.float64)
    mscale = 1.0
    if scaling == "linear":
        freq = base ** (-2 * k / rot) / factor
    elif scaling == "base":
        if rot > 2:
            base = base * factor ** (rot / (rot - 2))
        freq = base ** (-2 * k / rot)
    elif scaling == "parts":
        freq = base ** (-2 * k / rot)
        turns = original_len * freq / (2 * math.pi)
        keep = (torch.log(turns) / math.log(32.0)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / factor)
        mscale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    else:
        raise ValueError("scaling must be 'linear', 'base' or 'parts'")
    return freq.float().to(device), mscale


def _rotary_side(name, x, out, dtype, device):
    """(B, heads, N, d) and the stride array of one tensor of a rotary call; None for the
    strides of contiguous [B, heads, N, d] tensors."""
    for what, t in ((name, x), (f"{name}'s output", out)):
        if t.dtype != dtype or t.device != device or not t.is_cuda:
            raise ValueError(f"{what} must be a {dtype} CUDA tensor on {device}, got {t.dtype} "
                             f"on {t.device}")
        if t.dim() not in (3, 4) or t.shape != x.shape:
            raise ValueError(f"{what} must be [B, heads, N, d] or packed [tokens, heads, d]")
    if x.dim() == 4 and x.is_contiguous() and out.is_contiguous():
        return x.shape, None
    for what, t in ((name, x), (f"{name}'s output", out)):
        if t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{what} must be contiguous in its last dimension")
    if x.dim() == 3:
        N, heads, d = x.shape
        st = [0, x.stride(1), x.stride(0), 0, out.stride(1), out.stride(0)]
        return (1, heads, N, d), (_ll * 6)(*st)
    return x.shape, (_ll * 6)(*x.stride()[:3], *out.stride()[:3])


def _rotary(Q, K, inv_freq, positions, first, interleaved, mscale, Q_out, K_out, inverse, stream):
    dtype, device = Q.dtype, Q.device
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("Q and K must be bfloat16 or float32")
    Q_out = torch.empty_like(Q) if Q_out is None else Q_out
    (B, H, N, d), qs = _rotary_side("Q", Q, Q_out, dtype, device)
    Hkv, ks = 0, None
    if K is not None:
        K_out = torch.empty_like(K) if K_out is None else K_out
        (Bk, Hkv, Nk, dk), ks = _rotary_side("K", K, K_out, dtype, device)
        if (Bk, Nk, dk) != (B, N, d) or K.dim() != Q.dim():
            raise ValueError("Q and K must agree in batch, tokens and head dimension")
    elif K_out is not None:
        raise ValueError("K_out without K")
    R = 2 * inv_freq.numel()
    _check_like("inv_freq", inv_freq, (R // 2,), torch.float32, device)
    if positions is not None:
        _check_like("positions", positions, (N,) if Q.dim() == 3 else (B, N), torch.int32, device)
    _run("fa_rotary" if dtype == torch.bfloat16 else "fa_rotary_f32", device, stream, _ptr(Q),
         _ptr(Q_out), _ptr(K), _ptr(K_out), _ptr(inv_freq), _ptr(positions), int(first), B, H,
         Hkv, N, d, R, int(bool(interleaved)), inverse, float(mscale), qs, ks)
    return Q_out, K_out


def rotary(Q: torch.Tensor, K: Optional[torch.Tensor], inv_freq: torch.Tensor,
           positions: Optional[torch.Tensor] = None, first: int = 0, interleaved: bool = False,
           mscale: float = 1.0, Q_out: Optional[torch.Tensor] = None,
           K_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Rotary positions of Q [B, H, N, d] and K [B, Hkv, N, d] (or None) in one launch
    through ``fa_rotary`` (bf16) or ``fa_rotary_f32``; packed [tokens, heads, d] tensors
    too.  The first 2 * len(inv_freq) elements of each head are turned in pairs (k, k + R/2),
    or (2k, 2k + 1) when ``interleaved``, by position * inv_freq[k]; positions [B, N] (packed:
    [tokens]) int32, or ``first`` + the token's number.  Any strides with contiguous rows;
    ``Q_out=Q, K_out=K`` works in place.  Returns (Q_out, K_out)."""
    return _rotary(Q, K, inv_freq, positions, first, interleaved, mscale, Q_out, K_out, 0, stream)


def rotary_bwd(dQ_out: torch.Tensor, dK_out: Optional[torch.Tensor], inv_freq: torch.Tensor,
               positions: Optional[torch.Tensor] = None, first: int = 0,
               interleaved: bool = False, mscale: float = 1.0,
               dQ: Optional[torch.Tensor] = None, dK: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """The gradient of ``rotary``: gradients of its outputs to gradients of its inputs (the
    same map with the angles' signs turned).  Returns (dQ, dK)."""
    return _rotary(dQ_out, dK_out, inv_freq, positions, first, interleaved, mscale, dQ, dK, 1,
                   stream)


@functools.lru_cache(maxsize=256)
def tree_workspace_bytes(B: int, H: int, Hkv: int, T: int, d: int) -> int:
    return int(lib().fa_fwd_tree_workspace_bytes(B, H, Hkv, T, d))


def fwd_tree(Q: torch.Tensor, K_cache: torch.Tensor, V_cache: torch.Tensor,
             block_table: torch.Tensor, cache_lens: torch.Tensor,
             seqlens_q: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
             scale: Optional[float] = None, softcap: float = 0.0,
             O: Optional[torch.Tensor] = None, LSE: Optional[torch.Tensor] = None,
             want_lse: bool = True, workspace: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """Attention of T drafted tokens per sequence (T = 1: single-token decoding) over a paged
    cache through ``fa_fwd_tree`` (bf16).

    Q [B, H, T, d]; K_cache, V_cache [num_pages, Hkv, page, d]; block_table [B, max_pages]
    int32; cache_lens [B] int32, drafted tokens included (they are the cache's last);
    seqlens_q [B] int32: drafted tokens of each sequence (default T); tree_mask [B, T]
    int64: bit u of row t lets drafted token t see drafted token u (default: a chain).
    Rows behind a sequence's drafted tokens are not written (outputs allocated here start
    as zeros and -inf when ``seqlens_q`` is given).  Returns (O, LSE); LSE is None when
    ``want_lse`` is False and none is passed."""
    if Q.dim() != 4 or K_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("Q must be [B, H, T, d], the caches [num_pages, Hkv, page, d] and "
                         "block_table [B, max_pages]")
    B, H, T, d = Q.shape
    num_pages, Hkv, page, _ = K_cache.shape
    max_pages = block_table.shape[1]
    device = Q.device
    cache = (num_pages, Hkv, page, d)
    _check_bhnd("Q", Q, (B, H, T, d), torch.bfloat16)
    _check_like("K_cache", K_cache, cache, torch.bfloat16, device)
    _check_like("V_cache", V_cache, cache, torch.bfloat16, device)
    _check_like("block_table", block_table, (B, max_pages), torch.int32, device)
    _check_like("cache_lens", cache_lens, (B,), torch.int32, device)
    _check_like("seqlens_q", seqlens_q, (B,), torch.int32, device, optional=True)
    _check_like("tree_mask", tree_mask, (B, T), torch.int64, device, optional=True)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q) if seqlens_q is None else torch.zeros_like(Q)
    else:
        _check_like("O", O, (B, H, T, d), torch.bfloat16, device)
    if LSE is not None:
        _check_like("LSE", LSE, (B, H, T), torch.float32, device)
    elif want_lse:
        LSE = torch.empty((B, H, T), device=device, dtype=torch.float32) if seqlens_q is None \
            else torch.full((B, H, T), float("-inf"), device=device)
    if workspace is None:
        workspace = torch.empty(max(tree_workspace_bytes(B, H, Hkv, T, d), 16), device=device,
                                dtype=torch.uint8)
    ws_bytes = _check_workspace(workspace, device)
    _run("fa_fwd_tree", device, stream, _ptr(Q), _ptr(K_cache), _ptr(V_cache), _ptr(O), _ptr(LSE),
         _ptr(block_table), _ptr(cache_lens), _ptr(seqlens_q), _ptr(tree_mask), B, H, Hkv, T,
         num_pages, page, max_pages, d, float(scale), float(softcap), _ptr(workspace), ws_bytes)
    return O, LSE


def merge(O_acc: torch.Tensor, LSE_acc: torch.Tensor, O_part: torch.Tensor,
          LSE_part: torch.Tensor, O_out: Optional[torch.Tensor] = None,
          stream: Optional[torch.cuda.Stream] = None):
    """Merge a partial result over a block of keys into a float32 accumulator in place
    through ``fa_merge``.  O_acc [B, H, N, d] float32, LSE_acc [B, H, N] float32 (-inf:
    empty), O_part [B, H, N, d] bf16, LSE_part [B, H, N] float32; O_out, if given, gets
    the merged O as bf16.  Returns (O_acc, LSE_acc)."""
    B, H, N, d = O_acc.shape
    _check_bhnd("O_acc", O_acc, (B, H, N, d), torch.float32)
    _check_bhnd("LSE_acc", LSE_acc, (B, H, N), torch.float32)
    _check_bhnd("O_part", O_part, (B, H, N, d), torch.bfloat16)
    _check_bhnd("LSE_part", LSE_part, (B, H, N), torch.float32)
    if O_out is not None:
        _check_bhnd("O_out", O_out, (B, H, N, d), torch.bfloat16)
    with torch.cuda.device(O_acc.device):
        st = lib().fa_merge(_ptr(O_acc), _ptr(LSE_acc), _ptr(O_part), _ptr(LSE_part),
                            _ptr(O_out), B, H, N, d, _stream_handle(stream))
    _check("fa_merge", st)
    return O_acc, LSE_acc


def accumulate(acc: torch.Tensor, part: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """acc += part (float32 += bf16, same shape, contiguous) through ``fa_accumulate``;
    ``out``, if given, receives acc rounded to bf16.  Returns acc."""
    if acc.dtype != torch.float32 or part.dtype != torch.bfloat16:
        raise ValueError("acc must be float32 and part bfloat16")
    if acc.shape != part.shape or (out is not None and out.shape != acc.shape):
        raise ValueError("acc, part and out must have the same shape")
    for name, t in (("acc", acc), ("part", part), ("out", out)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if out is not None and out.dtype != torch.bfloat16:
        raise ValueError("out must be bfloat16")
    with torch.cuda.device(acc.device):
        st = lib().fa_accumulate(_ptr(acc), _ptr(part), _ptr(out), acc.numel(),
                                 _stream_handle(stream))
    _check("fa_accumulate", st)
    return acc


class trace_kernels:
    """Context manager: record the given torch.cuda.Events at kernel boundaries of the
    library calls made inside it (fa_trace_events).  events[0] before the first kernel
    of each call, events[k] after its k-th kernel."""

    def __init__(self, events):
        for e in events:
            e.record()  # make sure the underlying cudaEvent_t exists
        self._arr = (_vp * len(events))(*[e.cuda_event for e in events])
        self._n = len(events)

    def __enter__(self):
        _check("fa_trace_events", lib().fa_trace_events(self._arr, self._n))
        return self

    def __exit__(self, *exc):
        lib().fa_trace_events(None, 0)


def check_device_error(stream: Optional[torch.cuda.Stream] = None) -> None:
    """Synchronise the stream and raise FAError if a kernel reported a wait timeout."""
    _check("fa_check_device_error", lib().fa_check_device_error(_stream_handle(stream)))
