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


def _run(name: str, index: int, *args) -> None:
    """Call ``name`` on the current stream of device ``index``, with that device current.
    The host's part of a small call takes longer than its kernel, so nothing is looked up
    twice: the raw handle of the current stream instead of a Stream object (0.2 us against
    7 us), and no device change where the device is current."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    handle = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st != FA_OK:
        _check(name, st)


def _on(stream: torch.cuda.Stream, t: torch.Tensor):
    """Context in which a call given ``stream`` runs: what it allocates (a workspace that is
    freed on return among it) then belongs to that stream, and what it fills is filled there."""
    if not t.is_cuda or stream.device_index != t.get_device():
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


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


def _like(t: Optional[torch.Tensor], shape: tuple, dtype, index: int) -> bool:
    """t is None, or a contiguous tensor of this shape and dtype on CUDA device ``index``."""
    return t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == index
                         and t.is_contiguous())


def _check_like(name: str, t: torch.Tensor, shape: tuple, dtype, index: int) -> None:
    if t is not None and _like(t, shape, dtype, index):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the inputs' device (cuda:{index}), not {t.device}")
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got "
                     f"{t.dtype} {tuple(t.shape)}")


def _check_all(index: int, *wanted) -> None:
    """Each of ``wanted`` is (name, tensor or None, shape, dtype)."""
    for name, t, shape, dtype in wanted:
        if not _like(t, shape, dtype, index):
            _check_like(name, t, shape, dtype, index)


def _check_workspace(t: torch.Tensor, index: int) -> int:
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError("workspace must be contiguous and on the inputs' device")
    return t.numel() * t.element_size()


def doc_ranges(doc_ids: torch.Tensor, starts: Optional[torch.Tensor] = None,
               ends: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """The documents of a batch as ``fwd_mod`` and ``bwd_mod`` take them, through
    ``fa_doc_ranges``: doc_ids [B, N] int32 (an id per key token, negative for padding)
    -> (starts, ends), [B, N] int32 each, the run of equal ids every token lies in.  One
    call serves every layer's forward and backward calls over the batch."""
    if stream is not None:
        with _on(stream, doc_ids):
            return doc_ranges(doc_ids, starts, ends)
    if doc_ids.dim() != 2:
        raise ValueError("doc_ids must have two dimensions [B, N]")
    B, N = shape = doc_ids.shape
    index = doc_ids.get_device()
    _check_bhnd("doc_ids", doc_ids, shape, torch.int32)
    _check_all(index, ("starts", starts, shape, torch.int32), ("ends", ends, shape, torch.int32))
    starts = torch.empty_like(doc_ids) if starts is None else starts
    ends = torch.empty_like(doc_ids) if ends is None else ends
    _run("fa_doc_ranges", index, doc_ids.data_ptr(), starts.data_ptr(), ends.data_ptr(),
         B, N)
    return starts, ends


def _mod_args(Q, K, V, slopes, prefix, docs, *more):
    """Check a _mod call's inputs (``more``: further tensors as (name, tensor, True for Q's
    shape or False for K's)); its sizes, device and the pointers of its modifications."""
    if Q.dim() != 4 or K.dim() != 4:
        raise ValueError("Q must be [B, H, Nq, d] and K, V [B, Hkv, Nk, d]")
    B, H, Nq, d = q_shape = Q.shape
    Hkv, Nk = K.shape[1], K.shape[2]
    k_shape = (B, Hkv, Nk, d)
    bf16, index = torch.bfloat16, Q.get_device()
    _check_bhnd("Q", Q, q_shape, bf16)
    if not (_like(K, k_shape, bf16, index) and _like(V, k_shape, bf16, index)):
        _check_like("K", K, k_shape, bf16, index)
        _check_like("V", V, k_shape, bf16, index)
    for name, t, like_q in more:
        shape = q_shape if like_q else k_shape
        if not _like(t, shape, bf16, index):
            _check_like(name, t, shape, bf16, index)
    starts, ends = (None, None) if docs is None else docs
    if docs is not None and (starts is None or ends is None):
        raise ValueError("docs must be the pair that doc_ranges returns")
    if slopes is not None or prefix is not None or docs is not None:
        _check_all(index, ("slopes", slopes, (H,), torch.float32),
                   ("prefix", prefix, (B,), torch.int32),
                   ("docs[0]", starts, (B, Nk), torch.int32),
                   ("docs[1]", ends, (B, Nk), torch.int32))
    return B, H, Hkv, Nq, Nk, d, index, (_ptr(slopes), _ptr(prefix), _ptr(starts), _ptr(ends))


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
    if stream is not None:
        with _on(stream, Q):
            return fwd_mod(Q, K, V, scale, causal, softcap, slopes, prefix, docs, O, LSE, want_lse)
    B, H, Hkv, Nq, Nk, d, index, mods = _mod_args(Q, K, V, slopes, prefix, docs, ("O", O, True))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if LSE is not None:
        _check_like("LSE", LSE, (B, H, Nq), torch.float32, index)
    elif want_lse:
        LSE = Q.new_empty((B, H, Nq), dtype=torch.float32)
    _run("fa_fwd_mod", index, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
         _ptr(LSE), *mods, B, H, Hkv, Nq, Nk, d, float(scale), int(bool(causal)), float(softcap))
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
    if stream is not None:
        with _on(stream, Q):
            return bwd_mod(Q, K, V, O, dO, LSE, scale, causal, softcap, slopes, prefix, docs, dQ,
                           dK, dV, workspace)
    B, H, Hkv, Nq, Nk, d, index, mods = _mod_args(
        Q, K, V, slopes, prefix, docs, ("O", O, True), ("dO", dO, True), ("dQ", dQ, True),
        ("dK", dK, False), ("dV", dV, False))
    _check_like("LSE", LSE, (B, H, Nq), torch.float32, index)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    if workspace is None:
        workspace = Q.new_empty(max(workspace_bytes(B, H, Nq, d), 16), dtype=torch.uint8)
    ws_bytes = _check_workspace(workspace, index)
    _run("fa_bwd_mod", index, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
         dO.data_ptr(), LSE.data_ptr(), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), *mods, B, H,
         Hkv, Nq, Nk, d, float(scale), int(bool(causal)), float(softcap), workspace.data_ptr(),
         ws_bytes)
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
    if not (0 < factor < math.inf and 0 < base < math.inf and 0 < original_len < math.inf):
        raise ValueError("base, factor and original_len must be positive and finite")
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


def _rotary_strides(name, x, out, dtype, index):
    """The stride array of one tensor of a rotary call; None for contiguous [B, heads, N, d]
    tensors."""
    for what, t in ((name, x), (f"{name}'s output", out)):
        if t.dtype is not dtype or t.get_device() != index:
            raise ValueError(f"{what} must be a {dtype} CUDA tensor on the inputs' device, got "
                             f"{t.dtype} on {t.device}")
        if t.dim() not in (3, 4) or t.shape != x.shape:
            raise ValueError(f"{what} must be [B, heads, N, d] or packed [tokens, heads, d]")
        if t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{what} must be contiguous in its last dimension")
    i, o = x.stride(), out.stride()
    if x.dim() == 3:
        return (_ll * 6)(0, i[1], i[0], 0, o[1], o[0])
    return (_ll * 6)(*i[:3], *o[:3])


def _dense_like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of t's shape, whatever t's strides: what the attention calls take.
    (Naming the memory format costs 0.1 us, which the usual small call need not pay.)"""
    if t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _rotary(Q, K, inv_freq, positions, first, interleaved, mscale, Q_out, K_out, inverse, stream):
    if stream is not None:
        with _on(stream, Q):
            return _rotary(Q, K, inv_freq, positions, first, interleaved, mscale, Q_out, K_out,
                           inverse, None)
    dtype, index = Q.dtype, Q.get_device()
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("Q and K must be bfloat16 or float32")
    if not Q.is_cuda:
        raise ValueError("Q must be a CUDA tensor")
    packed = Q.dim() == 3
    if not packed and Q.dim() != 4:
        raise ValueError("Q must be [B, heads, N, d] or packed [tokens, heads, d]")
    Q_out = _dense_like(Q) if Q_out is None else Q_out
    q_shape = Q.shape
    qs = ks = None
    if packed or not (Q.is_contiguous() and _like(Q_out, q_shape, dtype, index)):
        qs = _rotary_strides("Q", Q, Q_out, dtype, index)
    if packed:
        (N, H, d), B = q_shape, 1
    else:
        B, H, N, d = q_shape
    Hkv = 0
    if K is not None:
        k_shape = K.shape
        Hkv = k_shape[1] if len(k_shape) > 1 else 0
        if k_shape != ((N, Hkv, d) if packed else (B, Hkv, N, d)):
            raise ValueError("Q and K must agree in batch, tokens and head dimension")
        K_out = _dense_like(K) if K_out is None else K_out
        if packed or not (_like(K, k_shape, dtype, index) and _like(K_out, k_shape, dtype, index)):
            ks = _rotary_strides("K", K, K_out, dtype, index)
    elif K_out is not None:
        raise ValueError("K_out without K")
    half = inv_freq.numel()
    if not _like(inv_freq, (half,), torch.float32, index):
        _check_like("inv_freq", inv_freq, (half,), torch.float32, index)
    if positions is not None:
        shape = (N,) if packed else (B, N)
        if not _like(positions, shape, torch.int32, index):
            _check_like("positions", positions, shape, torch.int32, index)
    _run("fa_rotary" if dtype is torch.bfloat16 else "fa_rotary_f32", index, Q.data_ptr(),
         Q_out.data_ptr(), _ptr(K), _ptr(K_out), inv_freq.data_ptr(), _ptr(positions), int(first), B, H,
         Hkv, N, d, 2 * half, int(bool(interleaved)), inverse, float(mscale), qs, ks)
    return Q_out, K_out


def rotary(Q: torch.Tensor, K: Optional[torch.Tensor], inv_freq: torch.Tensor,
           positions: Optional[torch.Tensor] = None, first: int = 0, interleaved: bool = False,
           mscale: float = 1.0, Q_out: Optional[torch.Tensor] = None,
           K_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Rotary positions of Q [B, H, N, d] and K [B, Hkv, N, d] (or None) in one launch
    through ``fa_rotary`` (bf16) or ``fa_rotary_f32``; packed [tokens, heads, d] tensors
    too.  The first 2 * len(inv_freq) elements of each head are turned in pairs (k, k + R/2),
    or (2k, 2k + 1) when ``interleaved``, by position * inv_freq[k]; positions [B, N] (packed:
    [tokens]) int32, or ``first`` + the token's number.  Any strides with contiguous rows
    (a slice of a fused projection as it is); ``Q_out=Q, K_out=K`` works in place, and outputs
    that are not given are contiguous, as the attention calls take them.  Returns (Q_out,
    K_out)."""
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
    if stream is not None:
        with _on(stream, Q):
            return fwd_tree(Q, K_cache, V_cache, block_table, cache_lens, seqlens_q, tree_mask,
                            scale, softcap, O, LSE, want_lse, workspace)
    if Q.dim() != 4 or K_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("Q must be [B, H, T, d], the caches [num_pages, Hkv, page, d] and "
                         "block_table [B, max_pages]")
    B, H, T, d = Q.shape
    num_pages, Hkv, page, _ = K_cache.shape
    max_pages = block_table.shape[1]
    index, bf16, i32 = Q.get_device(), torch.bfloat16, torch.int32
    cache = (num_pages, Hkv, page, d)
    _check_bhnd("Q", Q, (B, H, T, d), bf16)
    if not (_like(K_cache, cache, bf16, index) and _like(V_cache, cache, bf16, index)
            and _like(block_table, (B, max_pages), i32, index)
            and _like(cache_lens, (B,), i32, index)):
        _check_like("K_cache", K_cache, cache, bf16, index)
        _check_like("V_cache", V_cache, cache, bf16, index)
        _check_like("block_table", block_table, (B, max_pages), i32, index)
        _check_like("cache_lens", cache_lens, (B,), i32, index)
    if seqlens_q is not None:
        _check_like("seqlens_q", seqlens_q, (B,), i32, index)
    if tree_mask is not None:
        _check_like("tree_mask", tree_mask, (B, T), torch.int64, index)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is not None:
        _check_like("O", O, (B, H, T, d), bf16, index)
    else:
        O = torch.empty_like(Q) if seqlens_q is None else torch.zeros_like(Q)
    if LSE is not None:
        _check_like("LSE", LSE, (B, H, T), torch.float32, index)
    elif want_lse:
        LSE = Q.new_empty((B, H, T), dtype=torch.float32)
        if seqlens_q is not None:
            LSE.fill_(-math.inf)
    if workspace is None:
        workspace = Q.new_empty(max(tree_workspace_bytes(B, H, Hkv, T, d), 16), dtype=torch.uint8)
    ws_bytes = _check_workspace(workspace, index)
    _run("fa_fwd_tree", index, Q.data_ptr(), K_cache.data_ptr(), V_cache.data_ptr(),
         O.data_ptr(), _ptr(LSE), block_table.data_ptr(), cache_lens.data_ptr(), _ptr(seqlens_q),
         _ptr(tree_mask), B, H, Hkv, T, num_pages, page, max_pages, d, float(scale),
         float(softcap), workspace.data_ptr(), ws_bytes)
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
