"""Thin ctypes binding over libfa.so (include/fa.h). Argument marshalling only.

Every step of attention runs in the library's CUDA kernels; this module only checks
tensor metadata, allocates outputs with torch and passes raw device pointers and the
current CUDA stream. There is no fallback: if libfa.so is missing or the GPU is not an
sm_103 part, calls raise.
"""

from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")

FA_OK = 0
_lib = None

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float


class _Rotary(ctypes.Structure):  # fa_rotary
    _fields_ = [("inv_freq", _vp), ("axes", ctypes.c_char_p), ("naxes", _i), ("rot", _i), ("interleaved", _i)]


class _Batch(ctypes.Structure):  # fa_paged_batch
    _fields_ = [("block_table", _vp), ("table_stride", ctypes.c_longlong), ("plan", _vp),
                ("plan_bytes", ctypes.c_size_t)] + [(n, _i) for n in (
                    "S", "T", "max_q", "max_pages", "page_size", "Hq", "Hkv", "d", "causal", "window")]


class _Cache(ctypes.Structure):  # fa_paged_cache
    _fields_ = [("k", _vp), ("v", _vp)] + [(f"{x}_stride{i}", ctypes.c_longlong) for x in "kv" for i in range(3)] + [
        ("num_pages", _i)]


class _Cache4(ctypes.Structure):  # fa_paged_cache4
    _fields_ = [(n, _vp) for n in ("k", "v", "k_scale", "v_scale")] + [
        (f"{x}_stride{i}", ctypes.c_longlong) for x in ("k", "v", "k_scale", "v_scale") for i in range(2)] + [
        ("num_pages", _i)]


class _Rows(ctypes.Structure):  # fa_paged_rows
    _fields_ = [("base", _vp)] + [(f"stride{i}", ctypes.c_longlong) for i in range(3)] + [("bytes", _i)]


# Arguments that change with each call are packed into bytes, in a third of the time that ctypes takes for an array.
_ll2, _ll4, _ll8, _ll12 = (struct.Struct(f"{n}q").pack for n in (2, 4, 8, 12))
_pack_cache = struct.Struct("PP6qi4x").pack  # _Cache
_pack_rows = struct.Struct("P3qi4x").pack  # _Rows


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({strerror(status)})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libfa.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m online_softmax_09_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.fa_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp]
        L.fa_fwd.restype = _i
        L.fa_fwd_stats.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp]
        L.fa_fwd_stats.restype = _i
        L.fa_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
        L.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.fa_bwd.argtypes = [_vp] * 9 + [_vp, ctypes.c_size_t] + [_i, _i, _i, _i, _i, _i, _f, _vp]
        L.fa_bwd.restype = _i
        L.fa_bwd_noalloc.argtypes = [_vp] * 9 + [_i, _i, _i, _i, _i, _i, _f, _vp]
        L.fa_bwd_noalloc.restype = _i
        L.fa_bwd_window.argtypes = [_vp] * 9 + [_vp, ctypes.c_size_t] + [_i, _i, _i, _i, _i, _i, _f, _vp]
        L.fa_bwd_window.restype = _i
        L.fa_bwd_prepare.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_size_t, _i, _i, _i, _i, _i, _vp]
        L.fa_bwd_prepare.restype = _i
        L.fa_bwd_compute.argtypes = [_vp] * 7 + [ctypes.c_size_t, _i, _i, _i, _i, _i, _i, _f, _vp]
        L.fa_bwd_compute.restype = _i
        L.fa_bwd_finalize.argtypes = [_vp, _vp, ctypes.c_size_t, _i, _i, _i, _i, _i, _f, _vp]
        L.fa_bwd_finalize.restype = _i
        L.fa_fwd_window.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp]
        L.fa_fwd_window.restype = _i
        L.fa_fwd_splitkv_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i]
        L.fa_fwd_splitkv_workspace_bytes.restype = ctypes.c_size_t
        L.fa_fwd_splitkv_auto.argtypes = [_i] * 7
        L.fa_fwd_splitkv_auto.restype = _i
        L.fa_fwd_splitkv.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp,
                                     ctypes.c_size_t, _vp]
        L.fa_fwd_splitkv.restype = _i
        L.fa_naive_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
        L.fa_naive_workspace_bytes.restype = ctypes.c_size_t
        L.fa_naive_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _i, _i, _i, _i, _i, _i, _f, _vp]
        L.fa_naive_fwd.restype = _i
        L.fa_fwd_bwd_host_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
        L.fa_fwd_bwd_host_workspace_bytes.restype = ctypes.c_size_t
        L.fa_fwd_bwd_host.argtypes = [_vp] * 9 + [_i, _i, _i, _i, _i, _i, _f, _vp, ctypes.c_size_t, _vp]
        L.fa_fwd_bwd_host.restype = _i
        L.fa_selftest_wait_timeout.argtypes = [_vp, _vp]
        L.fa_selftest_wait_timeout.restype = _i
        L.fa_softmax_rows.argtypes = [_vp, _vp, _vp, ctypes.c_longlong, _i, _vp]
        L.fa_softmax_rows.restype = _i
        ll = ctypes.c_longlong
        for fn in (L.fa_rope, L.fa_rope_bwd):
            fn.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, ll, ll, _vp, _i, _i, _i, _i, _i, _vp]
            fn.restype = _i
        L.fa_paged_plan_bytes.argtypes = [_i]
        L.fa_paged_plan_bytes.restype = ctypes.c_size_t
        L.fa_paged_plan.argtypes = [_vp, _vp, _vp, _vp]
        L.fa_paged_plan.restype = _i
        L.fa_paged_append.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ll, _vp]
        L.fa_paged_append.restype = _i
        L.fa_fwd_paged_workspace_bytes.argtypes = [_vp]
        L.fa_fwd_paged_workspace_bytes.restype = ctypes.c_size_t
        L.fa_fwd_paged.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, ctypes.c_size_t, _vp]
        L.fa_fwd_paged.restype = _i
        L.fa_paged_append4.argtypes = [_vp] * 11 + [ll, _vp]
        L.fa_paged_append4.restype = _i
        L.fa_fwd_paged4_workspace_bytes.argtypes = [_vp]
        L.fa_fwd_paged4_workspace_bytes.restype = ctypes.c_size_t
        L.fa_fwd_paged4.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, ctypes.c_size_t, _vp]
        L.fa_fwd_paged4.restype = _i
        for fn in (L.fa_paged_weights, L.fa_paged_weights4):
            fn.argtypes = [_vp] * 8 + [_f, _vp]
            fn.restype = _i
        L.fa_paged_evict.argtypes = [_vp, _vp, _vp, _i, _i, _vp, _vp, _i, _i, _i, _vp, ll, _i, _vp, _vp, _vp]
        L.fa_paged_evict.restype = _i
        L.fa_check.argtypes = [_vp]
        L.fa_check.restype = _i
        L.fa_strerror.argtypes = [_i]
        L.fa_strerror.restype = ctypes.c_char_p
        L.fa_version.argtypes = []
        L.fa_version.restype = _i
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().fa_strerror(int(status)).decode()


def _stream_handle(stream, device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return int(s.cuda_stream)


def _check_qkv(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous 4-D bfloat16 CUDA tensor [B, H, N, d]")
    B, Hq, N, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
        raise ValueError("k and v must be [B, Hkv, N, d] with the same B, N, d as q")
    return B, Hq, k.shape[1], N, d


def forward(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
            stream=None, counters=None):
    """O, LSE = attention(q, k, v). q [B,Hq,N,d], k/v [B,Hkv,N,d] bf16 CUDA tensors."""
    B, Hq, Hkv, N, d = _check_qkv(q, k, v)
    o = out if out is not None else torch.empty_like(q)
    l = lse if lse is not None else torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    sc = 0.0 if scale is None else float(scale)
    h = _stream_handle(stream, q.device)
    if counters is None:
        r = lib().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                         B, Hq, Hkv, N, d, int(bool(causal)), sc, h)
    else:
        r = lib().fa_fwd_stats(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                               B, Hq, Hkv, N, d, int(bool(causal)), sc, counters.data_ptr(), h)
    if r != FA_OK:
        raise FAError(r, "fa_fwd")
    return o, l


def forward_window(q, k, v, window: int, scale: float | None = None, out=None, lse=None, stream=None):
    """Causal sliding-window attention (fa_fwd_window): query i sees keys i-window < j <= i."""
    B, Hq, Hkv, N, d = _check_qkv(q, k, v)
    o = out if out is not None else torch.empty_like(q)
    l = lse if lse is not None else torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    sc = 0.0 if scale is None else float(scale)
    r = lib().fa_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                            B, Hq, Hkv, N, d, int(window), sc, _stream_handle(stream, q.device))
    if r != FA_OK:
        raise FAError(r, "fa_fwd_window")
    return o, l


def forward_splitkv(q, k, v, causal: bool = False, num_splits: int = 0, scale: float | None = None,
                    out=None, lse=None, workspace=None, stream=None):
    """Split-KV forward (fa_fwd_splitkv); num_splits <= 0 lets the library choose."""
    B, Hq, Hkv, N, d = _check_qkv(q, k, v)
    o = out if out is not None else torch.empty_like(q)
    l = lse if lse is not None else torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    if workspace is None:
        used = int(num_splits) if num_splits > 0 else splitkv_auto(
            B, Hq, Hkv, N, d, causal, torch.cuda.get_device_properties(q.device).multi_processor_count)
        n = int(lib().fa_fwd_splitkv_workspace_bytes(B, Hq, Hkv, N, d, used))
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    sc = 0.0 if scale is None else float(scale)
    r = lib().fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                             B, Hq, Hkv, N, d, int(bool(causal)), sc, int(num_splits), workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _stream_handle(stream, q.device))
    if r != FA_OK:
        raise FAError(r, "fa_fwd_splitkv")
    return o, l


def splitkv_auto(B: int, Hq: int, Hkv: int, N: int, d: int, causal: bool, num_sms: int) -> int:
    """The split count fa_fwd_splitkv picks for num_splits <= 0 on a GPU with num_sms SMs."""
    r = lib().fa_fwd_splitkv_auto(B, Hq, Hkv, N, d, int(bool(causal)), num_sms)
    if r < 0:
        raise FAError(r, "fa_fwd_splitkv_auto")
    return r


def forward_naive(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None, workspace=None,
                  stream=None):
    """Baseline standard attention with S and P in HBM (fa_naive_fwd)."""
    B, Hq, Hkv, N, d = _check_qkv(q, k, v)
    o = out if out is not None else torch.empty_like(q)
    l = lse if lse is not None else torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(int(lib().fa_naive_workspace_bytes(B, Hq, Hkv, N, d)), dtype=torch.uint8,
                                device=q.device)
    sc = 0.0 if scale is None else float(scale)
    r = lib().fa_naive_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(), workspace.data_ptr(),
                           workspace.numel() * workspace.element_size(), B, Hq, Hkv, N, d, int(bool(causal)), sc,
                           _stream_handle(stream, q.device))
    if r != FA_OK:
        raise FAError(r, "fa_naive_fwd")
    return o, l


def workspace_bytes(B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, Hq, Hkv, N, d))


def backward(q, k, v, o, do, lse, causal: bool = False, scale: float | None = None,
             dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV of attention given the forward's o and lse and the output gradient do."""
    B, Hq, Hkv, N, d = _check_qkv(q, k, v)
    for name, t in (("o", o), ("do", do)):
        if t.shape != q.shape or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must match q")
    dq = dq if dq is not None else torch.empty_like(q)
    dk = dk if dk is not None else torch.empty_like(k)
    dv = dv if dv is not None else torch.empty_like(v)
    nbytes = workspace_bytes(B, Hq, Hkv, N, d)
    ws = workspace if workspace is not None else torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    sc = 0.0 if scale is None else float(scale)
    r = lib().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                     dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
                     B, Hq, Hkv, N, d, int(bool(causal)), sc, _stream_handle(stream, q.device))
    if r != FA_OK:
        raise FAError(r, "fa_bwd")
    return dq, dk, dv


def backward_noalloc(q, k, v, o, do, lse, causal: bool = False, scale: float | None = None,
                     dq=None, dk=None, dv=None, stream=None):
    """fa_bwd_noalloc: the backward without a caller workspace (the library's fixed scratch
    array; calls that overlap on one device race on it)."""
    B, Hq, Hkv, N, d = _check_qkv(q, k, v)
    for name, t in (("o", o), ("do", do)):
        if t.shape != q.shape or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must match q")
    dq = dq if dq is not None else torch.empty_like(q)
    dk = dk if dk is not None else torch.empty_like(k)
    dv = dv if dv is not None else torch.empty_like(v)
    sc = 0.0 if scale is None else float(scale)
    r = lib().fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                             dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, N, d, int(bool(causal)), sc,
                             _stream_handle(stream, q.device))
    if r != FA_OK:
        raise FAError(r, "fa_bwd_noalloc")
    return dq, dk, dv


def backward_window(q, k, v, o, do, lse, window: int, scale: float | None = None,
                    dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of causal sliding-window attention (fa_bwd_window)."""
    B, Hq, Hkv, N, d = _check_qkv(q, k, v)
    dq = dq if dq is not None else torch.empty_like(q)
    dk = dk if dk is not None else torch.empty_like(k)
    dv = dv if dv is not None else torch.empty_like(v)
    ws = workspace if workspace is not None else torch.empty(workspace_bytes(B, Hq, Hkv, N, d), dtype=torch.uint8,
                                                              device=q.device)
    sc = 0.0 if scale is None else float(scale)
    r = lib().fa_bwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(),
                            ws.numel() * ws.element_size(), B, Hq, Hkv, N, d, int(window), sc,
                            _stream_handle(stream, q.device))
    if r != FA_OK:
        raise FAError(r, "fa_bwd_window")
    return dq, dk, dv


def backward_stages(q, k, v, o, do, lse, dq, dk, dv, workspace, causal: bool = False,
                    scale: float | None = None, stream=None, between=None, only=None):
    """Run fa_bwd_prepare, fa_bwd_compute and fa_bwd_finalize; ``between(i)`` (optional)
    is called before stage i (0, 1, 2) and after the last (3), e.g. to record CUDA events.
    ``only`` (optional): the stage indices to run, e.g. ``(1,)`` for the compute stage alone on a
    workspace an earlier prepare filled."""
    B, Hq, Hkv, N, d = _check_qkv(q, k, v)
    sc = 0.0 if scale is None else float(scale)
    h = _stream_handle(stream, q.device)
    nb = workspace.numel() * workspace.element_size()
    L = lib()
    calls = (
        lambda: L.fa_bwd_prepare(o.data_ptr(), do.data_ptr(), lse.data_ptr(), workspace.data_ptr(), nb,
                                 B, Hq, Hkv, N, d, h),
        lambda: L.fa_bwd_compute(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(), dk.data_ptr(),
                                 dv.data_ptr(), workspace.data_ptr(), nb, B, Hq, Hkv, N, d, int(bool(causal)), sc, h),
        lambda: L.fa_bwd_finalize(dq.data_ptr(), workspace.data_ptr(), nb, B, Hq, Hkv, N, d, sc, h),
    )
    for i, call in enumerate(calls):
        if only is not None and i not in only:
            continue
        if between is not None:
            between(i)
        r = call()
        if r != FA_OK:
            raise FAError(r, ("fa_bwd_prepare", "fa_bwd_compute", "fa_bwd_finalize")[i])
    if between is not None:
        between(3)
    return dq, dk, dv


def fwd_bwd_host_workspace_bytes(B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    """Device workspace bytes for fa_fwd_bwd_host."""
    n = lib().fa_fwd_bwd_host_workspace_bytes(B, Hq, Hkv, N, d)
    if n == 0:
        raise ValueError("invalid sizes")
    return n


def fwd_bwd_host(q, k, v, do, causal: bool = False, scale: float | None = None, out=None, workspace=None,
                 device=None, stream=None):
    """Forward and backward on host (CPU, ideally pinned) bf16 tensors (fa_fwd_bwd_host).

    Returns host tensors ``(o, lse, dq, dk, dv)``; ``out`` may supply them (o, dq, dk, dv bf16
    and lse fp32, contiguous CPU tensors). ``workspace`` is a CUDA uint8 tensor of at least
    fwd_bwd_host_workspace_bytes(...) bytes (allocated when None). Asynchronous: the outputs
    are ready after the stream is synchronised (e.g. check())."""
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do)):
        if t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous 4-D bfloat16 CPU tensor [B, H, N, d]")
    B, Hq, N, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[2] != N or k.shape[3] != d or do.shape != q.shape:
        raise ValueError("k, v must be [B, Hkv, N, d] and do [B, Hq, N, d] with the same B, N, d as q")
    Hkv = k.shape[1]
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    if out is None:
        pin = q.is_pinned()
        out = (torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=pin),
               torch.empty((B, Hq, N), dtype=torch.float32, pin_memory=pin),
               torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=pin),
               torch.empty(k.shape, dtype=torch.bfloat16, pin_memory=pin),
               torch.empty(k.shape, dtype=torch.bfloat16, pin_memory=pin))
    o, lse, dq, dk, dv = out
    for t, shape, dt in ((o, q.shape, torch.bfloat16), (lse, (B, Hq, N), torch.float32), (dq, q.shape, torch.bfloat16),
                         (dk, k.shape, torch.bfloat16), (dv, k.shape, torch.bfloat16)):
        if t.is_cuda or tuple(t.shape) != tuple(shape) or t.dtype != dt or not t.is_contiguous():
            raise ValueError("out must be contiguous CPU tensors (o, lse, dq, dk, dv) of the input shapes")
    nbytes = fwd_bwd_host_workspace_bytes(B, Hq, Hkv, N, d)
    ws = workspace if workspace is not None else torch.empty(nbytes, dtype=torch.uint8, device=dev)
    sc = 0.0 if scale is None else float(scale)
    r = lib().fa_fwd_bwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(), o.data_ptr(), lse.data_ptr(),
                              dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, N, d, int(bool(causal)), sc,
                              ws.data_ptr(), ws.numel() * ws.element_size(), _stream_handle(stream, dev))
    if r != FA_OK:
        raise FAError(r, "fa_fwd_bwd_host")
    return o, lse, dq, dk, dv


def selftest_wait_timeout(device=None, stream=None) -> int:
    """Run fa_selftest_wait_timeout: one warp waits on a barrier nothing completes until the
    bounded wait gives up (2 s). Returns the kernel's result code (2: gave up and raised its
    abort flag); the device status then holds the timeout, which check() reports."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    res = torch.zeros(1, dtype=torch.int32, device=dev)
    r = lib().fa_selftest_wait_timeout(res.data_ptr(), _stream_handle(stream, dev))
    if r != FA_OK:
        raise FAError(r, "fa_selftest_wait_timeout")
    (stream if stream is not None else torch.cuda.current_stream(dev)).synchronize()
    return int(res.item())


def softmax_rows(x, out=None, lse=None, with_lse: bool = True, stream=None):
    """Row-wise online softmax of a contiguous fp32 CUDA tensor [..., n] (fa_softmax_rows)."""
    if not x.is_cuda or x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    n = x.shape[-1]
    rows = x.numel() // n
    p = out if out is not None else torch.empty_like(x)
    l = lse if lse is not None else (torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
                                     if with_lse else None)
    r = lib().fa_softmax_rows(x.data_ptr(), p.data_ptr(), l.data_ptr() if l is not None else None, rows, n,
                              _stream_handle(stream, x.device))
    if r != FA_OK:
        raise FAError(r, "fa_softmax_rows")
    return p, l


class Rotary:
    """Frequencies of a rotary position embedding (fa_rotary): ``inv_freq`` fp32 CUDA [rot / 2] in radians per
    position, rot a multiple of 16; dims from rot on pass through. ``interleaved``: pairs (2i, 2i + 1) instead of (i, i + rot / 2).
    ``axes``: the axis of each pair, for positions with several axes (e.g. time, height, width)."""

    def __init__(self, inv_freq, interleaved: bool = False, axes=None):
        if not inv_freq.is_cuda or inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 \
                or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous 1-D float32 CUDA tensor [rot / 2]")
        self.inv_freq = inv_freq
        self.index = inv_freq.get_device()
        self.rot = 2 * inv_freq.numel()
        self.interleaved = bool(interleaved)
        ids = None if axes is None else [int(a) for a in axes]
        if ids is not None and (len(ids) != inv_freq.numel() or any(not 0 <= a < 4 for a in ids)):
            raise ValueError("axes must name an axis 0..3 for each of the rot / 2 pairs")
        self.naxes = 1 if ids is None else max(ids) + 1
        self._c = _Rotary(inv_freq.data_ptr(), None if ids is None else bytes(ids) + b"\0", self.naxes, self.rot,
                          int(self.interleaved))
        self._ref = ctypes.addressof(self._c)


def _dev_index(t):
    i = t.get_device()
    if i != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on cuda:{i}, which is not the current device (use torch.cuda.device)")
    return i


def _stream_of(stream, index):
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)


def _empty(shape, dtype, device, stream):
    """A tensor that belongs to ``stream`` (the caller's, or the current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _strides_of(name, t, shape, index):
    """The strides of ``t``, a bf16 tensor of ``shape`` on GPU ``index`` whose last dim is contiguous."""
    s = t.stride()
    if t.dtype != torch.bfloat16 or t.get_device() != index or t.shape != shape or s[-1] != 1:
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor {list(shape)} with contiguous last dim, on the "
                         "device of the others")
    return s


def _rope(name, fn, q, k, positions, rotary, q_out, k_out, stream):
    shape = q.shape
    if len(shape) != 4 or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor [B, Hq, N, d]")
    B, Hq, N, d = shape
    i = q.get_device()
    if i != torch._C._cuda_getDevice():
        _dev_index(q)
    A, n, pshape = rotary.naxes, positions.numel(), positions.shape
    if positions.dtype != torch.int32 or positions.get_device() != i or rotary.index != i or pshape[-1:] != (N,) \
            or (n != A * N and n != A * B * N) or (A > 1 and pshape[0] != A) or len(pshape) > 3 \
            or not positions.is_contiguous():
        want = f"[{A}, {N}] or [{A}, {B}, {N}]" if A > 1 else f"[{N}] or [{B}, {N}]"
        raise ValueError(f"positions must be a contiguous int32 CUDA tensor {want}, and the rotary on q's device")
    st = _strides_of("q", q, shape, i)[:3]
    if k is not None:
        kshape = k.shape
        if len(kshape) != 4 or kshape[0] != B or kshape[2:] != shape[2:]:
            raise ValueError("k must be [B, Hkv, N, d] with the same B, N, d as q")
        ks = _strides_of("k", k, kshape, i)[:3]
        Hkv, kp = kshape[1], k.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    else:
        Hkv, kp, kop = 0, None, None
    if q_out is None:
        q_out = _empty(shape, torch.bfloat16, q.device, stream)
        st += (Hq * N * d, N * d, d)
    else:
        st += _strides_of("q_out", q_out, shape, i)[:3]
    if k is not None:
        if k_out is None:
            k_out = _empty(kshape, torch.bfloat16, q.device, stream)
            st += ks + (Hkv * N * d, N * d, d)
        else:
            st += ks + _strides_of("k_out", k_out, kshape, i)[:3]
        kop = k_out.data_ptr()
    else:
        st += (0,) * 6
    if N == 0 or B == 0:
        return q_out, k_out
    r = fn(q.data_ptr(), q_out.data_ptr(), kp, kop, _ll12(*st), positions.data_ptr(), n // A,
           N if B > 1 and n == A * B * N else 0, rotary._ref, B, Hq, Hkv, N, d, _stream_of(stream, i))
    if r != FA_OK:
        raise FAError(r, name)
    return q_out, k_out


def rope(q, k, positions, rotary, q_out=None, k_out=None, stream=None):
    """Rotated (q, k) (fa_rope). q [B,Hq,N,d], k [B,Hkv,N,d] or None: bf16 CUDA, any strides with contiguous
    last dim (e.g. views of a fused projection), 16-byte aligned; outputs are contiguous unless given. positions:
    int32 CUDA [N] or [B,N]; with several axes [A,N] or [A,B,N]. An output may be its input, the same tensor; it
    must not overlap anything else."""
    return _rope("fa_rope", (_lib or lib()).fa_rope, q, k, positions, rotary, q_out, k_out, stream)


def rope_backward(dq, dk, positions, rotary, q_out=None, k_out=None, stream=None):
    """Gradients of rope's q and k from those of its outputs (fa_rope_bwd); arguments as for rope."""
    return _rope("fa_rope_bwd", (_lib or lib()).fa_rope_bwd, dq, dk, positions, rotary, q_out, k_out, stream)


class PagedPlan:
    """The layout of one serving step over a paged cache (fa_paged_batch, its plan and a workspace); made by
    paged_plan and taken by paged_append and forward_paged of every layer of the step. It holds the workspace and
    counters of forward_paged, so calls that overlap on the GPU (two streams, two captured graphs replayed at once)
    need a plan each; a captured graph needs its plan for as long as it is replayed."""

    def __init__(self, S, T, max_q, max_pages, page_size, Hq, Hkv, d, causal, window, device, stream):
        L = lib()
        if S < 0:
            raise ValueError("cu_q must hold S + 1 values")
        if any(not -2 ** 31 <= n < 2 ** 31 for n in (S, T, max_q, max_pages, page_size, Hq, Hkv, d, window)):
            raise ValueError("sizes and window must fit 32 bits")  # ctypes would cut them off
        self.key = (S, T, max_q, max_pages, page_size, Hq, Hkv, d, causal, window, device)
        self.device, self.index = device, device.index
        self.q_shape, self.kv_shape, self.lse_shape, self.page_shape = (T, Hq, d), (T, Hkv, d), (T, Hq), (Hkv, page_size, d)
        self.buffer = _empty(int(L.fa_paged_plan_bytes(S)), torch.uint8, device, stream)
        self._kept = None  # the last stream on whose account the buffers and the table are kept
        self._c = _Batch(None, 0, self.buffer.data_ptr(), self.buffer.numel(), S, T, max_q, max_pages, page_size, Hq,
                         Hkv, d, causal, window)
        self._ref = ctypes.addressof(self._c)
        self.ws_bytes = max(int(L.fa_fwd_paged_workspace_bytes(self._ref)),
                            int(L.fa_fwd_paged4_workspace_bytes(self._ref)))  # for either kind of cache
        self.workspace = _empty(max(self.ws_bytes, 16), torch.uint8, device, stream)

    def _use(self, stream, index):
        """The raw stream of a call; what the plan holds outlives its use on a stream that it does not belong to
        (the table is the caller's and may belong to any)."""
        raw = _stream_of(stream, index)
        if raw != self._kept and not torch.cuda.is_current_stream_capturing():
            s = stream if stream is not None else torch.cuda.current_stream(index)
            for t in (self.buffer, self.workspace, self.table):
                t.record_stream(s)
            self._kept = raw
        return raw

    def _cache(self, k_cache, v_cache):
        shape, i = k_cache.shape, self.index
        ka, kb, kc, kd = k_cache.stride()
        va, vb, vc, vd = v_cache.stride()
        if shape[1:] != self.page_shape or v_cache.shape != shape or k_cache.dtype != torch.bfloat16 \
                or v_cache.dtype != torch.bfloat16 or kd != 1 or vd != 1 or k_cache.get_device() != i \
                or v_cache.get_device() != i:
            raise ValueError("k_cache and v_cache must be bfloat16 CUDA tensors [pages, Hkv, page_size, d] "
                             f"(here [pages, {', '.join(map(str, self.page_shape))}]) with contiguous last dim")
        return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), ka, kb, kc, va, vb, vc, shape[0])


def paged_plan(cu_q, kv_lens, block_table, num_tokens: int, max_q: int, page_size: int, Hq: int, Hkv: int, d: int,
               causal: bool = True, window: int = 0, plan=None, stream=None):
    """Lay out one step's ragged batch over a paged cache (fa_paged_plan). cu_q int32 CUDA [S+1]: the new tokens of
    sequence s are rows cu_q[s] .. cu_q[s+1]-1 of the step's num_tokens; kv_lens int32 CUDA [S]: its cached tokens,
    the new ones included; block_table int32 CUDA [S, max_pages]; max_q bounds the new tokens of a sequence.
    ``plan``: an earlier plan of the same sizes, laid out anew in place (as a captured graph needs). Lengths stay on
    the device; a sequence whose lengths are out of range is left out, and check() reports it."""
    for name, t in (("cu_q", cu_q), ("kv_lens", kv_lens)):
        if not t.is_cuda or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 1-D int32 CUDA tensor")
    S = cu_q.numel() - 1
    if not block_table.is_cuda or block_table.dtype != torch.int32 or block_table.dim() != 2 \
            or block_table.shape[0] != S or kv_lens.numel() != S or block_table.shape[1] < 1 \
            or block_table.stride(1) != 1 or not cu_q.device == kv_lens.device == block_table.device:
        raise ValueError("block_table must be an int32 CUDA tensor [S, max_pages], cu_q [S + 1] and kv_lens [S], "
                         "on one device")
    i = _dev_index(cu_q)
    key = (S, int(num_tokens), int(max_q), block_table.shape[1], int(page_size), int(Hq), int(Hkv), int(d),
           int(bool(causal)), int(window), cu_q.device)
    if plan is None:
        plan = PagedPlan(*key, stream)
    elif plan.key != key:
        raise ValueError("plan was made for other sizes")
    plan.table = block_table
    plan._kept = None
    plan._c.block_table = block_table.data_ptr()
    plan._c.table_stride = block_table.stride(0)
    r = lib().fa_paged_plan(cu_q.data_ptr(), kv_lens.data_ptr(), plan._ref, plan._use(stream, i))
    if r != FA_OK:
        raise FAError(r, "fa_paged_plan")
    return plan


def paged_append(q, k, v, k_cache, v_cache, plan, rotary=None, positions=None, q_out=None, stream=None):
    """Put a step's k and v [T,Hkv,d] into the cache, k rotated by ``rotary`` (None: as it is), and return q
    [T,Hq,d] rotated (q None: nothing) (fa_paged_append). k_cache, v_cache: bf16 CUDA [pages, Hkv, page_size, d],
    any strides with contiguous last dim. positions: int32 CUDA [T], or [A,T] for several axes; None: each token's
    position in its sequence."""
    i = plan.index
    if i != torch._C._cuda_getDevice():
        _dev_index(k)
    qp = qop = None
    if q is not None:
        if rotary is None:
            raise ValueError("q is only rotated: it needs a rotary")
        shape = plan.q_shape
        qs = _strides_of("q", q, shape, i)
        if q_out is None:
            q_out = _empty(shape, torch.bfloat16, q.device, stream)
            st = qs[:2] + (shape[1] * shape[2], shape[2])
        else:
            st = qs[:2] + _strides_of("q_out", q_out, shape, i)[:2]
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    else:
        st = (0, 0, 0, 0)
    shape = plan.kv_shape
    T = shape[0]
    st += _strides_of("k", k, shape, i)[:2] + _strides_of("v", v, shape, i)[:2]
    pp = None
    if positions is not None:
        A = rotary.naxes if rotary is not None else 0
        if positions.dtype != torch.int32 or positions.get_device() != i or not positions.is_contiguous() \
                or positions.shape not in (((T,), (1, T)) if A == 1 else ((A, T),)):
            raise ValueError("positions must be a contiguous int32 CUDA tensor [T], or [A, T] for several axes")
        pp = positions.data_ptr()
    if rotary is not None and rotary.index != i:
        raise ValueError("rotary is on another device")
    r = (_lib or lib()).fa_paged_append(qp, qop, k.data_ptr(), v.data_ptr(), _ll8(*st), plan._cache(k_cache, v_cache),
                              plan._ref, rotary._ref if rotary is not None else None, pp, T, plan._use(stream, i))
    if r != FA_OK:
        raise FAError(r, "fa_paged_append")
    return q_out


def forward_paged(q, k_cache, v_cache, plan, scale: float | None = None, out=None, lse=None, stream=None):
    """O [T,Hq,d], LSE [T,Hq]: attention of a step's new tokens over the paged cache (fa_fwd_paged). q [T,Hq,d] bf16
    CUDA, any strides with contiguous last dim, 16-byte aligned. Rows that belong to no sequence are left as they
    were. ``out`` must not overlap q (refused). Calls that overlap on the GPU need a plan each."""
    shape, i = plan.q_shape, plan.index
    st = _strides_of("q", q, shape, i)
    if i != torch._C._cuda_getDevice():
        _dev_index(q)
    if out is not None and not (_strides_of("out", out, shape, i) and out.is_contiguous()):
        raise ValueError("out must be contiguous")
    if lse is not None and (lse.dtype != torch.float32 or lse.get_device() != i or lse.shape != plan.lse_shape
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 CUDA tensor [T, Hq]")
    cache = plan._cache(k_cache, v_cache)
    raw = plan._use(stream, i)
    if out is None:
        out = _empty(shape, torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty(plan.lse_shape, torch.float32, q.device, stream)
    r = (_lib or lib()).fa_fwd_paged(q.data_ptr(), _ll2(st[0], st[1]), cache, plan._ref, out.data_ptr(),
                                     lse.data_ptr(), 0.0 if scale is None else float(scale),
                                     plan.workspace.data_ptr(), plan.ws_bytes, raw)
    if r != FA_OK:
        raise FAError(r, "fa_fwd_paged")
    return out, lse


class PagedCache4:
    """A paged cache in 4 bits (fa_paged_cache4, which has its layout): codes ``k``, ``v`` uint8 CUDA
    [pages, Hkv, page_size, d / 2] and scales ``k_scale``, ``v_scale`` bf16 CUDA [pages, Hkv, page_size, d / 32], the slots of
    a page and head dense. ``PagedCache4.empty`` allocates one."""

    def __init__(self, k, v, k_scale, v_scale):
        shape, i = tuple(k.shape), k.get_device()
        if len(shape) != 4:
            raise ValueError("codes must be [pages, Hkv, page_size, d / 2]")
        pages, Hkv, page, half = shape
        for name, t, dt, width in (("k", k, torch.uint8, half), ("v", v, torch.uint8, half),
                                   ("k_scale", k_scale, torch.bfloat16, half // 16),
                                   ("v_scale", v_scale, torch.bfloat16, half // 16)):
            if not t.is_cuda or t.get_device() != i or t.dtype != dt or tuple(t.shape) != (pages, Hkv, page, width) \
                    or t.stride(3) != 1 or t.stride(2) != width:
                raise ValueError(f"{name} must be a CUDA tensor {[pages, Hkv, page, width]} of {dt} with dense slots, on the "
                                 "device of the others")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_shape, self.num_pages, self.index = (Hkv, page, 2 * half), pages, i
        st = [n * t.element_size() for t in (k, v, k_scale, v_scale) for n in t.stride()[:2]]
        self._c = _Cache4(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *st, pages)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, num_pages: int, Hkv: int, page_size: int, d: int, device="cuda"):
        """A new cache; its contents are undefined."""
        code = [torch.empty(num_pages, Hkv, page_size, d // 2, dtype=torch.uint8, device=device) for _ in "kv"]
        scale = [torch.empty(num_pages, Hkv, page_size, d // 32, dtype=torch.bfloat16, device=device) for _ in "kv"]
        return cls(*code, *scale)

    def _for(self, plan):
        if self.page_shape != plan.page_shape or self.index != plan.index:
            raise ValueError(f"the cache holds pages {list(self.page_shape)} (Hkv, page_size, d) on cuda:{self.index}, the plan "
                             f"is for {list(plan.page_shape)} on cuda:{plan.index}")
        return self._ref


def paged_append4(q, k, v, cache, plan, rotary=None, positions=None, q_out=None, k_out=None, v_out=None, stream=None):
    """paged_append into a PagedCache4 (fa_paged_append4). ``k_out``, ``v_out`` bf16 CUDA [T,Hkv,d], if given, receive the values
    that the cache now stands for; they may be k and v."""
    i = plan.index
    if i != torch._C._cuda_getDevice():
        _dev_index(k)
    ref = cache._for(plan)
    qp = qop = None
    st = (0, 0, 0, 0)
    if q is not None:
        if rotary is None:
            raise ValueError("q is only rotated: it needs a rotary")
        shape = plan.q_shape
        st = _strides_of("q", q, shape, i)[:2]
        if q_out is None:
            q_out = _empty(shape, torch.bfloat16, q.device, stream)
            st += (shape[1] * shape[2], shape[2])
        else:
            st += _strides_of("q_out", q_out, shape, i)[:2]
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    shape = plan.kv_shape
    T = shape[0]
    st += _strides_of("k", k, shape, i)[:2] + _strides_of("v", v, shape, i)[:2]
    out = [None, None]
    for j, (name, t) in enumerate((("k_out", k_out), ("v_out", v_out))):
        if t is None:
            st += (0, 0)
        else:
            st += _strides_of(name, t, shape, i)[:2]
            out[j] = t.data_ptr()
    pp = None
    if positions is not None:
        A = rotary.naxes if rotary is not None else 0
        if positions.dtype != torch.int32 or positions.get_device() != i or not positions.is_contiguous() \
                or positions.shape not in (((T,), (1, T)) if A == 1 else ((A, T),)):
            raise ValueError("positions must be a contiguous int32 CUDA tensor [T], or [A, T] for several axes")
        pp = positions.data_ptr()
    if rotary is not None and rotary.index != i:
        raise ValueError("rotary is on another device")
    r = (_lib or lib()).fa_paged_append4(qp, qop, k.data_ptr(), v.data_ptr(), out[0], out[1], _ll12(*st), ref, plan._ref,
                                         rotary._ref if rotary is not None else None, pp, T, plan._use(stream, i))
    if r != FA_OK:
        raise FAError(r, "fa_paged_append4")
    return q_out


def forward_paged4(q, cache, plan, scale: float | None = None, out=None, lse=None, stream=None):
    """forward_paged over a PagedCache4 (fa_fwd_paged4): O [T,Hq,d], LSE [T,Hq]. Arguments and what is left unwritten as there."""
    shape, i = plan.q_shape, plan.index
    st = _strides_of("q", q, shape, i)
    if i != torch._C._cuda_getDevice():
        _dev_index(q)
    ref = cache._for(plan)
    if out is not None and not (_strides_of("out", out, shape, i) and out.is_contiguous()):
        raise ValueError("out must be contiguous")
    if lse is not None and (lse.dtype != torch.float32 or lse.get_device() != i or lse.shape != plan.lse_shape
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 CUDA tensor [T, Hq]")
    raw = plan._use(stream, i)
    if out is None:
        out = _empty(shape, torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty(plan.lse_shape, torch.float32, q.device, stream)
    r = (_lib or lib()).fa_fwd_paged4(q.data_ptr(), _ll2(st[0], st[1]), ref, plan._ref, out.data_ptr(), lse.data_ptr(),
                                      0.0 if scale is None else float(scale), plan.workspace.data_ptr(), plan.ws_bytes, raw)
    if r != FA_OK:
        raise FAError(r, "fa_fwd_paged4")
    return out, lse


def _check_weights(name, t, plan, pages):
    if t.dtype != torch.float32 or t.get_device() != plan.index or tuple(t.shape) != (pages,) + plan.page_shape[:2] \
            or t.stride(2) != 1:
        raise ValueError(f"{name} must be a float32 CUDA tensor {[pages, *plan.page_shape[:2]]} with dense slots, on the plan's "
                         "device")
    return t.stride()[:2]


def paged_weights(q, lse, keys, weights, plan, scale: float | None = None, out=None, stream=None):
    """Add the attention weight that cached tokens receive from a step's new tokens (fa_paged_weights, fa_paged_weights4).
    q and scale as given to forward_paged (or forward_paged4) and lse [T,Hq] as it returned it; keys: the bf16 k_cache or
    the PagedCache4; weights fp32 CUDA [pages, Hkv, page_size]. Returns ``out``: by default weights itself, added to in
    place; else a tensor like it, of which only the slots that some new token sees are written. The step's own tokens start from
    0, so call it once per step."""
    i = plan.index
    if i != torch._C._cuda_getDevice():
        _dev_index(q)
    qs = _strides_of("q", q, plan.q_shape, i)
    if lse.dtype != torch.float32 or lse.get_device() != i or lse.shape != plan.lse_shape or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 CUDA tensor [T, Hq]")
    if isinstance(keys, PagedCache4):
        cache, pages, fn, name = keys._for(plan), keys.num_pages, (_lib or lib()).fa_paged_weights4, "fa_paged_weights4"
    else:
        cache, pages, fn, name = plan._cache(keys, keys), keys.shape[0], (_lib or lib()).fa_paged_weights, "fa_paged_weights"
    if out is None:
        out = weights
    ws = _check_weights("weights", weights, plan, pages) + _check_weights("out", out, plan, pages)
    r = fn(q.data_ptr(), _ll2(qs[0], qs[1]), lse.data_ptr(), cache, plan._ref, weights.data_ptr(), out.data_ptr(), _ll4(*ws),
           0.0 if scale is None else float(scale), plan._use(stream, i))
    if r != FA_OK:
        raise FAError(r, name)
    return out


def _check_keep(max_keep, sinks, recent):
    max_keep, sinks, recent = int(max_keep), int(sinks), int(recent)
    if not 0 <= max_keep < 2 ** 31 - 2 ** 16:
        raise ValueError("max_keep must be at least 0 and at most 2^31 - 2^16 - 1, the most tokens of a sequence")
    if not (0 <= sinks < 2 ** 31 and 0 <= recent < 2 ** 31):
        raise ValueError("sinks and recent must be at least 0 and fit 32 bits")
    return max_keep, sinks, recent


def paged_evict(weights, caches, plan, keep, out_table, max_keep: int, sinks: int = 4, recent: int = 64, kept=None,
                kv_lens=None, stream=None):
    """Cut every sequence of the plan down to its keep heaviest tokens per kv head, copied in order into the pages of
    ``out_table`` (fa_paged_evict). weights fp32 CUDA [pages, Hkv, page_size] (moved along); caches: a PagedCache4, or the
    tensors to move, CUDA [pages, Hkv, page_size, ...] with dense slots, e.g. (k_cache, v_cache); keep int32 CUDA [S], at most
    max_keep; out_table int32 CUDA [S, out_pages] of pages that the plan's table does not name. The first ``sinks`` and the last
    ``recent`` tokens stay whatever their weight. Returns kept int32 [S,Hkv,max_keep] (the places that stay, then -1) and
    kv_lens int32 [S]. Later tokens need their true positions (paged_append's ``positions``)."""
    i, S = plan.index, plan.key[0]
    if i != torch._C._cuda_getDevice():
        _dev_index(weights)
    pages = weights.shape[0]
    ws = _check_weights("weights", weights, plan, pages)
    if isinstance(caches, PagedCache4):
        caches._for(plan)
        caches = (caches.k, caches.v, caches.k_scale, caches.v_scale)
    Hkv, page = plan.page_shape[:2]
    rows = b""
    for t in (*caches, weights):
        sh, st, e, n = t.shape, t.stride(), t.element_size(), 1
        dense = len(sh) >= 3
        for j in range(len(sh) - 1, 2, -1):
            dense = dense and (st[j] == n or sh[j] == 1)
            n *= sh[j]
        if not dense or sh[0] != pages or sh[1] != Hkv or sh[2] != page or t.get_device() != i:
            raise ValueError(f"what is moved must be CUDA tensors {[pages, Hkv, page]} [, ...] with dense slots, on the plan's "
                             "device")
        rows += _pack_rows(t.data_ptr(), st[0] * e, st[1] * e, st[2] * e, n * e)
    if keep.dtype != torch.int32 or keep.get_device() != i or keep.shape != (S,) or not keep.is_contiguous():
        raise ValueError(f"keep must be a contiguous int32 CUDA tensor {[S]} on the plan's device")
    ts = out_table.shape
    if out_table.dtype != torch.int32 or out_table.get_device() != i or len(ts) != 2 or ts[0] != S \
            or (out_table.stride(1) != 1 and ts[1] > 1):
        raise ValueError(f"out_table must be an int32 CUDA tensor [{S}, out_pages] with contiguous last dim, on the plan's "
                         "device")
    max_keep, sinks, recent = _check_keep(max_keep, sinks, recent)
    raw = plan._use(stream, i)
    shape = (S, Hkv, max_keep)
    if kept is None:
        kept = _empty(shape, torch.int32, weights.device, stream)
    elif kept.dtype != torch.int32 or kept.get_device() != i or kept.shape != shape or not kept.is_contiguous():
        raise ValueError(f"kept must be a contiguous int32 CUDA tensor {list(shape)}")
    if kv_lens is None:
        kv_lens = _empty((S,), torch.int32, weights.device, stream)
    elif kv_lens.dtype != torch.int32 or kv_lens.get_device() != i or kv_lens.shape != (S,) or not kv_lens.is_contiguous():
        raise ValueError(f"kv_lens must be a contiguous int32 CUDA tensor {[S]}")
    r = (_lib or lib()).fa_paged_evict(weights.data_ptr(), _ll2(*ws), rows, len(caches) + 1, pages, plan._ref,
                                       keep.data_ptr(), max_keep, sinks, recent, out_table.data_ptr(), out_table.stride(0),
                                       ts[1], kept.data_ptr(), kv_lens.data_ptr(), raw)
    if r != FA_OK:
        raise FAError(r, "fa_paged_evict")
    return kept, kv_lens


def check(stream=None, device=None) -> None:
    """Synchronise the stream and raise if a kernel reported a device-side failure."""
    dev = device if device is not None else torch.cuda.current_device()
    r = lib().fa_check(_stream_handle(stream, dev))
    if r != FA_OK:
        raise FAError(r, "fa_check")


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)
