"""ctypes binding of ``libkda.so`` over torch tensors (marshalling only).

Every step of the computation runs in the CUDA kernels behind the C ABI in
``include/kda.h``; this module only checks tensor placement, dtype and shape,
allocates outputs that the caller did not provide, and passes raw device
pointers plus the current CUDA stream.  If the compiled library is missing,
loading fails with an error -- there is no fallback implementation.

With ``stream=`` a call runs on that stream.  The caller orders it behind what
writes its inputs and in front of what reads its outputs, as with any work on
several streams; memory that the call allocates itself, and memory that is let
go of while the call is still to run, is taken care of here.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkda.so")

KDA_OK = 0
KDA_ERR_INVALID_ARG = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_CUDA = 3
KDA_ERR_TIMEOUT = 4
KDA_ERR_TOO_LARGE = 5
KDA_BF16 = 0
KDA_FP32 = 1

_DTYPE_CODE = {torch.bfloat16: KDA_BF16, torch.float32: KDA_FP32}
_lock = threading.Lock()
_lib = None


class KdaError(RuntimeError):
    """A KDA entry point returned a non-OK status."""

    def __init__(self, fn: str, status: int):
        self.status = int(status)
        super().__init__("%s failed: %s" % (fn, status_string(status)))


def load() -> ctypes.CDLL:
    """Load ``libkda.so`` (built by ``serving_kda_chunked_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libkda.so is not built (%s); build it with "
                "`python -m serving_kda_chunked_gb300.build`" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        u64 = ctypes.c_uint64
        lib.kda_prefill_chunked.argtypes = [
            vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, i32,
            vp, vp, vp, u64, vp]
        lib.kda_prefill_chunked.restype = ctypes.c_int
        lib.kda_gdn_prefill_chunked.argtypes = lib.kda_prefill_chunked.argtypes
        lib.kda_gdn_prefill_chunked.restype = ctypes.c_int
        lib.kda_prefill_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32, i32]
        lib.kda_prefill_workspace_size.restype = u64
        lib.kda_prefill_chunked_noalloc.argtypes = [
            vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, i32, vp, vp, vp]
        lib.kda_prefill_chunked_noalloc.restype = ctypes.c_int
        lib.kda_prefill_chunked_host.argtypes = lib.kda_prefill_chunked.argtypes
        lib.kda_prefill_chunked_host.restype = ctypes.c_int
        lib.kda_prefill_host_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32, i32]
        lib.kda_prefill_host_workspace_size.restype = u64
        lib.kda_noalloc_scratch_bytes.argtypes = []
        lib.kda_noalloc_scratch_bytes.restype = u64
        lib.kda_prefill_check.argtypes = [vp, vp]
        lib.kda_prefill_check.restype = ctypes.c_int
        lib.kda_prefill_noalloc_check.argtypes = [vp]
        lib.kda_prefill_noalloc_check.restype = ctypes.c_int
        lib.kda_decode_step.argtypes = [
            vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
        lib.kda_decode_step.restype = ctypes.c_int
        lib.kda_gdn_decode_step.argtypes = lib.kda_decode_step.argtypes
        lib.kda_gdn_decode_step.restype = ctypes.c_int
        lib.kda_decode_step_pooled.argtypes = [
            vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]
        lib.kda_decode_step_pooled.restype = ctypes.c_int
        lib.kda_gdn_decode_step_pooled.argtypes = lib.kda_decode_step_pooled.argtypes
        lib.kda_gdn_decode_step_pooled.restype = ctypes.c_int
        f32 = ctypes.c_float
        lib.kda_mla_append.argtypes = [
            vp, i64, vp, i64, vp, vp, vp, i32, i32, i64, vp, i32, i32, i32, i32, i32, vp, i64,
            vp, i64, i64, i32, vp, i64, i64, vp]
        lib.kda_mla_append.restype = ctypes.c_int
        lib.kda_mla_prefill.argtypes = [
            vp, vp, vp, vp, vp, i32, i64, i64, i32, i32, i32, i32, i32, f32, i32, vp, vp, vp,
            u64, vp]
        lib.kda_mla_prefill.restype = ctypes.c_int
        lib.kda_mla_prefill_workspace_size.argtypes = [i32, i64, i32, i32]
        lib.kda_mla_prefill_workspace_size.restype = u64
        lib.kda_mla_decode.argtypes = [
            vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, f32, vp, vp, vp, u64, vp]
        lib.kda_mla_decode.restype = ctypes.c_int
        lib.kda_mla_decode_workspace_size.argtypes = [i32, i32, i32]
        lib.kda_mla_decode_workspace_size.restype = u64
        lib.kda_mla_tree_decode.argtypes = [
            vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, i32, f32, vp, vp, vp, u64, vp]
        lib.kda_mla_tree_decode.restype = ctypes.c_int
        lib.kda_mla_tree_decode_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.kda_mla_tree_decode_workspace_size.restype = u64
        for fn in (lib.kda_tree_step, lib.kda_gdn_tree_step):
            fn.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, vp, vp]
            fn.restype = ctypes.c_int
        for fn in (lib.kda_tree_commit, lib.kda_gdn_tree_commit):
            fn.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, vp]
            fn.restype = ctypes.c_int
        lib.kda_tree_verify.argtypes = [
            vp, i64, vp, i64, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp]
        lib.kda_tree_verify.restype = ctypes.c_int
        lib.kda_mla_check.argtypes = [vp, vp]
        lib.kda_mla_check.restype = ctypes.c_int
        lib.kda_status_string.argtypes = [i32]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_abi_version.argtypes = []
        lib.kda_abi_version.restype = i32
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().kda_status_string(int(status)).decode()


def abi_version() -> int:
    return int(load().kda_abi_version())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device=None):
    """Raw handle of ``stream`` (default: the current stream of ``device``, or
    of the current device); a given stream must live on ``device``."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif device is not None and stream.device != torch.device(device):
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
    return ctypes.c_void_p(int(stream.cuda_stream))


def _other_stream(stream, device):
    """``stream`` where the call runs beside the current stream of ``device``,
    else None."""
    if stream is None:
        return None
    if stream.device != device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
    if int(stream.cuda_stream) == torch._C._cuda_getCurrentRawStream(device.index):
        return None
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream), device=device)
    return stream


def _empty(shape, dtype, device, side, returned=True):
    """New memory of a call that runs on ``side`` (None: on the current stream).

    It comes from that stream's memory: a block of the current stream may still
    be in use there, and would be handed out there again once the call lets go
    of it, in both cases beside the call's kernels.  What is returned to the
    caller is recorded with the current stream as well."""
    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(side):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _record(side, *tensors):
    """The caller's tensors are in use on ``side`` too: the allocator does not
    hand their memory out again before the call has run."""
    if side is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(side)


def _same_device(device, **tensors):
    """Every given tensor (None skipped) must be on ``device``: the library
    runs on one device per call and rejects memory of any other."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError("%s is on %s, but q is on %s: all tensors of a call must be on "
                             "one device" % (name, t.device, device))


def _check_cuda(name, t, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the KDA kernels run on the GPU only)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def kda_prefill_workspace_size(N, T, H, dk, dv, dtype, chunk=64) -> int:
    """Workspace bytes ``kda_prefill_chunked`` needs (0: none)."""
    code = _DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load().kda_prefill_workspace_size(N, T, H, dk, dv, code, chunk))


def kda_prefill_check(workspace, stream=None) -> int:
    """Synchronise the stream and return the device status of the last
    prefill that used ``workspace`` (KDA_OK or KDA_ERR_TIMEOUT)."""
    dev = None if workspace is None else workspace.device
    with torch.cuda.device(dev):
        return int(load().kda_prefill_check(_ptr(workspace), _stream(stream, dev)))


def kda_prefill_noalloc_check(stream=None, device=None) -> int:
    """Synchronise the stream and return the device status of the last
    no-allocation prefill on ``device`` (default: the current device)."""
    with torch.cuda.device(device):
        return int(load().kda_prefill_noalloc_check(_stream(stream, device)))


def _prefill(fn, gate_shape, q, k, v, g, beta, cu_seqlens, S0, chunk, o, S_T, workspace,
             stream):
    _check_cuda("q", q)
    if q.dtype not in _DTYPE_CODE:
        raise ValueError("q must be bfloat16 or float32")
    T, H, dk = q.shape
    dv = v.shape[-1]
    _check_cuda("k", k, q.dtype, (T, H, dk))
    _check_cuda("v", v, q.dtype, (T, H, dv))
    _check_cuda("g", g, torch.float32, gate_shape(T, H, dk))
    _check_cuda("beta", beta, torch.float32, (T, H))
    _check_cuda("cu_seqlens", cu_seqlens, torch.int32)
    N = cu_seqlens.shape[0] - 1
    if S0 is not None:
        _check_cuda("S0", S0, torch.float32, (N, H, dk, dv))
    side = _other_stream(stream, q.device)
    brought = (q, k, v, g, beta, cu_seqlens, S0, o, S_T, workspace)
    if o is None:
        o = _empty((T, H, dv), q.dtype, q.device, side)
    _check_cuda("o", o, q.dtype, (T, H, dv))
    if S_T is None:
        S_T = _empty((N, H, dk, dv), torch.float32, q.device, side)
    _check_cuda("S_T", S_T, torch.float32, (N, H, dk, dv))
    need = kda_prefill_workspace_size(N, T, H, dk, dv, q.dtype, chunk)
    if workspace is None and need > 0:
        workspace = _empty((need,), torch.uint8, q.device, side, returned=False)
    ws_bytes = 0
    if workspace is not None:
        _check_cuda("workspace", workspace, torch.uint8)
        ws_bytes = workspace.numel()
    _same_device(q.device, k=k, v=v, g=g, beta=beta, cu_seqlens=cu_seqlens, S0=S0, o=o,
                 S_T=S_T, workspace=workspace)
    _record(side, *brought)
    with torch.cuda.device(q.device):
        st = getattr(load(), fn)(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
            N, T, H, dk, dv, _DTYPE_CODE[q.dtype], int(chunk), _ptr(o), _ptr(S_T),
            _ptr(workspace), ws_bytes, _stream(stream, q.device))
    if st != KDA_OK:
        raise KdaError(fn, st)
    return o, S_T


def _check_host(name, t, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cpu":
        raise ValueError("%s must be a host (CPU) tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def kda_prefill_host_workspace_size(N, T, H, dk, dv, dtype, chunk=64) -> int:
    """Device workspace bytes ``kda_prefill_chunked_host`` needs."""
    code = _DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load().kda_prefill_host_workspace_size(N, T, H, dk, dv, code, chunk))


def kda_prefill_chunked_host(q, k, v, g, beta, cu_seqlens, S0=None, *, chunk: int = 64,
                             o=None, S_T=None, workspace=None, device=None, stream=None):
    """``kda_prefill_chunked`` over HOST tensors (``kda_prefill_chunked_host``
    in kda.h): q, k, v, g, beta, cu_seqlens, S0 and the outputs o, S_T are CPU
    tensors (page-locked ones let the copies overlap the kernels); the call
    copies them to and from the GPU itself.  ``workspace`` is a CUDA uint8
    tensor (allocated on ``device``, default the current one, if omitted).
    Returns (o, S_T); they are complete once ``stream`` has reached this call's
    end (synchronise before reading them)."""
    _check_host("q", q)
    if q.dtype not in _DTYPE_CODE:
        raise ValueError("q must be bfloat16 or float32")
    T, H, dk = q.shape
    dv = v.shape[-1]
    _check_host("k", k, q.dtype, (T, H, dk))
    _check_host("v", v, q.dtype, (T, H, dv))
    _check_host("g", g, torch.float32, (T, H, dk))
    _check_host("beta", beta, torch.float32, (T, H))
    _check_host("cu_seqlens", cu_seqlens, torch.int32)
    N = cu_seqlens.shape[0] - 1
    if S0 is not None:
        _check_host("S0", S0, torch.float32, (N, H, dk, dv))
    pin = q.is_pinned()
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, pin_memory=pin)
    _check_host("o", o, q.dtype, (T, H, dv))
    if S_T is None:
        S_T = torch.empty((N, H, dk, dv), dtype=torch.float32, pin_memory=pin)
    _check_host("S_T", S_T, torch.float32, (N, H, dk, dv))
    if workspace is None:
        need = kda_prefill_host_workspace_size(N, T, H, dk, dv, q.dtype, chunk)
        dev = torch.device("cuda" if device is None else device)
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        workspace = _empty((max(need, 1),), torch.uint8, dev, _other_stream(stream, dev), returned=False)
    else:
        _check_cuda("workspace", workspace, torch.uint8)
        _record(_other_stream(stream, workspace.device), workspace)
    with torch.cuda.device(workspace.device):
        st = load().kda_prefill_chunked_host(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
            N, T, H, dk, dv, _DTYPE_CODE[q.dtype], int(chunk), _ptr(o), _ptr(S_T),
            _ptr(workspace), workspace.numel(), _stream(stream, workspace.device))
    if st != KDA_OK:
        raise KdaError("kda_prefill_chunked_host", st)
    return o, S_T


def kda_noalloc_scratch_bytes() -> int:
    """Size of the fixed device scratch behind ``kda_prefill_chunked_noalloc``."""
    return int(load().kda_noalloc_scratch_bytes())


def kda_prefill_chunked_noalloc(q, k, v, g, beta, cu_seqlens, S0=None, *, chunk: int = 64,
                                o=None, S_T=None, stream=None):
    """``kda_prefill_chunked`` without a workspace (``kda_prefill_chunked_noalloc``
    in kda.h): scratch lives in a fixed device array inside the library; calls
    that overlap on the GPU must not share it.  Outputs as ``kda_prefill_chunked``
    (pass ``o`` / ``S_T`` to keep the call free of allocation)."""
    _check_cuda("q", q)
    if q.dtype not in _DTYPE_CODE:
        raise ValueError("q must be bfloat16 or float32")
    T, H, dk = q.shape
    dv = v.shape[-1]
    _check_cuda("k", k, q.dtype, (T, H, dk))
    _check_cuda("v", v, q.dtype, (T, H, dv))
    _check_cuda("g", g, torch.float32, (T, H, dk))
    _check_cuda("beta", beta, torch.float32, (T, H))
    _check_cuda("cu_seqlens", cu_seqlens, torch.int32)
    N = cu_seqlens.shape[0] - 1
    if S0 is not None:
        _check_cuda("S0", S0, torch.float32, (N, H, dk, dv))
    side = _other_stream(stream, q.device)
    brought = (q, k, v, g, beta, cu_seqlens, S0, o, S_T)
    if o is None:
        o = _empty((T, H, dv), q.dtype, q.device, side)
    _check_cuda("o", o, q.dtype, (T, H, dv))
    if S_T is None:
        S_T = _empty((N, H, dk, dv), torch.float32, q.device, side)
    _check_cuda("S_T", S_T, torch.float32, (N, H, dk, dv))
    _same_device(q.device, k=k, v=v, g=g, beta=beta, cu_seqlens=cu_seqlens, S0=S0, o=o,
                 S_T=S_T)
    _record(side, *brought)
    with torch.cuda.device(q.device):
        st = load().kda_prefill_chunked_noalloc(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
            N, T, H, dk, dv, _DTYPE_CODE[q.dtype], int(chunk), _ptr(o), _ptr(S_T),
            _stream(stream, q.device))
    if st != KDA_OK:
        raise KdaError("kda_prefill_chunked_noalloc", st)
    return o, S_T


def kda_prefill_chunked(q, k, v, g, beta, cu_seqlens, S0=None, *, chunk: int = 64,
                        o=None, S_T=None, workspace=None, stream=None):
    """Chunked KDA prefill over a packed batch (``kda_prefill_chunked`` in kda.h).

    q, k [T, H, dk] and v [T, H, dv] in bf16 or fp32 (all the same); g
    [T, H, dk] fp32 log-gates; beta [T, H] fp32; cu_seqlens [N+1] int32 on the
    device; S0 [N, H, dk, dv] fp32 or None.  Returns (o, S_T); pass ``o`` /
    ``S_T`` to write into existing buffers (``S_T`` may be ``S0``).
    ``workspace``: a uint8 CUDA tensor of at least
    ``kda_prefill_workspace_size(...)`` bytes; allocated here when omitted.
    """
    return _prefill("kda_prefill_chunked", lambda T, H, dk: (T, H, dk), q, k, v, g, beta,
                    cu_seqlens, S0, chunk, o, S_T, workspace, stream)


def kda_gdn_prefill_chunked(q, k, v, g, beta, cu_seqlens, S0=None, *, chunk: int = 64,
                            o=None, S_T=None, workspace=None, stream=None):
    """Chunked Gated DeltaNet prefill (``kda_gdn_prefill_chunked`` in kda.h):
    as ``kda_prefill_chunked`` with one log-gate per head, g [T, H] fp32."""
    return _prefill("kda_gdn_prefill_chunked", lambda T, H, dk: (T, H), q, k, v, g, beta,
                    cu_seqlens, S0, chunk, o, S_T, workspace, stream)


def _decode(fn, gate_shape, q, k, v, g, beta, S, o, stream):
    _check_cuda("q", q)
    if q.dtype not in _DTYPE_CODE:
        raise ValueError("q must be bfloat16 or float32")
    B, H, dk = q.shape
    dv = v.shape[-1]
    _check_cuda("k", k, q.dtype, (B, H, dk))
    _check_cuda("v", v, q.dtype, (B, H, dv))
    _check_cuda("g", g, torch.float32, gate_shape(B, H, dk))
    _check_cuda("beta", beta, torch.float32, (B, H))
    _check_cuda("S", S, torch.float32, (B, H, dk, dv))
    side = _other_stream(stream, q.device)
    brought = (q, k, v, g, beta, S, o)
    if o is None:
        o = _empty((B, H, dv), q.dtype, q.device, side)
    _check_cuda("o", o, q.dtype, (B, H, dv))
    _same_device(q.device, k=k, v=v, g=g, beta=beta, S=S, o=o)
    _record(side, *brought)
    with torch.cuda.device(q.device):
        st = getattr(load(), fn)(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), B, H, dk, dv,
            _DTYPE_CODE[q.dtype], _ptr(o), _stream(stream, q.device))
    if st != KDA_OK:
        raise KdaError(fn, st)
    return o


def kda_decode_step(q, k, v, g, beta, S, *, o=None, stream=None):
    """One batched KDA decode step (``kda_decode_step`` in kda.h).

    q, k [B, H, dk], v [B, H, dv] (bf16 or fp32); g [B, H, dk] fp32; beta
    [B, H] fp32; S [B, H, dk, dv] fp32, updated in place.  Returns o.
    """
    return _decode("kda_decode_step", lambda B, H, dk: (B, H, dk), q, k, v, g, beta, S, o,
                   stream)


def kda_gdn_decode_step(q, k, v, g, beta, S, *, o=None, stream=None):
    """One batched Gated DeltaNet decode step (``kda_gdn_decode_step`` in
    kda.h): as ``kda_decode_step`` with one log-gate per head, g [B, H] fp32."""
    return _decode("kda_gdn_decode_step", lambda B, H, dk: (B, H), q, k, v, g, beta, S, o,
                   stream)


def _decode_pooled(fn, gate_shape, q, k, v, g, beta, S_pool, slots, o, stream):
    _check_cuda("q", q)
    if q.dtype not in _DTYPE_CODE:
        raise ValueError("q must be bfloat16 or float32")
    B, H, dk = q.shape
    dv = v.shape[-1]
    _check_cuda("k", k, q.dtype, (B, H, dk))
    _check_cuda("v", v, q.dtype, (B, H, dv))
    _check_cuda("g", g, torch.float32, gate_shape(B, H, dk))
    _check_cuda("beta", beta, torch.float32, (B, H))
    _check_cuda("S_pool", S_pool, torch.float32)
    if S_pool.dim() != 4 or tuple(S_pool.shape[1:]) != (H, dk, dv):
        raise ValueError("S_pool must have shape [P, %d, %d, %d]" % (H, dk, dv))
    _check_cuda("slots", slots, torch.int32, (B,))
    side = _other_stream(stream, q.device)
    brought = (q, k, v, g, beta, S_pool, slots, o)
    if o is None:
        o = _empty((B, H, dv), q.dtype, q.device, side)
    _check_cuda("o", o, q.dtype, (B, H, dv))
    _same_device(q.device, k=k, v=v, g=g, beta=beta, S_pool=S_pool, slots=slots, o=o)
    _record(side, *brought)
    with torch.cuda.device(q.device):
        st = getattr(load(), fn)(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S_pool), _ptr(slots),
            S_pool.shape[0], B, H, dk, dv, _DTYPE_CODE[q.dtype], _ptr(o),
            _stream(stream, q.device))
    if st != KDA_OK:
        raise KdaError(fn, st)
    return o


def kda_decode_step_pooled(q, k, v, g, beta, S_pool, slots, *, o=None, stream=None):
    """Batched decode over a pool of states (``kda_decode_step_pooled`` in kda.h).

    S_pool [P, H, dk, dv] fp32; slots [B] int32 on the device (a value outside
    [0, P) skips that sequence).  The named slots are updated in place.
    Returns o [B, H, dv].
    """
    return _decode_pooled("kda_decode_step_pooled", lambda B, H, dk: (B, H, dk), q, k, v, g,
                          beta, S_pool, slots, o, stream)


def kda_gdn_decode_step_pooled(q, k, v, g, beta, S_pool, slots, *, o=None, stream=None):
    """Gated DeltaNet decode over a pool of states (``kda_gdn_decode_step_pooled``
    in kda.h): as ``kda_decode_step_pooled`` with g [B, H] fp32."""
    return _decode_pooled("kda_gdn_decode_step_pooled", lambda B, H, dk: (B, H), q, k, v, g,
                          beta, S_pool, slots, o, stream)


MLA_LATENT, MLA_ROPE, MLA_NOPE, MLA_DV = 512, 64, 128, 128
_MLA_ROW, _MLA_QK = MLA_LATENT + MLA_ROPE, MLA_NOPE + MLA_ROPE
_MLA_SCALE = _MLA_QK ** -0.5
_mla = None
_calls = None


def _mla_lib():
    """The library, bound once."""
    global _mla
    if _mla is None:
        _mla = load()
    return _mla


def _mla_calls():
    """The latent-attention calls and those for drafted tokens in their common form, compiled
    (``csrc/py_mla.cpp``): a decode step launches them every few tens of
    microseconds.  They give NotImplemented for what is not of that form; the
    functions below then check and marshal it themselves."""
    global _calls
    if _calls is None:
        from .build import CALLS_LIB
        if not os.path.exists(CALLS_LIB):
            raise RuntimeError(
                "%s is not built; build it with `python -m serving_kda_chunked_gb300.build`"
                % os.path.basename(CALLS_LIB))
        lib = _mla_lib()
        spec = importlib.util.spec_from_loader(
            "_kda_torch", importlib.machinery.ExtensionFileLoader("_kda_torch", CALLS_LIB))
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
            "kda_mla_append", "kda_mla_prefill", "kda_mla_prefill_workspace_size", "kda_mla_decode",
            "kda_mla_decode_workspace_size", "kda_mla_tree_decode", "kda_mla_tree_decode_workspace_size",
            "kda_tree_step", "kda_gdn_tree_step", "kda_tree_commit", "kda_gdn_tree_commit",
            "kda_tree_verify")), KdaError)
        _calls = module
    return _calls


def _first(name, t, ndim):
    """Type, device and number of dimensions of a call's first tensor, which
    the others have to match."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in _DTYPE_CODE:
        raise ValueError("%s must be bfloat16 or float32" % name)
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor (the KDA kernels run on the GPU only)" % name)
    if t.dim() != ndim:
        raise ValueError("%s must have %d dimensions, got shape %s" % (name, ndim, tuple(t.shape)))
    return t.dtype, dev


def _need(name, t, dtype, shape, dev, rows=False):
    """A tensor of this type, shape and device, contiguous (``rows``: along its
    last dimension, so that views of a projection's output can be passed)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not (t.is_contiguous() or (rows and t.stride(-1) == 1)):
        raise ValueError("%s must be contiguous%s" % (name, " along its last dimension" if rows else ""))
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor (the KDA kernels run on the GPU only)" % name)
        raise ValueError("%s is on %s, but the call is on cuda:%d: all tensors of a call must be "
                         "on one device" % (name, t.device, dev))
    return t.data_ptr()


def _call(fn, dev, stream, *args):
    """Call on device ``dev`` and ``stream`` (default: its current stream)."""
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else int(stream.cuda_stream)
    if torch.cuda.current_device() == dev:
        st = getattr(_mla_lib(), fn)(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = getattr(_mla_lib(), fn)(*args, raw)
    if st != KDA_OK:
        raise KdaError(fn, st)


def _given(name, t, dtype, shape, dev, device, side):
    """(tensor, address) of an output; allocated when omitted."""
    if t is None:
        t = _empty(shape, dtype, device, side)
        return t, t.data_ptr()
    address = _need(name, t, dtype, shape, dev)
    _record(side, t)
    return t, address


def _scratch(workspace, need, dev, device, side):
    """(tensor, address, bytes) of the workspace; allocated when omitted."""
    if workspace is not None:
        n = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
        address = _need("workspace", workspace, torch.uint8, (n,), dev)
        _record(side, workspace)
        return workspace, address, n
    if not need:
        return None, None, 0
    workspace = _empty((need,), torch.uint8, device, side, returned=False)
    return workspace, workspace.data_ptr(), need


def _cache_shape(cache):
    if not isinstance(cache, torch.Tensor):
        raise TypeError("cache must be a torch.Tensor")
    if cache.dim() != 3 or cache.shape[2] != _MLA_ROW:
        raise ValueError("cache must have shape [n_pages, page, %d]" % _MLA_ROW)
    return cache.shape


def kda_mla_append(c, k_r, slots, cache, *, positions=None, rope=None, interleaved=False,
                   k_out=None, q_r=None, q_out=None, stream=None):
    """Tokens into the paged latent cache (``kda_mla_append`` in kda.h).

    c [T, 512] latents and k_r [T, 64] position keys (bf16 or fp32, rows may
    be strided); slots [T] int32; cache [n_pages, page, 576].  With ``rope``
    [max_pos, 64] fp32 (cosines, then sines) and ``positions`` [T] int32 the
    position keys are rotated on the way.  ``k_out`` [T, 64] also receives
    them; ``q_r`` [T, H, 64] (strided) is rotated into ``q_out`` (allocated if
    omitted).  Returns q_out (None without q_r).
    """
    if stream is None:
        done = (_calls or _mla_calls()).append(c, k_r, slots, cache, positions, rope, interleaved,
                                               k_out, q_r, q_out)
        if done is not NotImplemented:
            return done
    dt, dev = _first("c", c, 2)
    T = c.shape[0]
    pc = _need("c", c, dt, (T, MLA_LATENT), dev, True)
    pk = _need("k_r", k_r, dt, (T, MLA_ROPE), dev, True)
    ps = _need("slots", slots, torch.int32, (T,), dev)
    cs = _cache_shape(cache)
    pcache = _need("cache", cache, dt, cs, dev)
    side = _other_stream(stream, c.device)
    pp = pr = pko = pq = pqo = None
    max_pos = kos = H = qt = qh = ot = oh = 0
    if (rope is None) != (positions is None):
        raise ValueError("positions and rope go together")
    if rope is not None:
        pp = _need("positions", positions, torch.int32, (T,), dev)
        max_pos = rope.shape[0]
        pr = _need("rope", rope, torch.float32, (max_pos, MLA_ROPE), dev)
    if k_out is not None:
        pko = _need("k_out", k_out, dt, (T, MLA_ROPE), dev, True)
        kos = k_out.stride(0)
    if q_r is not None:
        H = q_r.shape[1] if isinstance(q_r, torch.Tensor) and q_r.dim() == 3 else -1
        pq = _need("q_r", q_r, dt, (T, H, MLA_ROPE), dev, True)
        if q_out is None:
            q_out, pqo = _given("q_out", None, dt, (T, H, MLA_ROPE), dev, c.device, side)
        else:
            pqo = _need("q_out", q_out, dt, (T, H, MLA_ROPE), dev, True)
            _record(side, q_out)
        qt, qh, _ = q_r.stride()
        ot, oh, _ = q_out.stride()
    elif q_out is not None:
        raise ValueError("q_out needs q_r")
    _record(side, c, k_r, slots, cache, positions, rope, k_out, q_r)
    _call("kda_mla_append", dev, stream, pc, c.stride(0), pk, k_r.stride(0), ps, pp, pr, max_pos,
          1 if interleaved else 0, T, pcache, cs[0], cs[1], MLA_LATENT, MLA_ROPE, _DTYPE_CODE[dt],
          pko, kos, pq, qt, qh, H, pqo, ot, oh)
    return q_out


def kda_mla_prefill_workspace_size(N, Tq, H, dtype) -> int:
    """Workspace bytes ``kda_mla_prefill`` needs (0: none)."""
    code = _DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_mla_lib().kda_mla_prefill_workspace_size(N, Tq, H, code))


def kda_mla_decode_workspace_size(B, H, dtype) -> int:
    """Workspace bytes ``kda_mla_decode`` needs."""
    code = _DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_mla_lib().kda_mla_decode_workspace_size(B, H, code))


def kda_mla_check(workspace, stream=None) -> int:
    """Synchronise the stream and return the device status of the last
    latent-attention call that used ``workspace``."""
    dev = None if workspace is None else workspace.device
    with torch.cuda.device(dev):
        return int(load().kda_mla_check(_ptr(workspace), _stream(stream, dev)))


def kda_mla_prefill(q, kv, k_r, cu_q, cu_k, *, scale=None, causal=True, o=None, lse=None,
                    workspace=None, stream=None):
    """Expanded latent attention over packed prompts (``kda_mla_prefill`` in kda.h).

    q [Tq, H, 192], kv [Tk, H, 256] (key, then value, of each head), k_r
    [Tk, 64] shared position keys, all bf16 or fp32; cu_q, cu_k [N+1] int32 on
    the device.  ``scale`` defaults to 192 ** -0.5.  With ``causal`` the
    queries are the last tokens of their sequence's keys.  Returns
    (o [Tq, H, 128], lse [Tq, H] fp32).
    """
    if stream is None:
        done = (_calls or _mla_calls()).prefill(q, kv, k_r, cu_q, cu_k, scale, causal, o, lse,
                                                workspace)
        if done is not NotImplemented:
            return done
    dt, dev = _first("q", q, 3)
    Tq, H, _ = q.shape
    pq = _need("q", q, dt, (Tq, H, _MLA_QK), dev)
    Tk = kv.shape[0] if isinstance(kv, torch.Tensor) and kv.dim() else -1
    pkv = _need("kv", kv, dt, (Tk, H, MLA_NOPE + MLA_DV), dev)
    pk = _need("k_r", k_r, dt, (Tk, MLA_ROPE), dev)
    N = (cu_q.shape[0] if isinstance(cu_q, torch.Tensor) and cu_q.dim() else 0) - 1
    pcq = _need("cu_q", cu_q, torch.int32, (N + 1,), dev)
    pck = _need("cu_k", cu_k, torch.int32, (N + 1,), dev)
    device = q.device
    side = _other_stream(stream, device)
    o, po = _given("o", o, dt, (Tq, H, MLA_DV), dev, device, side)
    lse, pl = _given("lse", lse, torch.float32, (Tq, H), dev, device, side)
    code = _DTYPE_CODE[dt]
    need = _mla_lib().kda_mla_prefill_workspace_size(N, Tq, H, code)
    workspace, pw, nw = _scratch(workspace, need, dev, device, side)
    _record(side, q, kv, k_r, cu_q, cu_k)
    _call("kda_mla_prefill", dev, stream, pq, pkv, pk, pcq, pck, N, Tq, Tk, H, MLA_NOPE, MLA_ROPE,
          MLA_DV, code, _MLA_SCALE if scale is None else scale, 1 if causal else 0, po, pl, pw, nw)
    return o, lse


def kda_mla_decode(q, cache, table, seq_lens, *, scale=None, o=None, lse=None, workspace=None,
                   stream=None):
    """Absorbed latent attention of one token per sequence over the paged
    cache (``kda_mla_decode`` in kda.h).

    q [B, H, 576] (W_K multiplied in), cache [n_pages, page, 576], both bf16
    or fp32; table [B, max_pages] and seq_lens [B] int32 on the device.
    ``scale`` defaults to 192 ** -0.5, that of the expanded heads.  Returns
    (o [B, H, 512], lse [B, H] fp32).
    """
    if stream is None:
        done = (_calls or _mla_calls()).decode(q, cache, table, seq_lens, scale, o, lse, workspace)
        if done is not NotImplemented:
            return done
    dt, dev = _first("q", q, 3)
    B, H, _ = q.shape
    pq = _need("q", q, dt, (B, H, _MLA_ROW), dev)
    cs = _cache_shape(cache)
    pc = _need("cache", cache, dt, cs, dev)
    width = table.shape[1] if isinstance(table, torch.Tensor) and table.dim() == 2 else -1
    pt = _need("table", table, torch.int32, (B, width), dev)
    pn = _need("seq_lens", seq_lens, torch.int32, (B,), dev)
    device = q.device
    side = _other_stream(stream, device)
    o, po = _given("o", o, dt, (B, H, MLA_LATENT), dev, device, side)
    lse, pl = _given("lse", lse, torch.float32, (B, H), dev, device, side)
    code = _DTYPE_CODE[dt]
    need = _mla_lib().kda_mla_decode_workspace_size(B, H, code)
    workspace, pw, nw = _scratch(workspace, need, dev, device, side)
    _record(side, q, cache, table, seq_lens)
    _call("kda_mla_decode", dev, stream, pq, pc, pt, pn, B, H, cs[0], cs[1], width, MLA_LATENT,
          MLA_ROPE, code, _MLA_SCALE if scale is None else scale, po, pl, pw, nw)
    return o, lse


def kda_mla_tree_decode_workspace_size(B, T, H, dtype) -> int:
    """Workspace bytes ``kda_mla_tree_decode`` needs."""
    code = _DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_mla_lib().kda_mla_tree_decode_workspace_size(B, T, H, code))


def kda_mla_tree_decode(q, cache, table, ctx_lens, parents, *, scale=None, o=None, lse=None,
                        workspace=None, stream=None):
    """Absorbed latent attention of a tree of drafted tokens per sequence
    over the paged cache (``kda_mla_tree_decode`` in kda.h).

    q [B, T, H, 576], cache [n_pages, page, 576], both bf16 or fp32; table
    [B, max_pages], ctx_lens [B] (tokens in front of the tree, whose rows are
    those of tokens ctx_lens .. ctx_lens + T - 1) and parents [B, T] int32 on
    the device.  Returns (o [B, T, H, 512], lse [B, T, H] fp32).
    """
    if stream is None:
        done = (_calls or _mla_calls()).tree_decode(q, cache, table, ctx_lens, parents, scale, o, lse, workspace)
        if done is not NotImplemented:
            return done
    dt, dev = _first("q", q, 4)
    B, T, H, _ = q.shape
    pq = _need("q", q, dt, (B, T, H, _MLA_ROW), dev)
    cs = _cache_shape(cache)
    pc = _need("cache", cache, dt, cs, dev)
    width = table.shape[1] if isinstance(table, torch.Tensor) and table.dim() == 2 else -1
    pt = _need("table", table, torch.int32, (B, width), dev)
    pn = _need("ctx_lens", ctx_lens, torch.int32, (B,), dev)
    pp = _need("parents", parents, torch.int32, (B, T), dev)
    device = q.device
    side = _other_stream(stream, device)
    o, po = _given("o", o, dt, (B, T, H, MLA_LATENT), dev, device, side)
    lse, pl = _given("lse", lse, torch.float32, (B, T, H), dev, device, side)
    code = _DTYPE_CODE[dt]
    need = _mla_lib().kda_mla_tree_decode_workspace_size(B, T, H, code)
    workspace, pw, nw = _scratch(workspace, need, dev, device, side)
    _record(side, q, cache, table, ctx_lens, parents)
    _call("kda_mla_tree_decode", dev, stream, pq, pc, pt, pn, pp, B, T, H, cs[0], cs[1], width,
          MLA_LATENT, MLA_ROPE, code, _MLA_SCALE if scale is None else scale, po, pl, pw, nw)
    return o, lse


def _tree_inputs(k, v, g, beta, S, slots, scalar_gate):
    """What a tree's step and commit check alike: type, device, sizes and addresses."""
    dt, dev = _first("k", k, 4)
    B, T, H, dk = k.shape
    dv = v.shape[-1] if isinstance(v, torch.Tensor) and v.dim() else -1
    pk = _need("k", k, dt, (B, T, H, dk), dev)
    pv = _need("v", v, dt, (B, T, H, dv), dev)
    pg = _need("g", g, torch.float32, (B, T, H) if scalar_gate else (B, T, H, dk), dev)
    pb = _need("beta", beta, torch.float32, (B, T, H), dev)
    P = B
    ps = None
    if slots is not None:
        P = S.shape[0] if isinstance(S, torch.Tensor) and S.dim() else -1
        ps = _need("slots", slots, torch.int32, (B,), dev)
    pS = _need("S", S, torch.float32, (P, H, dk, dv), dev)
    return dt, dev, (B, T, H, dk, dv), P, (pk, pv, pg, pb, pS, ps)


def _tree_step(fn, scalar_gate, q, k, v, g, beta, S, parents, slots, o, stream):
    if stream is None:
        done = (_calls or _mla_calls()).tree_step(scalar_gate, q, k, v, g, beta, S, parents, slots, o)
        if done is not NotImplemented:
            return done
    dt, dev, sizes, P, (pk, pv, pg, pb, pS, ps) = _tree_inputs(k, v, g, beta, S, slots, scalar_gate)
    B, T, H, dk, dv = sizes
    pq = _need("q", q, dt, (B, T, H, dk), dev)
    pp = _need("parents", parents, torch.int32, (B, T), dev)
    device = k.device
    side = _other_stream(stream, device)
    o, po = _given("o", o, dt, (B, T, H, dv), dev, device, side)
    _record(side, q, k, v, g, beta, S, parents, slots)
    _call(fn, dev, stream, pq, pk, pv, pg, pb, pS, ps, P, pp, B, T, H, dk, dv, _DTYPE_CODE[dt], po)
    return o


def kda_tree_step(q, k, v, g, beta, S, parents, *, slots=None, o=None, stream=None):
    """A KDA layer's outputs for a tree of drafted tokens per sequence; the
    states are read only (``kda_tree_step`` in kda.h).

    q, k [B, T, H, dk], v [B, T, H, dv] (bf16 or fp32); g [B, T, H, dk] and
    beta [B, T, H] fp32; parents [B, T] int32; S [B, H, dk, dv] fp32, or with
    ``slots`` [B] int32 a pool [P, H, dk, dv].  Returns o [B, T, H, dv].
    """
    return _tree_step("kda_tree_step", False, q, k, v, g, beta, S, parents, slots, o, stream)


def kda_gdn_tree_step(q, k, v, g, beta, S, parents, *, slots=None, o=None, stream=None):
    """A Gated DeltaNet layer's outputs for a tree of drafted tokens
    (``kda_gdn_tree_step`` in kda.h): as ``kda_tree_step`` with g [B, T, H]."""
    return _tree_step("kda_gdn_tree_step", True, q, k, v, g, beta, S, parents, slots, o, stream)


def _tree_commit(fn, scalar_gate, k, v, g, beta, S, path, slots, stream):
    if stream is None:
        if (_calls or _mla_calls()).tree_commit(scalar_gate, k, v, g, beta, S, path, slots) is not NotImplemented:
            return
    dt, dev, sizes, P, (pk, pv, pg, pb, pS, ps) = _tree_inputs(k, v, g, beta, S, slots, scalar_gate)
    B, T, H, dk, dv = sizes
    pp = _need("path", path, torch.int32, (B, T), dev)
    _record(_other_stream(stream, k.device), k, v, g, beta, S, path, slots)
    _call(fn, dev, stream, pk, pv, pg, pb, pS, ps, P, pp, B, T, H, dk, dv, _DTYPE_CODE[dt])


def kda_tree_commit(k, v, g, beta, S, path, *, slots=None, stream=None):
    """States advanced in place along the accepted path of a tree of drafted
    tokens (``kda_tree_commit`` in kda.h).

    k, v, g, beta, S and ``slots`` as for ``kda_tree_step``; path [B, T] int32
    holds nodes up to the first value outside [0, T) (``kda_tree_verify``'s).
    """
    _tree_commit("kda_tree_commit", False, k, v, g, beta, S, path, slots, stream)


def kda_gdn_tree_commit(k, v, g, beta, S, path, *, slots=None, stream=None):
    """Gated DeltaNet states advanced along the accepted path
    (``kda_gdn_tree_commit`` in kda.h): as ``kda_tree_commit`` with g [B, T, H]."""
    _tree_commit("kda_gdn_tree_commit", True, k, v, g, beta, S, path, slots, stream)


def _vocabulary(name, t, dt, B, T, V, dev):
    """(address, elements between rows) of probabilities [B, T, V], whose rows
    may be the front of longer ones."""
    address = _need(name, t, dt, (B, T, V), dev, True)
    row = t.stride(1) if T > 1 else (t.stride(0) if B > 1 else V)
    if B > 1 and t.stride(0) != T * row:
        raise ValueError("%s must have evenly spaced rows, got strides %s" % (name, t.stride()))
    return address, row


def kda_tree_verify(target, tokens, parents, uniform, *, draft=None, path=None, count=None,
                    next_token=None, stream=None):
    """Which drafted tokens the target model accepts, and the token behind
    the last of them (``kda_tree_verify`` in kda.h).

    target [B, T, V] probabilities (bf16 or fp32) of what follows each node;
    ``draft`` [B, T, V] those from which a node's children were drawn, None
    where they were chosen; rows of both may be the front of longer ones.
    tokens, parents [B, T] int32; uniform [B, T] fp32 random numbers.  Returns
    (path [B, T], count [B], next_token [B]), all int32.
    """
    if stream is None:
        done = (_calls or _mla_calls()).tree_verify(target, tokens, parents, uniform, draft, path, count, next_token)
        if done is not NotImplemented:
            return done
    dt, dev = _first("target", target, 3)
    B, T, V = target.shape
    pt, ts = _vocabulary("target", target, dt, B, T, V, dev)
    pd, ds = _vocabulary("draft", draft, dt, B, T, V, dev) if draft is not None else (None, 0)
    px = _need("tokens", tokens, torch.int32, (B, T), dev)
    pp = _need("parents", parents, torch.int32, (B, T), dev)
    pu = _need("uniform", uniform, torch.float32, (B, T), dev)
    device = target.device
    side = _other_stream(stream, device)
    path, ppath = _given("path", path, torch.int32, (B, T), dev, device, side)
    count, pcount = _given("count", count, torch.int32, (B,), dev, device, side)
    next_token, pnext = _given("next_token", next_token, torch.int32, (B,), dev, device, side)
    _record(side, target, draft, tokens, parents, uniform)
    _call("kda_tree_verify", dev, stream, pt, ts, pd, ds, px, pp, pu, B, T, V, _DTYPE_CODE[dt],
          ppath, pcount, pnext)
    return path, count, next_token
