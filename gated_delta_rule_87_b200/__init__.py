"""Gated delta rule (KDA / Gated DeltaNet) on B200: Python binding.

A thin ctypes layer over the C ABI in ``include/gated_delta.h``
(``libgated_delta.so``, built in-tree for sm_100a).  It only marshals
arguments: every step of the computation runs in the library's CUDA kernels.
PyTorch is used for device memory and streams.  There is no CPU path: if the
library is missing or no CUDA device is present the calls raise.

``stream`` is the stream that a call runs on (default: the current one of the
tensors' device).  Outputs and workspaces that a call allocates belong to it, and
tensors of other streams that it is given are kept until it is past them (the
caller keeps them for a stream that torch does not own); the caller orders it with
the streams that write those tensors and read the results.
No call is recorded by autograd: the gradients are calls of their own (``*_bwd``).

Operator (thethings.ai "The argument, in one page", table "Everything, in
one table", rows "KDA" and "Gated DeltaNet"; column-vector keys):

    S_t = Diag(exp(g_t)) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T
    o_t = S_t^T q_t
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Optional, Tuple

__all__ = [
    "lib", "library_path", "KdaError", "kda_chunk_fwd", "gdn_chunk_fwd", "kda_decode_step",
    "gdn_decode_step", "kda_recurrent_fwd", "gdn_recurrent_fwd", "state_gather", "state_scatter",
    "chunk_workspace_size", "check_device_status", "EXPORTED_SYMBOLS",
    "checked_library_path", "use_library", "bounds_checked", "bounds_violations",
    "kda_chunk_fwd_host",
    "glr_scan_fwd", "glr_scan_bwd", "glr_step", "gated_norm_fwd", "gated_norm_bwd",
    "add_norm_fwd", "add_norm_bwd", "GLR_CHUNK",
    "trace_enable", "trace_read", "ERASE_THEN_DECAY", "DECAY_THEN_ERASE",
    "KDA_OK", "KDA_ERR_INVALID_ARG", "KDA_ERR_UNSUPPORTED", "KDA_ERR_CUDA",
    "KDA_ERR_DEVICE_CHECK", "KDA_ERR_WORKSPACE",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_PKG, "libgated_delta.so")
# the bounds-checked build of the same sources (see kda_bounds_checked)
checked_library_path = os.path.join(_PKG, "libgated_delta_checked.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_DEVICE_CHECK, \
    KDA_ERR_WORKSPACE = range(6)
KDA_F32, KDA_BF16 = 0, 1
# device codes in a workspace's status word (kda_check_device_status)
KDA_DEVICE_OK, KDA_DEVICE_BAD_CU_SEQLENS, KDA_DEVICE_TIMEOUT = 0, 1, 2
# decay order (KDA): the table's literal order, or the decay applied before the erase
ERASE_THEN_DECAY, DECAY_THEN_ERASE = "erase_then_decay", "decay_then_erase"
# gated linear recurrence: b_t = x_t, or (1 - a_t) x_t; tokens between two saved states
_GLR_INPUT = {"given": 0, "complement": 1}
GLR_CHUNK = 64
_GATE = {None: 0, "silu": 1, "sigmoid": 2}
_ORDER = {ERASE_THEN_DECAY: 0, DECAY_THEN_ERASE: 1}

EXPORTED_SYMBOLS = (
    "kda_chunk_fwd", "kda_chunk_fwd_workspace_size", "gdn_chunk_fwd",
    "gdn_chunk_fwd_workspace_size", "kda_decode_step", "gdn_decode_step",
    "kda_check_device_status", "kda_status_string", "kda_last_error", "kda_abi_version",
    "kda_trace_enable", "kda_trace_read", "kda_chunk_fwd_noalloc", "kda_chunk_fwd_ex",
    "gdn_chunk_fwd_ex", "kda_recurrent_fwd", "gdn_recurrent_fwd", "kda_state_gather",
    "kda_state_scatter", "kda_selftest_wait_timeout", "kda_bounds_checked",
    "kda_bounds_violations", "kda_chunk_fwd_host", "kda_chunk_fwd_host_buffer_size",
    "glr_chunk_states_size", "glr_scan_fwd_workspace_size", "glr_scan_fwd",
    "glr_scan_bwd_workspace_size", "glr_scan_bwd", "glr_selftest_wait_timeout", "glr_step",
    "kda_gated_norm_fwd",
    "kda_gated_norm_bwd_workspace_size", "kda_gated_norm_bwd", "kda_add_norm_fwd",
    "kda_add_norm_bwd_workspace_size", "kda_add_norm_bwd",
)

_lock = threading.Lock()
_lib = None

_vp, _fp, _i32, _sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_i64, _int, _f = ctypes.c_int64, ctypes.c_int, ctypes.c_float
_SIGS = {
    "kda_chunk_fwd_ex": ([_vp] * 9 + [_i64, _vp] + [_i32] * 6 + [_int, _int, _vp, _sz, _vp], _int),
    "gdn_chunk_fwd_ex": ([_vp] * 9 + [_i64, _vp] + [_i32] * 7 + [_int, _vp, _sz, _vp], _int),
    "kda_recurrent_fwd": ([_vp] * 8 + [_i64] + [_i32] * 5 + [_int, _int, _vp], _int),
    "gdn_recurrent_fwd": ([_vp] * 8 + [_i64] + [_i32] * 6 + [_int, _vp], _int),
    "kda_state_gather": ([_vp, _vp, _i64, _vp] + [_i32] * 4 + [_vp], _int),
    "kda_state_scatter": ([_vp, _vp, _vp, _i64] + [_i32] * 4 + [_vp], _int),
    "kda_chunk_fwd": ([_vp] * 9 + [_i32] * 6 + [ctypes.c_int, _vp, _sz, _vp], ctypes.c_int),
    "gdn_chunk_fwd": ([_vp] * 9 + [_i32] * 7 + [ctypes.c_int, _vp, _sz, _vp], ctypes.c_int),
    "kda_chunk_fwd_workspace_size": ([_i32] * 6 + [ctypes.c_int], _sz),
    "gdn_chunk_fwd_workspace_size": ([_i32] * 7 + [ctypes.c_int], _sz),
    "kda_decode_step": ([_vp] * 7 + [_i32] * 4 + [ctypes.c_int, _vp], ctypes.c_int),
    "gdn_decode_step": ([_vp] * 7 + [_i32] * 5 + [ctypes.c_int, _vp], ctypes.c_int),
    "kda_check_device_status": ([_vp, _vp, ctypes.POINTER(_i32)], ctypes.c_int),
    "kda_selftest_wait_timeout": ([_vp, _i32, _vp], ctypes.c_int),
    "kda_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "kda_last_error": ([], ctypes.c_char_p),
    "kda_abi_version": ([], _i32),
    "kda_trace_enable": ([_i32], ctypes.c_int),
    "kda_chunk_fwd_noalloc": ([_vp] * 9 + [_i32] * 6 + [ctypes.c_int, _vp], ctypes.c_int),
    "kda_trace_read": ([ctypes.c_char_p, _i32, ctypes.POINTER(ctypes.c_float), _i32], _i32),
    "kda_bounds_checked": ([], _i32),
    "kda_chunk_fwd_host_buffer_size": ([_i32] * 5 + [ctypes.c_int, _i32], _sz),
    "kda_chunk_fwd_host": ([_vp] * 8 + [_i32] * 5 + [ctypes.c_int, _i32, _vp, _sz, _vp], ctypes.c_int),
    "glr_chunk_states_size": ([_i32] * 3, _sz),
    "glr_scan_fwd_workspace_size": ([_i32] * 3, _sz),
    "glr_scan_bwd_workspace_size": ([_i32] * 4, _sz),
    "glr_scan_fwd": ([_vp, _i64, _vp, _i64] + [_vp] * 4 + [_i64, _vp, _vp] + [_i32] * 4
                     + [_int, _int, _vp, _sz, _vp], _int),
    "glr_scan_bwd": ([_vp, _i64, _vp, _vp, _i64, _vp, _i64] + [_vp] * 6 + [_i32] * 4
                     + [_int, _int, _vp, _sz, _vp], _int),
    "glr_selftest_wait_timeout": ([_i32] + [_vp] * 4 + [_i32, _i32, _vp, _sz, _vp], _int),
    "glr_step": ([_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i32, _i32, _int, _int, _vp], _int),
    "kda_gated_norm_fwd": ([_vp, _i64, _vp, _i64, _vp, _vp, _i64, _i32, _i32, _f, _int, _int, _vp],
                           _int),
    "kda_gated_norm_bwd_workspace_size": ([_i32], _sz),
    "kda_gated_norm_bwd": ([_vp, _i64] * 3 + [_vp] * 4 + [_i64, _i32, _i32, _f, _int, _int, _vp,
                                                          _sz, _vp], _int),
    "kda_add_norm_fwd": ([_vp] * 6 + [_i64, _i32, _f, _int, _int, _vp], _int),
    "kda_add_norm_bwd_workspace_size": ([_i32], _sz),
    "kda_add_norm_bwd": ([_vp] * 10 + [_i64, _i32, _f, _int, _int, _vp, _sz, _vp], _int),
    "kda_bounds_violations": ([_vp, ctypes.POINTER(ctypes.c_uint32)], ctypes.c_int),
}


class KdaError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{detail} (status {status})")


_libs = {}                   # path -> loaded CDLL
_active_path = library_path  # the library the calls below go through


def _load(path: str) -> ctypes.CDLL:
    with _lock:
        L = _libs.get(path)
        if L is None:
            if not os.path.exists(path):
                raise ImportError(
                    f"{path} is missing: build it with "
                    "`python -m gated_delta_rule_87_b200.build` (nvcc, sm_100a)")
            L = ctypes.CDLL(path)
            for name, (args, res) in _SIGS.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = res
            _libs[path] = L
    return L


def lib() -> ctypes.CDLL:
    """Load ``libgated_delta.so`` (raises if it has not been built), or the
    library selected by :func:`use_library`."""
    global _lib
    L = _libs.get(_active_path)
    if L is None:
        L = _load(_active_path)
    if _active_path == library_path:
        _lib = L
    return L


@contextlib.contextmanager
def use_library(path: str):
    """Route every call of this module through the library at ``path`` (for
    instance :data:`checked_library_path`) inside the ``with`` block."""
    global _active_path
    prev = _active_path
    L = _load(path)
    _active_path = path
    try:
        yield L
    finally:
        _active_path = prev


def bounds_checked() -> bool:
    """True when the active library is the bounds-checked build."""
    return bool(lib().kda_bounds_checked())


def bounds_violations() -> int:
    """Waits for the current stream and returns the out-of-bounds accesses the
    active library's kernels caught (and skipped) since the last call."""
    n = ctypes.c_uint32(0)
    _check(lib().kda_bounds_violations(_stream_handle(None, None), ctypes.byref(n)),
           "kda_bounds_violations")
    return int(n.value)


def _check(status: int, what: str):
    if status != KDA_OK:
        L = lib()
        msg = L.kda_last_error().decode() or L.kda_status_string(status).decode()
        raise KdaError(status, f"{what}: {msg}")


# --------------------------------------------------------------------------- #
# torch plumbing
# --------------------------------------------------------------------------- #
def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _host_ptr(t) -> Optional[int]:
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError("tensors must live in host memory")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream_handle(stream, device) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def _raw_stream(torch, dev) -> int:
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # 1.3 us less than the Stream object
    return raw(dev) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _here(torch, dev, stream) -> bool:
    """Whether ``dev`` is the current device and ``stream`` (None: any) its current stream."""
    return torch.cuda.current_device() == dev and (stream is None
                                                   or stream.cuda_stream == _raw_stream(torch, dev))


def _there(torch, dev, stream, call, *args, **kw):
    """``call`` with ``dev`` and ``stream`` as the current ones.  What it allocates
    (outputs, workspace) then belongs to the stream that uses it: memory freed on
    another stream is not written while that one still reads it, and a workspace
    that the caller drops is not handed out again before the stream is past it.
    Tensors of other streams are recorded, so the same holds for them; not on a
    stream that torch does not own, which may be gone when they are freed."""
    with torch.cuda.device(dev):
        if stream is None:
            return call(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream.cuda_stream, device=dev)
        elif stream.device.index != dev:
            raise ValueError(f"stream must belong to CUDA device {dev}")
        with torch.cuda.stream(stream):
            out = call(*args, **kw)
        if not isinstance(stream, torch.cuda.ExternalStream):
            for t in (*args, *kw.values()):
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(stream)
        return out


def _f32(t, name):
    torch = _torch()
    if t is not None and t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    return t


def chunk_workspace_size(B: int, T: int, H_qk: int, H_v: int, d_k: int, d_v: int,
                         num_seqs: int, io_dtype: int, gate: str = "channel") -> int:
    L = lib()
    if gate == "channel":
        return int(L.kda_chunk_fwd_workspace_size(B, T, H_v, d_k, d_v, num_seqs, io_dtype))
    return int(L.gdn_chunk_fwd_workspace_size(B, T, H_qk, H_v, d_k, d_v, num_seqs, io_dtype))


def _alloc_workspace(nbytes: int, device):
    torch = _torch()
    # 256-byte alignment: torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _order_code(order) -> int:
    if order not in _ORDER:
        raise ValueError(f"order must be one of {sorted(_ORDER)}, got {order!r}")
    return _ORDER[order]


def _slots(state_slots, state_pool, N):
    torch = _torch()
    if state_slots is None:
        if state_pool is not None:
            raise ValueError("state_pool needs state_slots")
        return None, 0
    if state_pool is None:
        raise ValueError("state_slots needs state_pool")
    if state_slots.dtype != torch.int32 or state_slots.numel() != N:
        raise ValueError(f"state_slots must be int32 with {N} entries")
    return state_slots, state_pool.shape[0]


def _chunk_fwd(gate, q, k, v, g, beta, initial_state, cu_seqlens, output_final_state,
               o, final_state, workspace, stream, order=ERASE_THEN_DECAY, state_pool=None,
               state_slots=None):
    torch = _torch()
    if stream is not None and q.is_cuda and not _here(torch, q.get_device(), stream):
        return _there(torch, q.get_device(), stream, _chunk_fwd, gate, q, k, v, g, beta,
                      initial_state, cu_seqlens, output_final_state, o, final_state, workspace,
                      None, order, state_pool, state_slots)
    if q.dim() != 4:
        raise ValueError("q, k, v must be [B, T, H, d]")
    B, T, H_qk, d_k = q.shape
    H_v, d_v = v.shape[2], v.shape[3]
    io = _dtype_code(q)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share a dtype")
    _f32(g, "g"), _f32(beta, "beta"), _f32(initial_state, "initial_state")
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        N = cu_seqlens.numel() - 1
    else:
        N = B
    dev = q.device
    if o is None:
        o = torch.empty((B, T, H_v, d_v), dtype=q.dtype, device=dev)
    slots, num_slots = _slots(state_slots, state_pool, N)
    if slots is not None:
        # pool mode: read and update pool[state_slots[n]] in place
        if initial_state is not None or final_state is not None:
            raise ValueError("with state_pool, pass neither initial_state nor final_state")
        _f32(state_pool, "state_pool")
        initial_state = final_state = state_pool
    elif final_state is None and output_final_state:
        final_state = torch.empty((N, H_v, d_k, d_v), dtype=torch.float32, device=dev)
    need = chunk_workspace_size(B, T, H_qk, H_v, d_k, d_v, N if cu_seqlens is not None else 0,
                                io, gate)
    if workspace is None or workspace.numel() < need:
        workspace = _alloc_workspace(need, dev)
    L = lib()
    args_common = [_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(o), _ptr(initial_state),
                   _ptr(final_state), _ptr(slots), num_slots, _ptr(cu_seqlens), N]
    sh = _stream_handle(stream, dev)
    if gate == "channel":
        st = L.kda_chunk_fwd_ex(*args_common, B, T, H_v, d_k, d_v, _order_code(order), io,
                                _ptr(workspace), workspace.numel(), sh)
        _check(st, "kda_chunk_fwd_ex")
    else:
        st = L.gdn_chunk_fwd_ex(*args_common, B, T, H_qk, H_v, d_k, d_v, io, _ptr(workspace),
                                workspace.numel(), sh)
        _check(st, "gdn_chunk_fwd_ex")
    return o, final_state, workspace


def kda_chunk_fwd(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *,
                  output_final_state: bool = True, o=None, final_state=None, workspace=None,
                  stream=None, order: str = ERASE_THEN_DECAY, state_pool=None,
                  state_slots=None):
    """KDA prefill.  q, k [B,T,H,d_k]; v [B,T,H,d_v] (bf16 or fp32); g [B,T,H,d_k]
    fp32 log-decay; beta [B,T,H] fp32; initial_state [N,H,d_k,d_v] fp32 or None;
    cu_seqlens int32 [N+1] (device) for packed sequences with B = 1.
    ``order`` places the decay after (default) or before the erase.  With
    ``state_pool`` [num_slots,H,d_k,d_v] and ``state_slots`` int32 [N], sequence
    n starts from pool[state_slots[n]] and its final state is written back
    there (slots outside the pool: start from zeros, no final state).
    Returns (o, final_state, workspace); final_state is the pool in pool mode."""
    return _chunk_fwd("channel", q, k, v, g, beta, initial_state, cu_seqlens,
                      output_final_state, o, final_state, workspace, stream, order, state_pool,
                      state_slots)


def kda_chunk_fwd_host(q, k, v, g, beta, initial_state=None, *, o, final_state=None,
                       device_buffer=None, pieces: int = 4, stream=None, device=None):
    """KDA prefill from pinned HOST tensors (dense batch; layouts as
    kda_chunk_fwd), the copies overlapped with the kernels (see the C call).
    ``o`` (and ``final_state`` if given) are host tensors the results land in
    once the stream is synchronised.  ``device_buffer`` (uint8, on the device)
    is allocated when None.  Returns the device buffer (its first bytes hold
    the status word for check_device_status)."""
    torch = _torch()
    if q.is_cuda or o.is_cuda:
        raise ValueError("kda_chunk_fwd_host takes host tensors")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    index = torch.device(dev).index if not isinstance(dev, int) else dev
    if stream is not None and index is not None and not _here(torch, index, stream):
        return _there(torch, index, stream, kda_chunk_fwd_host, q, k, v, g, beta, initial_state,
                      o=o, final_state=final_state, device_buffer=device_buffer, pieces=pieces,
                      device=dev)
    B, T, H, d_k = q.shape
    d_v = v.shape[3]
    io = _dtype_code(q)
    _f32(g, "g"), _f32(beta, "beta"), _f32(initial_state, "initial_state")
    _f32(final_state, "final_state")
    L = lib()
    need = int(L.kda_chunk_fwd_host_buffer_size(B, T, H, d_k, d_v, io, pieces))
    if device_buffer is None or device_buffer.numel() < need:
        device_buffer = torch.empty(need, dtype=torch.uint8, device=dev)
    sh = _stream_handle(stream, dev)
    hp = _host_ptr
    _check(L.kda_chunk_fwd_host(hp(q), hp(k), hp(v), hp(g), hp(beta), hp(o),
                                hp(initial_state), hp(final_state), B, T, H, d_k, d_v, io,
                                pieces, _ptr(device_buffer), device_buffer.numel(), sh),
           "kda_chunk_fwd_host")
    return device_buffer


def gdn_chunk_fwd(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *,
                  output_final_state: bool = True, o=None, final_state=None, workspace=None,
                  stream=None, state_pool=None, state_slots=None):
    """Gated DeltaNet prefill.  q, k [B,T,H_qk,d_k]; v [B,T,H_v,d_v]; g, beta
    [B,T,H_v] fp32 (scalar log-decay per head-token).  ``state_pool`` /
    ``state_slots`` as in kda_chunk_fwd.  Returns (o, final_state, workspace)."""
    return _chunk_fwd("scalar", q, k, v, g, beta, initial_state, cu_seqlens,
                      output_final_state, o, final_state, workspace, stream, ERASE_THEN_DECAY,
                      state_pool, state_slots)


def _decode(gate, q, k, v, g, beta, state, o, stream):
    torch = _torch()
    if stream is not None and q.is_cuda and not _here(torch, q.get_device(), stream):
        return _there(torch, q.get_device(), stream, _decode, gate, q, k, v, g, beta, state, o,
                      None)
    N, H_qk, d_k = q.shape
    H_v, d_v = v.shape[1], v.shape[2]
    io = _dtype_code(q)
    _f32(g, "g"), _f32(beta, "beta"), _f32(state, "state")
    if o is None:
        o = torch.empty((N, H_v, d_v), dtype=q.dtype, device=q.device)
    L = lib()
    sh = _stream_handle(stream, q.device)
    ptrs = [_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(o), _ptr(state)]
    if gate == "channel":
        _check(L.kda_decode_step(*ptrs, N, H_v, d_k, d_v, io, sh), "kda_decode_step")
    else:
        _check(L.gdn_decode_step(*ptrs, N, H_qk, H_v, d_k, d_v, io, sh), "gdn_decode_step")
    return o


def _recurrent(gate, q, k, v, g, beta, state, state_slots, order, o, stream):
    torch = _torch()
    if stream is not None and q.is_cuda and not _here(torch, q.get_device(), stream):
        return _there(torch, q.get_device(), stream, _recurrent, gate, q, k, v, g, beta, state,
                      state_slots, order, o, None)
    if q.dim() != 4:
        raise ValueError("q, k, v must be [N, T, H, d]")
    N, T, H_qk, d_k = q.shape
    H_v, d_v = v.shape[2], v.shape[3]
    io = _dtype_code(q)
    _f32(g, "g"), _f32(beta, "beta"), _f32(state, "state")
    slots, num_slots = _slots(state_slots, state if state_slots is not None else None, N)
    if o is None:
        o = torch.empty((N, T, H_v, d_v), dtype=q.dtype, device=q.device)
    L = lib()
    sh = _stream_handle(stream, q.device)
    ptrs = [_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(o), _ptr(state), _ptr(slots)]
    if gate == "channel":
        _check(L.kda_recurrent_fwd(*ptrs, num_slots, N, T, H_v, d_k, d_v, _order_code(order), io,
                                   sh), "kda_recurrent_fwd")
    else:
        _check(L.gdn_recurrent_fwd(*ptrs, num_slots, N, T, H_qk, H_v, d_k, d_v, io, sh),
               "gdn_recurrent_fwd")
    return o


def kda_recurrent_fwd(q, k, v, g, beta, state, *, state_slots=None,
                      order: str = ERASE_THEN_DECAY, o=None, stream=None):
    """T tokens for each of N sequences, token by token, state updated in place
    (read once, written once).  q, k [N,T,H,d_k]; v [N,T,H,d_v]; g [N,T,H,d_k];
    beta [N,T,H].  ``state`` is [N,H,d_k,d_v], or a pool [num_slots,H,d_k,d_v]
    indexed by ``state_slots`` (int32 [N]; a slot outside the pool is a padding
    entry: zero output, no state).  Returns o [N,T,H,d_v]."""
    return _recurrent("channel", q, k, v, g, beta, state, state_slots, order, o, stream)


def gdn_recurrent_fwd(q, k, v, g, beta, state, *, state_slots=None, o=None, stream=None):
    """Gated DeltaNet form of kda_recurrent_fwd: q, k [N,T,H_qk,d_k]; v [N,T,H_v,d_v];
    g, beta [N,T,H_v].  Returns o [N,T,H_v,d_v]."""
    return _recurrent("scalar", q, k, v, g, beta, state, state_slots, ERASE_THEN_DECAY, o,
                      stream)


def state_gather(pool, state_slots, *, out=None, stream=None):
    """out[n] = pool[state_slots[n]] (zeros for a slot outside the pool)."""
    torch = _torch()
    if stream is not None and pool.is_cuda and not _here(torch, pool.get_device(), stream):
        return _there(torch, pool.get_device(), stream, state_gather, pool, state_slots, out=out)
    _f32(pool, "pool")
    N = state_slots.numel()
    _slots(state_slots, pool, N)
    _, H, d_k, d_v = pool.shape
    if out is None:
        out = torch.empty((N, H, d_k, d_v), dtype=torch.float32, device=pool.device)
    _check(lib().kda_state_gather(_ptr(pool), _ptr(state_slots), pool.shape[0], _ptr(out), N, H,
                                  d_k, d_v, _stream_handle(stream, pool.device)),
           "kda_state_gather")
    return out


def state_scatter(src, pool, state_slots, *, stream=None):
    """pool[state_slots[n]] = src[n] (skipped for a slot outside the pool)."""
    torch = _torch()
    if stream is not None and pool.is_cuda and not _here(torch, pool.get_device(), stream):
        return _there(torch, pool.get_device(), stream, state_scatter, src, pool, state_slots)
    _f32(src, "src"), _f32(pool, "pool")
    N = state_slots.numel()
    _slots(state_slots, pool, N)
    _, H, d_k, d_v = pool.shape
    _check(lib().kda_state_scatter(_ptr(src), _ptr(pool), _ptr(state_slots), pool.shape[0], N, H,
                                   d_k, d_v, _stream_handle(stream, pool.device)),
           "kda_state_scatter")
    return pool


def kda_decode_step(q, k, v, g, beta, state, *, o=None, stream=None):
    """One KDA decode step; ``state`` [N,H,d_k,d_v] fp32 is updated in place.
    q, k [N,H,d_k]; v [N,H,d_v]; g [N,H,d_k]; beta [N,H].  Returns o [N,H,d_v]."""
    return _decode("channel", q, k, v, g, beta, state, o, stream)


def gdn_decode_step(q, k, v, g, beta, state, *, o=None, stream=None):
    """One Gated DeltaNet decode step (scalar gate, q/k heads shared by groups of
    v heads); ``state`` is updated in place.  Returns o [N,H_v,d_v]."""
    return _decode("scalar", q, k, v, g, beta, state, o, stream)


# --------------------------------------------------------------------------- #
# gated linear recurrence and the norms around a mixer block
# --------------------------------------------------------------------------- #
# These calls are small next to their launches' cost on the host: arguments are
# looked at once, in plain code.
def _dense(t, shape, dtype, name, dev):
    """Pointer of a contiguous tensor of this shape, type and device, or None."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must live on CUDA device {dev}")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _rows(t, shape, dtype, name, dev, inner=1):
    """(pointer, elements from one row to the next) of a tensor whose last
    ``inner`` axes are contiguous and whose leading axes step evenly."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must live on CUDA device {dev}")
    width = shape[-1] if inner == 1 else shape[-1] * shape[-2]
    if t.is_contiguous():
        return t.data_ptr(), width
    step, strides = 1, t.stride()
    for i in range(len(shape) - 1, len(shape) - 1 - inner, -1):
        if shape[i] != 1 and strides[i] != step:
            raise ValueError(f"{name}: the last {inner} axes must be contiguous")
        step *= shape[i]
    ld = None
    for i in range(len(shape) - 1 - inner, -1, -1):
        if shape[i] == 1:
            continue
        if ld is None:
            ld = strides[i]
            step = ld * shape[i]
        elif strides[i] != step:
            raise ValueError(f"{name}: the leading axes must step evenly (one row stride)")
        else:
            step *= shape[i]
    ld = width if ld is None else ld
    if ld < width:
        raise ValueError(f"{name}: rows must not overlap")
    return t.data_ptr(), ld


def _bytes(t, name, dev):
    """Pointer and size of a workspace."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must live on CUDA device {dev}")
    return _ptr(t), t.numel() * t.element_size()


def _device_of(t) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must live on a CUDA device")
    return dev


def _like(torch, t):
    """An empty contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _done(status, what):
    if status:
        _check(status, what)


def _glr_input(name) -> int:
    if name not in _GLR_INPUT:
        raise ValueError(f"input_gate must be one of {sorted(_GLR_INPUT)}, got {name!r}")
    return _GLR_INPUT[name]


def _glr_shape(torch, x, cu_seqlens, dev):
    """(B, T, D, sequences, pointer of cu_seqlens)."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    if cu_seqlens is None:
        return B, T, D, B, None
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [N + 1]")
    return B, T, D, cu_seqlens.numel() - 1, _dense(cu_seqlens, cu_seqlens.shape, torch.int32, "cu_seqlens", dev)


def _glr_slots(torch, state_slots, pool, N, D, dev, name):
    """(pointer of the slots, rows of the pool)."""
    if pool.dim() != 2:
        raise ValueError(f"{name} must be [num_slots, {D}]")
    return _dense(state_slots, (N,), torch.int32, "state_slots", dev), pool.shape[0]


def glr_scan_fwd(x, g, initial_state=None, cu_seqlens=None, *, input_gate: str = "given",
                 output_final_state: bool = True, output_chunk_states: bool = False, h=None,
                 final_state=None, chunk_states=None, workspace=None, stream=None,
                 state_pool=None, state_slots=None):
    """Gated linear recurrence h_t = exp(g_t) h_{t-1} + b_t over sequences.
    x [B,T,D] (bf16 or fp32); g [B,T,D] fp32 log-decay; ``input_gate`` "given"
    (b = x) or "complement" (b = (1 - exp(g)) x); initial_state [N,D] fp32 or
    None; cu_seqlens int32 [N+1] (device) for packed sequences with B = 1.  x and
    g may be slices of wider rows.  ``state_pool`` [num_slots,D] with
    ``state_slots`` as in kda_chunk_fwd.  ``output_chunk_states`` (or a
    ``chunk_states`` tensor [ceil(B T / 64), D] fp32) keeps what glr_scan_bwd
    reads.  Returns (h, final_state, chunk_states, workspace)."""
    torch = _torch()
    dev = _device_of(x)
    if not _here(torch, dev, stream):
        return _there(torch, dev, stream, glr_scan_fwd, x, g, initial_state, cu_seqlens,
                      input_gate=input_gate, output_final_state=output_final_state,
                      output_chunk_states=output_chunk_states, h=h, final_state=final_state,
                      chunk_states=chunk_states, workspace=workspace, state_pool=state_pool,
                      state_slots=state_slots)
    io, code, f32, L = _dtype_code(x), _glr_input(input_gate), torch.float32, lib()
    B, T, D, N, cup = _glr_shape(torch, x, cu_seqlens, dev)
    shape, chunks = (B, T, D), (-(-B * T // GLR_CHUNK), D)
    xp, ld_x = _rows(x, shape, x.dtype, "x", dev)
    gp, ld_g = _rows(g, shape, f32, "g", dev)
    slots, rows = None, N
    if (state_slots is None) != (state_pool is None):
        raise ValueError("state_pool and state_slots go together")
    if state_pool is not None:
        if initial_state is not None or final_state is not None:
            raise ValueError("with state_pool, pass neither initial_state nor final_state")
        slots, rows = _glr_slots(torch, state_slots, state_pool, N, D, dev, "state_pool")
        initial_state = final_state = state_pool
    elif final_state is None and output_final_state:
        final_state = torch.empty((N, D), dtype=f32, device=x.device)
    if h is None:
        h = _like(torch, x)
    if chunk_states is None and output_chunk_states:
        chunk_states = torch.empty(chunks, dtype=f32, device=x.device)
    need = L.glr_scan_fwd_workspace_size(B, T, D)
    if workspace is None or workspace.numel() < need:
        workspace = _alloc_workspace(need, x.device)
    wp, have = _bytes(workspace, "workspace", dev)
    _done(L.glr_scan_fwd(
        xp, ld_x, gp, ld_g, _dense(h, shape, x.dtype, "h", dev),
        _dense(initial_state, (rows, D), f32, "initial_state", dev),
        _dense(final_state, (rows, D), f32, "final_state", dev), slots, rows,
        _dense(chunk_states, chunks, f32, "chunk_states", dev), cup, N, B, T, D, code, io, wp, have,
        _raw_stream(torch, dev)), "glr_scan_fwd")
    return h, final_state, chunk_states, workspace


def glr_scan_bwd(dh, x, g, initial_state=None, cu_seqlens=None, *, input_gate: str = "given",
                 dfinal_state=None, chunk_states=None, output_dinitial_state: bool = True,
                 dx=None, dg=None, dinitial_state=None, workspace=None, stream=None):
    """Gradients of glr_scan_fwd: dh [B,T,D] is the gradient of h, dfinal_state
    [N,D] that of the final state (None: zeros); x, g, initial_state, cu_seqlens
    and input_gate as in the forward call, ``chunk_states`` what it returned
    (None: computed again).  Returns (dx, dg, dinitial_state, workspace)."""
    torch = _torch()
    dev = _device_of(x)
    if not _here(torch, dev, stream):
        return _there(torch, dev, stream, glr_scan_bwd, dh, x, g, initial_state, cu_seqlens,
                      input_gate=input_gate, dfinal_state=dfinal_state, chunk_states=chunk_states,
                      output_dinitial_state=output_dinitial_state, dx=dx, dg=dg, dinitial_state=dinitial_state,
                      workspace=workspace)
    io, code, f32, L = _dtype_code(x), _glr_input(input_gate), torch.float32, lib()
    B, T, D, N, cup = _glr_shape(torch, x, cu_seqlens, dev)
    shape, chunks, states = (B, T, D), (-(-B * T // GLR_CHUNK), D), (N, D)
    dp, ld_dh = _rows(dh, shape, x.dtype, "dh", dev)
    xp, ld_x = _rows(x, shape, x.dtype, "x", dev)
    gp, ld_g = _rows(g, shape, f32, "g", dev)
    if dx is None:
        dx = _like(torch, x)
    if dg is None:
        dg = _like(torch, g)
    if dinitial_state is None and output_dinitial_state:
        dinitial_state = torch.empty(states, dtype=f32, device=x.device)
    need = L.glr_scan_bwd_workspace_size(B, T, D, chunk_states is not None)
    if workspace is None or workspace.numel() < need:
        workspace = _alloc_workspace(need, x.device)
    wp, have = _bytes(workspace, "workspace", dev)
    _done(L.glr_scan_bwd(
        dp, ld_dh, _dense(dfinal_state, states, f32, "dfinal_state", dev), xp, ld_x, gp, ld_g,
        _dense(initial_state, states, f32, "initial_state", dev),
        _dense(chunk_states, chunks, f32, "chunk_states", dev),
        _dense(dx, shape, x.dtype, "dx", dev), _dense(dg, shape, f32, "dg", dev),
        _dense(dinitial_state, states, f32, "dinitial_state", dev), cup, N, B, T, D, code, io, wp,
        have, _raw_stream(torch, dev)), "glr_scan_bwd")
    return dx, dg, dinitial_state, workspace


def glr_step(x, g, state, *, state_slots=None, input_gate: str = "given", h=None, stream=None):
    """One token of the gated linear recurrence for each of N sequences: x [N,D]
    (bf16 or fp32), g [N,D] fp32; ``state`` [N,D] fp32, or a pool [num_slots,D]
    indexed by ``state_slots`` (int32 [N]; a slot outside the pool is a padding
    entry), is updated in place.  Returns h [N,D]."""
    torch = _torch()
    dev = _device_of(x)
    if not _here(torch, dev, stream):
        return _there(torch, dev, stream, glr_step, x, g, state, state_slots=state_slots,
                      input_gate=input_gate, h=h)
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    io, code, f32, shape = _dtype_code(x), _glr_input(input_gate), torch.float32, x.shape
    N, D = shape
    xp, ld_x = _rows(x, shape, x.dtype, "x", dev)
    gp, ld_g = _rows(g, shape, f32, "g", dev)
    slots, rows = None, N
    if state_slots is not None:
        slots, rows = _glr_slots(torch, state_slots, state, N, D, dev, "state")
    if h is None:
        h = _like(torch, x)
    _done(lib().glr_step(
        xp, ld_x, gp, ld_g, _dense(h, shape, x.dtype, "h", dev),
        _dense(state, (rows, D), f32, "state", dev), slots, rows, N, D, code, io,
        _raw_stream(torch, dev)), "glr_step")
    return h


def _gate_code(gate, z) -> int:
    if gate not in _GATE:
        raise ValueError(f"gate must be None, 'silu' or 'sigmoid', got {gate!r}")
    if (z is None) != (gate is None):
        raise ValueError("z goes with a gate, and a gate with z")
    return _GATE[gate]


def _heads(shape):
    """(tokens, H, d) of [..., H, d]."""
    if len(shape) < 2:
        raise ValueError("x must be [..., H, d]")
    tokens = 1
    for n in shape[:-2]:
        tokens *= n
    return tokens, shape[-2], shape[-1]


def gated_norm_fwd(x, z=None, weight=None, *, gate: Optional[str] = "silu", eps: float = 1e-6,
                   y=None, stream=None):
    """Gated RMS norm over each head's channels: y = x / rms(x) * weight * s(z).
    x, z [...,H,d] (bf16 or fp32; z may be a slice of wider token rows), weight
    fp32 [d] or None; ``gate`` "silu", "sigmoid" or None (then no z).  Returns y."""
    torch = _torch()
    dev = _device_of(x)
    if not _here(torch, dev, stream):
        return _there(torch, dev, stream, gated_norm_fwd, x, z, weight, gate=gate, eps=eps, y=y)
    code, io, dtype, shape = _gate_code(gate, z), _dtype_code(x), x.dtype, x.shape
    tokens, H, d = _heads(shape)
    xp, ld_x = _rows(x, shape, dtype, "x", dev, 2)
    zp, ld_z = (None, 0) if z is None else _rows(z, shape, dtype, "z", dev, 2)
    if y is None:
        y = _like(torch, x)
    _done(lib().kda_gated_norm_fwd(
        xp, ld_x, zp, ld_z, _dense(weight, (d,), torch.float32, "weight", dev),
        _dense(y, shape, dtype, "y", dev), tokens, H, d, eps, code, io,
        _raw_stream(torch, dev)), "kda_gated_norm_fwd")
    return y


def gated_norm_bwd(dy, x, z=None, weight=None, *, gate: Optional[str] = "silu",
                   eps: float = 1e-6, output_dweight: bool = True, dx=None, dz=None,
                   dweight=None, workspace=None, stream=None):
    """Gradients of gated_norm_fwd.  Returns (dx, dz, dweight, workspace); dz is
    None without a gate, dweight None without a weight."""
    torch = _torch()
    dev = _device_of(x)
    if not _here(torch, dev, stream):
        return _there(torch, dev, stream, gated_norm_bwd, dy, x, z, weight, gate=gate, eps=eps,
                      output_dweight=output_dweight, dx=dx, dz=dz, dweight=dweight, workspace=workspace)
    code, io, dtype, shape, f32 = _gate_code(gate, z), _dtype_code(x), x.dtype, x.shape, torch.float32
    tokens, H, d = _heads(shape)
    dp, ld_dy = _rows(dy, shape, dtype, "dy", dev, 2)
    xp, ld_x = _rows(x, shape, dtype, "x", dev, 2)
    zp, ld_z = (None, 0) if z is None else _rows(z, shape, dtype, "z", dev, 2)
    if dx is None:
        dx = _like(torch, x)
    if z is None:
        dz = None
    elif dz is None:
        dz = _like(torch, x)
    if weight is None:
        dweight = None
    elif dweight is None and output_dweight:
        dweight = torch.empty(d, dtype=f32, device=x.device)
    L, wp, have = lib(), None, 0
    if dweight is not None:
        need = L.kda_gated_norm_bwd_workspace_size(d)
        if workspace is None or workspace.numel() < need:
            workspace = _alloc_workspace(need, x.device)
        wp, have = _bytes(workspace, "workspace", dev)
    _done(L.kda_gated_norm_bwd(
        dp, ld_dy, xp, ld_x, zp, ld_z, _dense(weight, (d,), f32, "weight", dev),
        _dense(dx, shape, dtype, "dx", dev), _dense(dz, shape, dtype, "dz", dev),
        _dense(dweight, (d,), f32, "dweight", dev), tokens, H, d, eps, code, io, wp, have,
        _raw_stream(torch, dev)), "kda_gated_norm_bwd")
    return dx, dz, dweight, workspace


def _width(shape):
    if len(shape) < 1:
        raise ValueError("the residual must be [..., D]")
    rows = 1
    for n in shape[:-1]:
        rows *= n
    return rows, shape[-1]


def add_norm_fwd(residual, y, weight=None, scale=None, *, eps: float = 1e-6, residual_out=None,
                 n=None, stream=None):
    """Residual add and RMS norm: residual_out = residual + scale * y, and
    n = residual_out / rms(residual_out) * weight.  residual [...,D] (bf16, or
    fp32 with either activation type), y [...,D]; scale, weight fp32 [D] or None.
    ``residual_out`` may be ``residual`` itself.  Returns (residual_out, n)."""
    torch = _torch()
    dev = _device_of(residual)
    if not _here(torch, dev, stream):
        return _there(torch, dev, stream, add_norm_fwd, residual, y, weight, scale, eps=eps,
                      residual_out=residual_out, n=n)
    shape, f32 = residual.shape, torch.float32
    rows, D = _width(shape)
    res, io = _dtype_code(residual), _dtype_code(y)
    if residual_out is None:
        residual_out = _like(torch, residual)
    if n is None:
        n = _like(torch, y)
    _done(lib().kda_add_norm_fwd(
        _dense(residual, shape, residual.dtype, "residual", dev), _dense(y, shape, y.dtype, "y", dev),
        _dense(scale, (D,), f32, "scale", dev), _dense(weight, (D,), f32, "weight", dev),
        _dense(residual_out, shape, residual.dtype, "residual_out", dev),
        _dense(n, shape, y.dtype, "n", dev), rows, D, eps, res, io,
        _raw_stream(torch, dev)), "kda_add_norm_fwd")
    return residual_out, n


def add_norm_bwd(dn, dresidual_out, residual_out, y=None, weight=None, scale=None, *,
                 eps: float = 1e-6, dresidual=None, dy=None, dscale=None, dweight=None,
                 workspace=None, stream=None):
    """Gradients of add_norm_fwd from those of both outputs (dresidual_out None:
    zeros) and the residual_out it wrote; ``y`` is needed with a scale.  Returns
    (dresidual, dy, dweight, dscale, workspace).  Without a scale and with one
    type dy IS dresidual, the same tensor; dweight (dscale) is None without a
    weight (a scale)."""
    torch = _torch()
    dev = _device_of(residual_out)
    if not _here(torch, dev, stream):
        return _there(torch, dev, stream, add_norm_bwd, dn, dresidual_out, residual_out, y, weight,
                      scale, eps=eps, dresidual=dresidual, dy=dy, dscale=dscale, dweight=dweight,
                      workspace=workspace)
    shape, f32, where = residual_out.shape, torch.float32, residual_out.device
    rows, D = _width(shape)
    res, io, dtype, rdtype = _dtype_code(residual_out), _dtype_code(dn), dn.dtype, residual_out.dtype
    if scale is not None and y is None:
        raise ValueError("the gradient of scale needs y")
    if dresidual is None:
        dresidual = _like(torch, residual_out)
    shared = dy is None and scale is None and dtype == rdtype
    if dy is None and not shared:
        dy = _like(torch, dn)
    if weight is None:
        dweight = None
    elif dweight is None:
        dweight = torch.empty(D, dtype=f32, device=where)
    if scale is None:
        dscale = None
    elif dscale is None:
        dscale = torch.empty(D, dtype=f32, device=where)
    L, wp, have = lib(), None, 0
    if dweight is not None or dscale is not None:
        need = L.kda_add_norm_bwd_workspace_size(D)
        if workspace is None or workspace.numel() < need:
            workspace = _alloc_workspace(need, where)
        wp, have = _bytes(workspace, "workspace", dev)
    _done(L.kda_add_norm_bwd(
        _dense(dn, shape, dtype, "dn", dev), _dense(dresidual_out, shape, rdtype, "dresidual_out", dev),
        _dense(residual_out, shape, rdtype, "residual_out", dev),
        _dense(y, shape, dtype, "y", dev) if scale is not None else None,
        _dense(scale, (D,), f32, "scale", dev), _dense(weight, (D,), f32, "weight", dev),
        _dense(dresidual, shape, rdtype, "dresidual", dev), _dense(dy, shape, dtype, "dy", dev),
        _dense(dscale, (D,), f32, "dscale", dev), _dense(dweight, (D,), f32, "dweight", dev), rows, D,
        eps, res, io, wp, have, _raw_stream(torch, dev)), "kda_add_norm_bwd")
    return dresidual, dresidual if shared else dy, dweight, dscale, workspace


def trace_enable(on: bool = True) -> None:
    """Record the device time of every library kernel launch (off by default)."""
    lib().kda_trace_enable(1 if on else 0)


def trace_read(capacity: int = 4096):
    """Wait for the traced launches; return [(kernel name, ms), ...] and clear."""
    L = lib()
    stride = 64
    names = ctypes.create_string_buffer(stride * capacity)
    ms = (ctypes.c_float * capacity)()
    n = L.kda_trace_read(names, stride, ms, capacity)
    return [(names.raw[i * stride:(i + 1) * stride].split(b"\0", 1)[0].decode(), float(ms[i]))
            for i in range(n)]


def selftest_wait_timeout(workspace, max_polls: int = 16, stream=None) -> None:
    """Run one bounded on-device wait that nothing completes; it expires and
    writes KDA_DEVICE_TIMEOUT into ``workspace``'s status word (read it with
    check_device_status).  Exercises the library's expired-wait path without
    faulting or hanging the GPU."""
    L = lib()
    _check(L.kda_selftest_wait_timeout(_ptr(workspace), int(max_polls),
                                       _stream_handle(stream, workspace.device)),
           "kda_selftest_wait_timeout")


def check_device_status(workspace, stream=None) -> Tuple[int, int]:
    """Synchronise ``stream`` and read the device status word of a prefill
    workspace.  Returns (status, device_code); raises on KDA_ERR_CUDA."""
    L = lib()
    code = ctypes.c_int32(0)
    st = L.kda_check_device_status(_ptr(workspace), _stream_handle(stream, workspace.device),
                                   ctypes.byref(code))
    if st == KDA_ERR_CUDA:
        _check(st, "kda_check_device_status")
    return st, code.value
