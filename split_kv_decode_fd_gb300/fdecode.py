"""ctypes binding of libfdecode (include/fdecode.h), taking PyTorch tensors.

Argument marshalling only: every step of the decode runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
CPU fallback: calls with CPU tensors raise, and a missing library raises.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
import threading
from typing import Optional, Sequence

import numpy as np

__all__ = [
    "FdError", "KvDesc", "library_path", "load_library", "workspace_bytes", "split_size", "plan_pieces",
    "Workspace", "decode", "decode_rows", "append_decode", "prefill", "attend", "attend_backend", "decode_host", "HostDecoder", "decode_static", "static_status", "split_partial", "combine", "workspace_status",
    "NewRows", "Kv4Desc", "append_rope", "append_rope_kv4", "kv4_block_bytes", "kv4_cache", "kv4_read", "decode_kv4",
]

FD_OK, FD_ERR_INVALID_ARG, FD_ERR_UNSUPPORTED, FD_ERR_WORKSPACE_TOO_SMALL = 0, 1, 2, 3
FD_ERR_BAD_INDEX, FD_ERR_CUDA, FD_ERR_TIMEOUT = 4, 5, 6
FD_F32, FD_BF16 = 0, 1
FD_KV_CONTIGUOUS, FD_KV_PAGED = 0, 1
FD_SPLITS_AUTO = 0
FD_AUTO_MAX_BATCH = 1024

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None
_LOCK = threading.Lock()


class FdError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib().fd_status_string(status).decode() if _LIB is not None else str(status)
        super().__init__(f"{where}: {msg} (status {status})")


class KvDesc(ctypes.Structure):
    _fields_ = [
        ("layout", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("capacity", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("max_pages_per_seq", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
    ]


class NewRows(ctypes.Structure):
    """``fd_new_rows``: the rows an append brings."""

    _fields_ = [
        ("dtype", ctypes.c_int),
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64 * 3),
        ("k_stride", ctypes.c_int64 * 3),
        ("v_stride", ctypes.c_int64 * 3),
        ("new_lens", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
        ("cos", ctypes.c_void_p),
        ("sin", ctypes.c_void_p),
        ("max_pos", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
    ]


class Kv4Desc(ctypes.Structure):
    """``fd_kv4_desc``: a 4-bit cache."""

    _fields_ = [
        ("layout", ctypes.c_int),
        ("kv", ctypes.c_void_p),
        ("capacity", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("max_pages_per_seq", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("k_exp", ctypes.c_int32),
        ("v_exp", ctypes.c_int32),
    ]


def library_path() -> str:
    return os.environ.get("FDECODE_LIB", os.path.join(_HERE, "libfdecode.so"))


def load_library(path: Optional[str] = None):
    """Load libfdecode.so (built in-tree by ``split_kv_decode_fd_gb300/build.py``)."""
    global _LIB
    with _LOCK:
        if _LIB is not None:
            return _LIB
        path = path or library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libfdecode.so not found at {path}; build it with "
                               "`python split_kv_decode_fd_gb300/build.py`")
        lib = ctypes.CDLL(path)
        c_i32, c_i64, c_sz, vp, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
        kvp, kv4p = ctypes.POINTER(KvDesc), ctypes.POINTER(Kv4Desc)
        sig = {
            "fd_workspace_bytes": (c_sz, [c_i32, c_i32, c_i32, c_i32, c_i32, c_i32]),
            "fd_workspace_init": (ctypes.c_int, [vp, c_sz, vp]),
            "fd_workspace_status": (ctypes.c_int, [vp, c_sz, vp]),
            "fd_split_size": (c_i32, [c_i32, c_i32]),
            "fd_decode": (ctypes.c_int, [vp, kvp, vp, vp, c_i32, c_i32, c_i32, vp, c_i32, c_i32, f32, c_i32, vp,
                                         c_sz, vp]),
            "fd_split_partial": (ctypes.c_int, [vp, kvp, c_i32, c_i32, c_i32, vp, c_i32, c_i32, f32, c_i32, vp,
                                                vp, vp, vp]),
            "fd_combine": (ctypes.c_int, [vp, vp, vp, vp, vp, c_i32, c_i32, c_i32, c_i32, vp]),
            "fd_decode_host": (ctypes.c_int, [vp, kvp, vp, vp, c_i32, c_i32, c_i32, vp, c_i32, c_i32, f32, c_i32,
                                              vp, c_sz, vp]),
            "fd_plan_pieces": (c_i64, [c_i32, c_i32, c_i32, c_i32, vp, c_i32, c_i32, c_i32, vp, c_i64]),
            "fd_decode_static": (ctypes.c_int, [vp, kvp, vp, vp, c_i32, c_i32, c_i32, vp, c_i32, c_i32, f32,
                                                c_i32, vp]),
            "fd_static_status": (ctypes.c_int, [vp]),
            "fd_decode_rows": (ctypes.c_int, [vp, c_i32, c_i32, kvp, vp, vp, c_i32, c_i32, c_i32, vp, c_i32,
                                              c_i32, f32, c_i32, vp, c_sz, vp]),
            "fd_append_decode": (ctypes.c_int, [vp, vp, vp, kvp, vp, vp, c_i32, c_i32, c_i32, vp, c_i32, c_i32, f32,
                                                c_i32, vp, c_sz, vp]),
            "fd_prefill": (ctypes.c_int, [vp, c_i32, c_i32, kvp, vp, vp, c_i32, c_i32, c_i32, vp, c_i32, c_i32, f32,
                                          vp, c_sz, vp]),
            "fd_attend": (ctypes.c_int, [vp, c_i32, c_i32, kvp, vp, vp, c_i32, c_i32, c_i32, vp, c_i32, c_i32, f32,
                                         c_i32, vp, c_sz, vp, ctypes.POINTER(c_i32)]),
            "fd_attend_backend": (c_i32, [c_i32, c_i32, c_i32, c_i32, c_i32]),
            "fd_backend_name": (ctypes.c_char_p, [c_i32]),
            "fd_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "fd_version": (c_i32, []),
            "fd_debug_stall": (None, [c_i32, c_i64]),
            "fd_kv4_block_bytes": (c_i32, [c_i32]),
            "fd_append_rope": (ctypes.c_int, [ctypes.POINTER(NewRows), kvp, vp, c_i32, c_i32, c_i32, c_i32, vp, c_i32,
                                              c_i32, vp, c_sz, vp]),
            "fd_append_rope_kv4": (ctypes.c_int, [ctypes.POINTER(NewRows), kv4p, vp, c_i32, c_i32, c_i32, c_i32, vp,
                                                  c_i32, c_i32, vp, c_sz, vp]),
            "fd_kv4_read": (ctypes.c_int, [kv4p, vp, vp, ctypes.c_int, c_i32, c_i32, c_i32, vp, vp, c_i32, c_i32, vp,
                                           c_sz, vp]),
            "fd_decode_kv4": (ctypes.c_int, [vp, c_i32, c_i32, kv4p, vp, vp, c_i32, c_i32, c_i32, vp, c_i32, c_i32,
                                             f32, c_i32, vp, c_sz, vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
        return lib


def _lib():
    return load_library()


def _check(status: int, where: str):
    if status != FD_OK:
        raise FdError(status, where)


# ------------------------------------------------------------------ host-only
def workspace_bytes(B, Hq, Hkv, D, n_splits=FD_SPLITS_AUTO, num_sms=0) -> int:
    n = _lib().fd_workspace_bytes(B, Hq, Hkv, D, n_splits, num_sms)
    if n == 0:
        raise FdError(FD_ERR_INVALID_ARG, "fd_workspace_bytes")
    return int(n)


def split_size(max_seq_len: int, n_splits: int) -> int:
    return int(_lib().fd_split_size(max_seq_len, n_splits))


def plan_pieces(B, Hq, Hkv, seq_lens: Optional[Sequence[int]], max_seq_len, n_splits=0, grid=152,
                kv_dtype="bf16") -> np.ndarray:
    """The pieces fd_decode runs: int32 [n, 7] of (cta, b, vkv, tok_begin, tok_end, slot, pieces_of_sequence)."""
    lib = _lib()
    dt = {"bf16": FD_BF16, "f32": FD_F32}[kv_dtype]
    lens = None if seq_lens is None else np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
    lp = None if lens is None else lens.ctypes.data
    n = lib.fd_plan_pieces(B, Hq, Hkv, dt, lp, max_seq_len, n_splits, grid, None, 0)
    if n < 0:
        raise FdError(FD_ERR_INVALID_ARG, "fd_plan_pieces")
    buf = np.zeros((max(n, 1), 7), dtype=np.int32)
    lib.fd_plan_pieces(B, Hq, Hkv, dt, lp, max_seq_len, n_splits, grid, buf.ctypes.data, n)
    return buf[:n]


# ------------------------------------------------------------------ device
_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream_handle(device, stream=None) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return int(s.cuda_stream)


def _need_cuda(t, name, dtype=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libfdecode has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _kv_desc(k, v, block_table):
    torch = _torch()
    _need_cuda(k, "k")
    _need_cuda(v, "v")
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have the same dtype and shape")
    dt = {torch.bfloat16: FD_BF16, torch.float32: FD_F32}.get(k.dtype)
    if dt is None:
        raise ValueError(f"unsupported KV dtype {k.dtype}")
    d = KvDesc()
    d.dtype = dt
    d.k = k.data_ptr()
    d.v = v.data_ptr()
    if block_table is None:
        d.layout = FD_KV_CONTIGUOUS
        d.capacity = k.shape[2]
    else:
        _need_cuda(block_table, "block_table", torch.int32)
        d.layout = FD_KV_PAGED
        d.block_table = block_table.data_ptr()
        d.max_pages_per_seq = block_table.shape[1]
        d.page_size = k.shape[2]
        d.num_pages = k.shape[0]
    return d


class Workspace:
    """Zero-initialised device scratch for the kernels, grown on demand.

    It holds the error word, the decode kernels' arrival counters and partial
    states, and the prefill's item queue, all left at zero between calls: calls
    that may run at the same time (on different streams) need a Workspace each.
    The default one, used when none is passed, is shared per device; append_rope,
    append_rope_kv4, kv4_read and decode_kv4 have one per stream.  A graph captured without a
    Workspace takes the newest of these that is large enough, or else the device's: pass one to
    a graph that is replayed beside other calls.

    A buffer that has been outgrown stays allocated as long as the Workspace does: a graph
    captured with it holds its address.  Each is at least twice as large as the one before, so
    together they take no more than twice the last one's bytes.
    """

    def __init__(self, device=None):
        self.device = device
        self.buf = None
        self._outgrown = []
        self._streams = set()  # handles of the streams that the caching allocator knows to use buf

    def get(self, nbytes: int, device):
        if self.buf is None or self.buf.numel() < nbytes or self.buf.device != device:
            self._replace(nbytes, device)
        return self.buf

    def _replace(self, nbytes, device):
        device = _torch().empty(0, dtype=_torch().uint8, device=device).device  # "cuda" has an index from here on
        old = self._outgrown + ([] if self.buf is None else [self.buf])
        here = [b for b in old if b.device == device]
        buf = next((b for b in here if b.numel() >= nbytes), None)
        if buf is None:
            least = max([128] + [b.numel() for b in here])
            buf = _torch().zeros(max(nbytes, 2 * least), dtype=_torch().uint8, device=device)
        self._outgrown = [b for b in old if b is not buf]
        self.buf = buf
        self._streams = set()


_DEFAULT_WS = {}


def _default_workspace(device) -> Workspace:
    key = (device.type, device.index)
    if key not in _DEFAULT_WS:
        _DEFAULT_WS[key] = Workspace(device)
    return _DEFAULT_WS[key]


def _geometry(q, k, block_table, seq_lens, max_seq_len):
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    if k.shape[3] != D:
        raise ValueError("head_dim of q and k differ")
    if max_seq_len is None:
        max_seq_len = k.shape[2] if block_table is None else block_table.shape[1] * k.shape[2]
    return B, Hq, Hkv, D, int(max_seq_len)


def decode(q, k, v, *, seq_lens=None, max_seq_len=None, block_table=None, scale=None, n_splits=FD_SPLITS_AUTO,
           out=None, lse=None, return_lse=True, workspace: Optional[Workspace] = None, stream=None):
    """Split-KV decode attention (``fd_decode``).

    q ``[B, Hq, D]`` fp32 CUDA; k, v contiguous ``[B, Hkv, T_cap, D]`` or, with
    ``block_table`` ``[B, max_pages]`` int32, paged ``[num_pages, Hkv, page, D]``
    (bf16 or fp32).  Returns ``(out [B, Hq, D], lse [B, Hq] or None)``.
    """
    torch = _torch()
    _need_cuda(q, "q", torch.float32)
    kv = _kv_desc(k, v, block_table)
    B, Hq, Hkv, D, max_seq_len = _geometry(q, k, block_table, seq_lens, max_seq_len)
    if seq_lens is not None:
        _need_cuda(seq_lens, "seq_lens", torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    _need_cuda(out, "out", torch.float32)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    ws = workspace or _default_workspace(q.device)
    nbytes = workspace_bytes(B, Hq, Hkv, D, n_splits)
    buf = ws.get(nbytes, q.device)
    st = _lib().fd_decode(q.data_ptr(), ctypes.byref(kv), out.data_ptr(), lse.data_ptr() if lse is not None else None,
                          B, Hq, Hkv, seq_lens.data_ptr() if seq_lens is not None else None, max_seq_len, D,
                          float(scale), int(n_splits), buf.data_ptr(), buf.numel(), _stream_handle(q.device, stream))
    _check(st, "fd_decode")
    return out, lse


def decode_rows(q, k, v, *, causal=True, seq_lens=None, max_seq_len=None, block_table=None, scale=None,
                n_splits=FD_SPLITS_AUTO, out=None, lse=None, return_lse=True, workspace: Optional[Workspace] = None,
                stream=None):
    """``fd_decode_rows``: q ``[B, Hq, n_q, D]`` (n_q query rows per head); returns
    ``(out [B, Hq, n_q, D], lse [B, Hq, n_q] or None)``.  With ``causal`` row i sees
    keys ``t < L_b - (n_q - 1 - i)``.
    """
    torch = _torch()
    _need_cuda(q, "q", torch.float32)
    if q.dim() != 4:
        raise ValueError("q must be [B, Hq, n_q, D]")
    kv = _kv_desc(k, v, block_table)
    B, Hq, n_q, D = q.shape
    Hkv = k.shape[1]
    if max_seq_len is None:
        max_seq_len = k.shape[2] if block_table is None else block_table.shape[1] * k.shape[2]
    if seq_lens is not None:
        _need_cuda(seq_lens, "seq_lens", torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, Hq, n_q, D), dtype=torch.float32, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, n_q), dtype=torch.float32, device=q.device)
    ws = workspace or _default_workspace(q.device)
    buf = ws.get(workspace_bytes(B, Hq * n_q, Hkv, D, n_splits), q.device)
    st = _lib().fd_decode_rows(q.data_ptr(), int(n_q), int(bool(causal)), ctypes.byref(kv), out.data_ptr(),
                               lse.data_ptr() if lse is not None else None, B, Hq, Hkv,
                               seq_lens.data_ptr() if seq_lens is not None else None, int(max_seq_len), D,
                               float(scale), int(n_splits), buf.data_ptr(), buf.numel(),
                               _stream_handle(q.device, stream))
    _check(st, "fd_decode_rows")
    return out, lse


def append_decode(q, k, v, k_new, v_new, *, seq_lens=None, max_seq_len=None, block_table=None, scale=None,
                  n_splits=FD_SPLITS_AUTO, out=None, lse=None, return_lse=True,
                  workspace: Optional[Workspace] = None, stream=None):
    """``fd_append_decode``: write ``k_new``/``v_new`` (``[B, Hkv, D]``, cache dtype) at
    position ``L_b`` of every sequence, then decode over ``L_b + 1`` keys.

    ``seq_lens``/``max_seq_len`` are the lengths before the append (default
    ``max_seq_len``: the cache capacity minus one).  ``k`` and ``v`` are written.
    Returns ``(out, lse)``.
    """
    torch = _torch()
    _need_cuda(q, "q", torch.float32)
    kv = _kv_desc(k, v, block_table)
    _need_cuda(k_new, "k_new", k.dtype)
    _need_cuda(v_new, "v_new", k.dtype)
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    if tuple(k_new.shape) != (B, Hkv, D) or tuple(v_new.shape) != (B, Hkv, D):
        raise ValueError("k_new and v_new must be [B, Hkv, D]")
    if max_seq_len is None:
        cap = k.shape[2] if block_table is None else block_table.shape[1] * k.shape[2]
        max_seq_len = cap - 1
    if seq_lens is not None:
        _need_cuda(seq_lens, "seq_lens", torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    ws = workspace or _default_workspace(q.device)
    buf = ws.get(workspace_bytes(B, Hq, Hkv, D, n_splits), q.device)
    st = _lib().fd_append_decode(q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), ctypes.byref(kv), out.data_ptr(),
                                 lse.data_ptr() if lse is not None else None, B, Hq, Hkv,
                                 seq_lens.data_ptr() if seq_lens is not None else None, int(max_seq_len), D,
                                 float(scale), int(n_splits), buf.data_ptr(), buf.numel(),
                                 _stream_handle(q.device, stream))
    _check(st, "fd_append_decode")
    return out, lse


def _rows_args(q, k, v, block_table, seq_lens, max_seq_len, scale, out, lse, return_lse):
    torch = _torch()
    _need_cuda(q, "q", torch.float32)
    if q.dim() != 4:
        raise ValueError("q must be [B, Hq, n_q, D]")
    kv = _kv_desc(k, v, block_table)
    B, Hq, n_q, D = q.shape
    if max_seq_len is None:
        max_seq_len = k.shape[2] if block_table is None else block_table.shape[1] * k.shape[2]
    if seq_lens is not None:
        _need_cuda(seq_lens, "seq_lens", torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, Hq, n_q, D), dtype=torch.float32, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, n_q), dtype=torch.float32, device=q.device)
    return kv, B, Hq, n_q, D, max_seq_len, scale, out, lse


def prefill(q, k, v, *, causal=True, seq_lens=None, max_seq_len=None, block_table=None, scale=None, out=None,
            lse=None, return_lse=True, workspace: Optional[Workspace] = None, stream=None):
    """``fd_prefill``: the ``decode_rows`` operation for long windows, on tcgen05 query tiles."""
    kv, B, Hq, n_q, D, max_seq_len, scale, out, lse = _rows_args(q, k, v, block_table, seq_lens, max_seq_len,
                                                                scale, out, lse, return_lse)
    ws = workspace or _default_workspace(q.device)
    buf = ws.get(256, q.device)
    st = _lib().fd_prefill(q.data_ptr(), int(n_q), int(bool(causal)), ctypes.byref(kv), out.data_ptr(),
                           lse.data_ptr() if lse is not None else None, B, Hq, k.shape[1],
                           seq_lens.data_ptr() if seq_lens is not None else None, int(max_seq_len), D, float(scale),
                           buf.data_ptr(), buf.numel(), _stream_handle(q.device, stream))
    _check(st, "fd_prefill")
    return out, lse


def attend_backend(n_q, Hq, Hkv, D, kv_dtype="bf16") -> str:
    """Name of the backend ``attend`` would run (``fd_attend_backend``)."""
    dt = {"bf16": FD_BF16, "f32": FD_F32}[kv_dtype]
    return _lib().fd_backend_name(_lib().fd_attend_backend(int(n_q), int(Hq), int(Hkv), int(D), dt)).decode()


def attend(q, k, v, *, causal=True, seq_lens=None, max_seq_len=None, block_table=None, scale=None,
           n_splits=FD_SPLITS_AUTO, out=None, lse=None, return_lse=True, workspace: Optional[Workspace] = None,
           stream=None):
    """``fd_attend``: phase dispatch for q ``[B, Hq, n_q, D]``; returns ``(out, lse, backend name)``."""
    kv, B, Hq, n_q, D, max_seq_len, scale, out, lse = _rows_args(q, k, v, block_table, seq_lens, max_seq_len,
                                                                scale, out, lse, return_lse)
    Hkv = k.shape[1]
    lib = _lib()
    be = lib.fd_attend_backend(int(n_q), Hq, Hkv, D, kv.dtype)
    need = 256 if be == 2 else workspace_bytes(B, Hq * n_q, Hkv, D, n_splits)
    ws = workspace or _default_workspace(q.device)
    buf = ws.get(need, q.device)
    chosen = ctypes.c_int32(-1)
    st = lib.fd_attend(q.data_ptr(), int(n_q), int(bool(causal)), ctypes.byref(kv), out.data_ptr(),
                       lse.data_ptr() if lse is not None else None, B, Hq, Hkv,
                       seq_lens.data_ptr() if seq_lens is not None else None, int(max_seq_len), D, float(scale),
                       int(n_splits), buf.data_ptr(), buf.numel(), _stream_handle(q.device, stream),
                       ctypes.byref(chosen))
    _check(st, "fd_attend")
    return out, lse, lib.fd_backend_name(chosen.value).decode()


def decode_static(q, k, v, *, out, lse=None, seq_lens=None, max_seq_len=None, block_table=None, scale=None,
                  n_splits=FD_SPLITS_AUTO, stream=None):
    """``fd_decode_static``: fd_decode for callers that may not allocate device memory.

    The caller passes every buffer (``out`` is required; ``lse`` optional); the
    library's scratch is a fixed device array inside libfdecode, shared by all
    calls, so calls must not overlap on the GPU.  Nothing is allocated here.
    """
    torch = _torch()
    _need_cuda(q, "q", torch.float32)
    _need_cuda(out, "out", torch.float32)
    kv = _kv_desc(k, v, block_table)
    B, Hq, Hkv, D, max_seq_len = _geometry(q, k, block_table, seq_lens, max_seq_len)
    if seq_lens is not None:
        _need_cuda(seq_lens, "seq_lens", torch.int32)
    if lse is not None:
        _need_cuda(lse, "lse", torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    st = _lib().fd_decode_static(q.data_ptr(), ctypes.byref(kv), out.data_ptr(),
                                 lse.data_ptr() if lse is not None else None, B, Hq, Hkv,
                                 seq_lens.data_ptr() if seq_lens is not None else None, max_seq_len, D,
                                 float(scale), int(n_splits), _stream_handle(q.device, stream))
    _check(st, "fd_decode_static")
    return out, lse


def static_status(device=None, stream=None) -> int:
    """``fd_static_status``: synchronise and return (then clear) the error word of the
    static scratch array that ``decode_static`` uses (0 = no error)."""
    torch = _torch()
    device = device or torch.device("cuda", torch.cuda.current_device())
    return int(_lib().fd_static_status(_stream_handle(device, stream)))


def decode_host(q_host, k, v, *, seq_lens_host=None, max_seq_len=None, block_table=None, scale=None,
                n_splits=FD_SPLITS_AUTO, out_host=None, lse_host=None, workspace: Optional[Workspace] = None,
                stream=None):
    """``fd_decode_host``: q, seq_lens and the outputs in (pinned) host memory; synchronous."""
    torch = _torch()
    if q_host.is_cuda or q_host.dtype != torch.float32 or not q_host.is_contiguous():
        raise ValueError("q_host must be a contiguous fp32 CPU tensor")
    kv = _kv_desc(k, v, block_table)
    B, Hq, Hkv, D, max_seq_len = _geometry(q_host, k, block_table, seq_lens_host, max_seq_len)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out_host is None:
        out_host = torch.empty((B, Hq, D), dtype=torch.float32, pin_memory=True)
    if lse_host is None:
        lse_host = torch.empty((B, Hq), dtype=torch.float32, pin_memory=True)
    if seq_lens_host is not None and (seq_lens_host.is_cuda or seq_lens_host.dtype != torch.int32):
        raise ValueError("seq_lens_host must be an int32 CPU tensor")
    ws = workspace or _default_workspace(k.device)
    nbytes = workspace_bytes(B, Hq, Hkv, D, n_splits)
    buf = ws.get(nbytes, k.device)
    st = _lib().fd_decode_host(q_host.data_ptr(), ctypes.byref(kv), out_host.data_ptr(), lse_host.data_ptr(),
                               B, Hq, Hkv, seq_lens_host.data_ptr() if seq_lens_host is not None else None,
                               max_seq_len, D, float(scale), int(n_splits), buf.data_ptr(), buf.numel(),
                               _stream_handle(k.device, stream))
    _check(st, "fd_decode_host")
    return out_host, lse_host


class HostDecoder:
    """``fd_decode_host`` with its arguments marshalled once, for a decode loop
    that passes the same host buffers and KV cache every step.

    ``q_host`` ``[B, Hq, D]`` fp32, ``out_host`` ``[B, Hq, D]`` and ``lse_host``
    ``[B, Hq]`` (optional), ``seq_lens_host`` ``[B]`` int32 (optional) are CPU
    tensors whose contents the caller rewrites between steps; pinned buffers
    (``pin_memory=True``) are read and written by the kernels in place, over the
    host link, and pageable ones are copied through the workspace.  Calling the
    object runs one synchronous step and returns ``(out_host, lse_host)``.
    """

    def __init__(self, q_host, k, v, *, out_host=None, lse_host=None, seq_lens_host=None, max_seq_len=None,
                 block_table=None, scale=None, n_splits=FD_SPLITS_AUTO, workspace: Optional[Workspace] = None,
                 stream=None):
        torch = _torch()
        if q_host.is_cuda or q_host.dtype != torch.float32 or not q_host.is_contiguous():
            raise ValueError("q_host must be a contiguous fp32 CPU tensor")
        self._kv = _kv_desc(k, v, block_table)
        B, Hq, Hkv, D, max_seq_len = _geometry(q_host, k, block_table, seq_lens_host, max_seq_len)
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        if out_host is None:
            out_host = torch.empty((B, Hq, D), dtype=torch.float32, pin_memory=True)
        for t, name, shape, dt in ((out_host, "out_host", (B, Hq, D), torch.float32),
                                   (lse_host, "lse_host", (B, Hq), torch.float32),
                                   (seq_lens_host, "seq_lens_host", (B,), torch.int32)):
            if t is not None and (t.is_cuda or t.dtype != dt or not t.is_contiguous() or tuple(t.shape) != shape):
                raise ValueError(f"{name} must be a contiguous {dt} CPU tensor of shape {shape}")
        ws = workspace or _default_workspace(k.device)
        buf = ws.get(workspace_bytes(B, Hq, Hkv, D, n_splits), k.device)
        self.q_host, self.out_host, self.lse_host, self.seq_lens_host = q_host, out_host, lse_host, seq_lens_host
        self._keep = (k, v, block_table, buf)
        vp, i32 = ctypes.c_void_p, ctypes.c_int32
        self._fn = _lib().fd_decode_host
        self._args = (vp(q_host.data_ptr()), ctypes.byref(self._kv), vp(out_host.data_ptr()),
                      vp(lse_host.data_ptr() if lse_host is not None else None), i32(B), i32(Hq), i32(Hkv),
                      vp(seq_lens_host.data_ptr() if seq_lens_host is not None else None), i32(max_seq_len), i32(D),
                      ctypes.c_float(scale), i32(int(n_splits)), vp(buf.data_ptr()), ctypes.c_size_t(buf.numel()),
                      vp(_stream_handle(k.device, stream)))

    def __call__(self):
        st = self._fn(*self._args)
        if st != FD_OK:
            raise FdError(st, "fd_decode_host")
        return self.out_host, self.lse_host


def split_partial(q, k, v, n_splits: int, *, seq_lens=None, max_seq_len=None, block_table=None, scale=None,
                  stream=None):
    """``fd_split_partial``: returns ``(o_part [B,Hq,n,D], m_part [B,Hq,n], l_part [B,Hq,n])``."""
    torch = _torch()
    _need_cuda(q, "q", torch.float32)
    kv = _kv_desc(k, v, block_table)
    B, Hq, Hkv, D, max_seq_len = _geometry(q, k, block_table, seq_lens, max_seq_len)
    if seq_lens is not None:
        _need_cuda(seq_lens, "seq_lens", torch.int32)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    o = torch.empty((B, Hq, n_splits, D), dtype=torch.float32, device=q.device)
    m = torch.empty((B, Hq, n_splits), dtype=torch.float32, device=q.device)
    l = torch.empty((B, Hq, n_splits), dtype=torch.float32, device=q.device)
    st = _lib().fd_split_partial(q.data_ptr(), ctypes.byref(kv), B, Hq, Hkv,
                                 seq_lens.data_ptr() if seq_lens is not None else None, max_seq_len, D, float(scale),
                                 int(n_splits), o.data_ptr(), m.data_ptr(), l.data_ptr(),
                                 _stream_handle(q.device, stream))
    _check(st, "fd_split_partial")
    return o, m, l


def combine(o_part, m_part, l_part, *, out=None, lse=None, return_lse=True, stream=None):
    """``fd_combine`` over partials in the ``fd_split_partial`` layout."""
    torch = _torch()
    for t, n in ((o_part, "o_part"), (m_part, "m_part"), (l_part, "l_part")):
        _need_cuda(t, n, torch.float32)
    B, Hq, n_splits, D = o_part.shape
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=o_part.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=o_part.device)
    st = _lib().fd_combine(o_part.data_ptr(), m_part.data_ptr(), l_part.data_ptr(), out.data_ptr(),
                           lse.data_ptr() if lse is not None else None, B, Hq, D, n_splits,
                           _stream_handle(o_part.device, stream))
    _check(st, "fd_combine")
    return out, lse


def workspace_status(workspace: Optional[Workspace] = None, device=None, stream=None) -> int:
    """Synchronise and return (then clear) the kernels' error word of a workspace (0 = no error).

    Errors that calls, or replays of graphs captured with them, raised in a buffer that the workspace has outgrown count too.
    Without a workspace: the default ones of ``stream``, or of every stream of the device, which is then waited for.
    """
    torch = _torch()
    device = device or torch.device("cuda", torch.cuda.current_device())
    if workspace is not None:
        spaces = [workspace]
    else:
        index = torch.cuda.current_device() if device.index is None else device.index
        handle = _stream_handle(device, stream)
        own = [w for (i, h), w in list(_STREAM_WS.items()) if i == index and (stream is None or h == handle)]
        if stream is None and own:
            torch.cuda.synchronize(device)
        spaces = [_default_workspace(device)] + own
    return max([FD_OK] + [_word(ws, stream) for ws in spaces if ws.buf is not None])


def _word(ws, stream):
    handle = _stream_handle(ws.buf.device, stream)
    return max(int(_lib().fd_workspace_status(b.data_ptr(), b.numel(), handle))
               for b in [ws.buf] + ws._outgrown if b.device == ws.buf.device)


# ------------------------------------------------------------------ rotating append, 4-bit cache
#
# These calls take a few microseconds on the device, less than Python takes to ask a
# tensor a dozen questions: the checks use the cheap ones (get_device() is -1 off the
# GPU, dtypes are singletons), and structures are packed in one go.
_ROWS = struct.Struct("@i4x3P9q4P3i4x")
_KV = struct.Struct("@2i2PqP3i4x")
_KV4 = struct.Struct("@i4xPqP5i4x")
assert _ROWS.size == ctypes.sizeof(NewRows) and _KV.size == ctypes.sizeof(KvDesc) and _KV4.size == ctypes.sizeof(Kv4Desc)


def _flat(t, name, dtype, index, shape=None):
    """Pointer of a contiguous CUDA tensor of ``dtype`` on device ``index``."""
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libfdecode has no CPU path)")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _opt(t, name, dtype, index, shape=None):
    """Pointer of an optional tensor (see ``_flat``); 0 without one."""
    return 0 if t is None else _flat(t, name, dtype, index, shape)


def _i32(x, name):
    """x as the library's int32 (ctypes would keep the lowest 32 bits)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit in 32 bits, got {x}")
    return x


def _index_of(t, name):
    if not isinstance(t, _torch().Tensor) or t.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor (libfdecode has no CPU path)")
    return t.get_device()


def _made(make, shape, dtype, device, stream):
    """A tensor for a call on ``stream``, filled there: a fill on the current stream could come after the call."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with _torch().cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


_STREAM_WS = {}  # (device index, stream handle) -> Workspace


def _scratch(workspace, index, nbytes, stream=None):
    """The workspace's buffer, zero-filled on the call's stream, and the stream's handle."""
    torch = _torch()
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    ws = _STREAM_WS.get((index, handle)) if workspace is None else workspace
    buf = None if ws is None else ws.buf
    if buf is None or buf.numel() < nbytes or buf.get_device() != index:
        if stream is None:
            ws = _grown(ws, index, nbytes, handle)
        else:
            with torch.cuda.stream(stream):
                ws = _grown(ws, index, nbytes, handle)
        buf = ws.buf
    if handle not in ws._streams:
        # freed with the Workspace, the memory waits for what is still running there
        buf.record_stream(torch.cuda.current_stream(index) if stream is None else stream)
        ws._streams.add(handle)
    return buf, handle


def _grown(ws, index, nbytes, handle):
    """The Workspace with a larger buffer; the stream's own default if it is None.  No buffer is made during a stream
    capture: its first zero-fill would then run only with the graph."""
    torch = _torch()
    default = ws is None or ws is _STREAM_WS.get((index, handle))
    if torch.cuda.is_current_stream_capturing():
        spaces = [_default_workspace(torch.device("cuda", index))] if default else []
        spaces += [w for (i, _), w in list(_STREAM_WS.items()) if default and i == index]
        sized = [w for w in spaces if w.buf is not None and w.buf.numel() >= nbytes]
        if not sized:
            raise RuntimeError("the workspace is too small and cannot grow during a stream capture: run the call once "
                               "before the capture, or pass a Workspace that has been used at this size")
        return sized[-1]
    device = torch.device("cuda", index)
    with _LOCK:  # two host threads may call on one stream
        if ws is None:
            ws = _STREAM_WS.setdefault((index, handle), Workspace(device))
        ws.get(nbytes, device)
    return ws


@functools.lru_cache(maxsize=256)
def _decode_bytes(B, Hq, Hkv, D, n_splits, index):
    """``workspace_bytes`` on device ``index``."""
    with _torch().cuda.device(index):
        return workspace_bytes(B, Hq, Hkv, D, n_splits)


def _launch(index, handle, fn, where, *args):
    """Call ``fn(*args, handle)`` with device ``index`` current (the library launches on the current device)."""
    torch = _torch()
    if index == torch.cuda.current_device():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st != FD_OK:
        raise FdError(st, where)


def kv4_block_bytes(D: int) -> int:
    """Bytes of one block (sixteen tokens of one KV head) of a 4-bit cache."""
    n = int(_lib().fd_kv4_block_bytes(int(D)))
    if n == 0:
        raise FdError(FD_ERR_UNSUPPORTED, "fd_kv4_block_bytes")
    return n


def kv4_cache(n, Hkv, tokens, D, device="cuda"):
    """A zeroed 4-bit cache: uint8 ``[n, Hkv, tokens / 16, 18 * D]``.

    Contiguous caches hold ``n`` sequences of ``tokens`` tokens, paged ones ``n`` pages.
    """
    if tokens % 16:
        raise ValueError("tokens must be a multiple of 16")
    return _torch().zeros((n, Hkv, tokens // 16, kv4_block_bytes(D)), dtype=_torch().uint8, device=device)


def _table(block_table, B, index):
    """Pointer and row length of a block table of B sequences."""
    at = _flat(block_table, "block_table", _torch().int32, index)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must be [{B}, max_pages]")
    return at, block_table.shape[1]


def _kv4_desc(kv4, block_table, B, k_exp, v_exp):
    """Descriptor, Hkv, D, tokens per sequence and device index of a 4-bit cache tensor."""
    index = _index_of(kv4, "kv4")
    at = _flat(kv4, "kv4", _torch().uint8, index)
    if kv4.dim() != 4 or kv4.shape[3] not in (18 * 64, 18 * 128):
        raise ValueError("kv4 must be uint8 [n, Hkv, tokens / 16, 18 * D] with D = 64 or 128")
    n, Hkv, blocks, size = kv4.shape
    tokens = blocks * 16
    if block_table is None:
        if n != B:
            raise ValueError(f"a contiguous kv4 must hold {B} sequences, got {n}")
        d = _KV4.pack(FD_KV_CONTIGUOUS, at, tokens, 0, 0, 0, 0, int(k_exp), int(v_exp))
    else:
        table, pages = _table(block_table, B, index)
        d = _KV4.pack(FD_KV_PAGED, at, 0, table, pages, tokens, n, int(k_exp), int(v_exp))
        tokens *= pages
    return Kv4Desc.from_buffer_copy(d), Hkv, size // 18, tokens, index


def _head_rows(t, name, B, n, heads, D, index, dtype):
    """Strides of ``t`` [B, n, heads, D], whose channels are contiguous."""
    if not isinstance(t, _torch().Tensor) or t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{index}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != n or shape[3] != D:
        raise ValueError(f"{name} must be [{B}, {n}, heads, {D}], got {tuple(shape)}")
    if heads is not None and shape[2] != heads:
        raise ValueError(f"{name} must have the cache's {heads} heads, got {shape[2]}")
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    if (st[0] | st[1] | st[2]) & 7:  # the stride of a single entry may be anything
        st = tuple(s if size > 1 else 0 for s, size in zip(st, shape))
    return st


def _append(fn, where, desc, k_new, v_new, Hkv, D, tokens, index, cos, sin, q, q_out, rot_dim, interleaved, positions,
            new_lens, seq_lens, max_seq_len, workspace, stream):
    torch = _torch()
    B, n = k_new.shape[0], _i32(k_new.shape[1], "n of k_new")
    max_seq_len = _i32(tokens - n if max_seq_len is None else max_seq_len, "max_seq_len")
    dtype = k_new.dtype
    dt = FD_BF16 if dtype is torch.bfloat16 else FD_F32 if dtype is torch.float32 else -1
    if dt < 0:
        raise ValueError(f"unsupported dtype of the new rows {dtype}")
    ks = _head_rows(k_new, "k_new", B, n, Hkv, D, index, dtype)
    vs = _head_rows(v_new, "v_new", B, n, Hkv, D, index, dtype)
    Hq, qp, qo, qs = 0, 0, 0, (0, 0, 0)
    if q is not None:
        qs = _head_rows(q, "q", B, n, None, D, index, dtype)
        Hq, qp = q.shape[2], q.data_ptr()
        if q_out is None:
            # rows that new_lens or a bad position leaves out are not written: they start as zeros
            make = torch.empty if new_lens is None and positions is None else torch.zeros
            q_out = _made(make, (B, Hq, n, D), torch.float32, q.device, stream)
            qo = q_out.data_ptr()
        else:
            qo = _flat(q_out, "q_out", torch.float32, index, (B, Hq, n, D))
    elif q_out is not None:
        raise ValueError("q_out without q")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    cp = sp = max_pos = rot = 0
    if cos is not None:
        cp, sp = _flat(cos, "cos", torch.float32, index), _flat(sin, "sin", torch.float32, index)
        if cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be [max_pos, rot_dim / 2]")
        max_pos, rot = cos.shape[0], 2 * cos.shape[1]
    if rot_dim is not None and rot_dim != rot:
        raise ValueError(f"rot_dim {rot_dim} does not fit tables of {rot // 2} pairs")
    rows = NewRows.from_buffer_copy(_ROWS.pack(
        dt, qp, k_new.data_ptr(), v_new.data_ptr(), qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2],
        _opt(new_lens, "new_lens", torch.int32, index, (B,)), _opt(positions, "positions", torch.int32, index, (B, n)),
        cp, sp, max_pos, rot, 1 if interleaved else 0))
    buf, handle = _scratch(workspace, index, 256, stream)
    _launch(index, handle, fn, where, rows, desc, qo, B, n, Hq, Hkv, _opt(seq_lens, "seq_lens", torch.int32, index, (B,)),
            max_seq_len, D, buf.data_ptr(), buf.numel())
    return q_out


def append_rope(k_new, v_new, k, v, cos=None, sin=None, *, q=None, q_out=None, rot_dim=None, interleaved=False,
                positions=None, new_lens=None, seq_lens=None, max_seq_len=None, block_table=None,
                workspace: Optional[Workspace] = None, stream=None):
    """``fd_append_rope``: rotate ``q`` and ``k_new`` by position, write ``k_new`` and ``v_new`` into the cache.

    ``k_new``, ``v_new`` ``[B, n, Hkv, D]`` and ``q`` ``[B, n, Hq, D]`` (optional), bf16 or fp32, may be
    strided views (slices of one fused projection); ``k``, ``v`` are the cache as in ``decode`` (bf16 or fp32),
    written in place.  ``cos``, ``sin`` fp32 ``[max_pos, rot_dim / 2]`` (None: no rotation).  Token ``j`` of sequence
    ``b`` goes to place ``seq_lens[b] + j``; with ``new_lens`` ``[B]`` only the last ``new_lens[b]`` of the ``n``
    rows are tokens.  ``seq_lens`` and ``max_seq_len`` are the lengths before the append.  ``positions``
    ``[B, n]`` int32 replaces the places as rows of the tables.  Without ``workspace`` the stream's own is taken (see
    ``Workspace``).  Returns the rotated queries, fp32
    ``[B, Hq, n, D]`` (``q_out`` if given, whose padding rows keep their contents; None without ``q``).
    """
    torch = _torch()
    index = _index_of(k, "k")
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 4:
        raise ValueError("k_new must be [B, n, Hkv, D]")
    if k.dim() != 4:
        raise ValueError("k and v must be [B, Hkv, T, D] or [num_pages, Hkv, page, D]")
    shape, dtype, B = k.shape, k.dtype, k_new.shape[0]
    dt = FD_BF16 if dtype is torch.bfloat16 else FD_F32 if dtype is torch.float32 else -1
    if dt < 0:
        raise ValueError(f"unsupported KV dtype {dtype}")
    at, vt = _flat(k, "k", dtype, index), _flat(v, "v", dtype, index, shape)
    tokens = shape[2]
    if block_table is None:
        if shape[0] != B:
            raise ValueError(f"a contiguous cache must hold {B} sequences, got {shape[0]}")
        d = _KV.pack(FD_KV_CONTIGUOUS, dt, at, vt, tokens, 0, 0, 0, 0)
    else:
        table, pages = _table(block_table, B, index)
        d = _KV.pack(FD_KV_PAGED, dt, at, vt, 0, table, pages, tokens, shape[0])
        tokens *= pages
    return _append(_lib().fd_append_rope, "fd_append_rope", KvDesc.from_buffer_copy(d), k_new, v_new, shape[1], shape[3],
                   tokens, index, cos, sin, q, q_out, rot_dim, interleaved, positions, new_lens, seq_lens, max_seq_len,
                   workspace, stream)


def append_rope_kv4(k_new, v_new, kv4, cos=None, sin=None, *, k_exp=0, v_exp=0, q=None, q_out=None, rot_dim=None,
                    interleaved=False, positions=None, new_lens=None, seq_lens=None, max_seq_len=None,
                    block_table=None, workspace: Optional[Workspace] = None, stream=None):
    """``fd_append_rope_kv4``: ``append_rope`` into a 4-bit cache (see ``kv4_cache``), written in place."""
    if not isinstance(k_new, _torch().Tensor) or k_new.dim() != 4:
        raise ValueError("k_new must be [B, n, Hkv, D]")
    desc, Hkv, D, tokens, index = _kv4_desc(kv4, block_table, k_new.shape[0], k_exp, v_exp)
    return _append(_lib().fd_append_rope_kv4, "fd_append_rope_kv4", desc, k_new, v_new, Hkv, D, tokens, index, cos, sin,
                   q, q_out, rot_dim, interleaved, positions, new_lens, seq_lens, max_seq_len, workspace, stream)


def kv4_read(kv4, n, *, starts=None, seq_lens=None, max_seq_len=None, block_table=None, k_exp=0, v_exp=0, dtype=None,
             k_out=None, v_out=None, workspace: Optional[Workspace] = None, stream=None):
    """``fd_kv4_read``: tokens ``starts[b] + i``, ``i < n``, of a 4-bit cache as values ``[B, Hkv, n, D]``.

    ``dtype`` bf16 or fp32: that of ``k_out`` or ``v_out`` if given, else bf16.  Rows at or past ``seq_lens[b]`` keep the contents of ``k_out`` and
    ``v_out`` (zeros when they are made here).  Returns ``(k_out, v_out)``.
    """
    torch = _torch()
    index = _index_of(kv4, "kv4")
    for t, name in ((block_table, "block_table"), (k_out, "k_out"), (v_out, "v_out")):
        if t is not None:
            _index_of(t, name)
    lead = kv4.shape if block_table is None else block_table.shape
    B = lead[0] if lead else 0
    desc, Hkv, D, tokens, index = _kv4_desc(kv4, block_table, B, k_exp, v_exp)
    if dtype is None:
        given = k_out if k_out is not None else v_out
        dtype = torch.bfloat16 if given is None else given.dtype
    dt = FD_BF16 if dtype is torch.bfloat16 else FD_F32 if dtype is torch.float32 else -1
    if dt < 0:
        raise ValueError(f"unsupported dtype {dtype}")
    n = _i32(n, "n of the rows")
    max_seq_len = _i32(tokens if max_seq_len is None else max_seq_len, "max_seq_len")
    shape = (B, Hkv, n, D)
    if k_out is None:
        k_out = _made(torch.zeros, shape, dtype, kv4.device, stream)
    if v_out is None:
        v_out = _made(torch.zeros, shape, dtype, kv4.device, stream)
    buf, handle = _scratch(workspace, index, 256, stream)
    _launch(index, handle, _lib().fd_kv4_read, "fd_kv4_read", desc, _flat(k_out, "k_out", dtype, index, shape),
            _flat(v_out, "v_out", dtype, index, shape), dt, B, n, Hkv, _opt(starts, "starts", torch.int32, index, (B,)),
            _opt(seq_lens, "seq_lens", torch.int32, index, (B,)), max_seq_len, D, buf.data_ptr(), buf.numel())
    return k_out, v_out


def decode_kv4(q, kv4, *, k_exp=0, v_exp=0, causal=True, seq_lens=None, max_seq_len=None, block_table=None, scale=None,
               n_splits=FD_SPLITS_AUTO, out=None, lse=None, return_lse=True, workspace: Optional[Workspace] = None,
               stream=None):
    """``fd_decode_kv4``: decode attention over a 4-bit cache.

    q ``[B, Hq, D]`` or ``[B, Hq, n_q, D]`` fp32 (``n_q`` up to 64 rows, masked as in ``decode_rows``); ``kv4`` as made by
    ``kv4_cache``.  Calls that may run at the same time need a ``workspace`` each; without one, each stream has its own (see
    ``Workspace``).  Returns ``(out, lse)`` shaped like q and q without its last axis.
    """
    torch = _torch()
    index = _index_of(q, "q")
    at = _flat(q, "q", torch.float32, index)
    shape = q.shape
    rank = len(shape)
    if rank != 3 and rank != 4:
        raise ValueError("q must be [B, Hq, D] or [B, Hq, n_q, D]")
    B, Hq = shape[0], shape[1]
    n_q = shape[2] if rank == 4 else 1
    desc, Hkv, D, tokens, on = _kv4_desc(kv4, block_table, B, k_exp, v_exp)
    if D != shape[-1]:
        raise ValueError("head_dim of q and kv4 differ")
    if on != index:
        raise ValueError("q and kv4 must be on one device")
    if out is None:
        out = _made(torch.empty, shape, torch.float32, q.device, stream)
        op = out.data_ptr()
    else:
        op = _flat(out, "out", torch.float32, index, shape)
    lp = 0
    if lse is not None:
        lp = _flat(lse, "lse", torch.float32, index, shape[:-1])
    elif return_lse:
        lse = _made(torch.empty, shape[:-1], torch.float32, q.device, stream)
        lp = lse.data_ptr()
    n_splits = _i32(n_splits, "n_splits")
    max_seq_len = _i32(tokens if max_seq_len is None else max_seq_len, "max_seq_len")
    buf, handle = _scratch(workspace, index, _decode_bytes(B, Hq * n_q, Hkv, D, n_splits, index), stream)
    _launch(index, handle, _lib().fd_decode_kv4, "fd_decode_kv4", at, n_q, 1 if causal else 0, desc, op, lp, B, Hq, Hkv,
            _opt(seq_lens, "seq_lens", torch.int32, index, (B,)), max_seq_len, D,
            1.0 / math.sqrt(D) if scale is None else float(scale), n_splits, buf.data_ptr(), buf.numel())
    return out, lse
