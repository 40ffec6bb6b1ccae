"""Thin ctypes binding of ``libcartattn.so`` (see ``include/cartattn.h``).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch provides device memory (outputs and workspaces are
allocated with ``torch.empty`` on the inputs' device) and the current stream.
If the library has not been built, every call raises -- there is no other
implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading
from typing import Optional

import torch

from . import build as _build

CART_BF16 = 0
CART_F32 = 1

STATUS = {0: "ok", -1: "bad geometry", -2: "null or misaligned pointer", -3: "unsupported dtype",
          -4: "workspace too small", -5: "CUDA error", -6: "device is not sm_103",
          -7: "a kernel gave up waiting"}

_lock = threading.Lock()
_lib = None


class CartError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({STATUS.get(status, 'unknown')})")
        self.status = status


class _Geom(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("n", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("d", ctypes.c_int), ("p", ctypes.c_int),
                ("frozen_prefix", ctypes.c_int), ("scale", ctypes.c_float),
                ("rope_theta", ctypes.c_double), ("window", ctypes.c_int)]


def library_path() -> str:
    return _build.LIB


def lib():
    """Load the in-tree library; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with `python -m trained_kv_prefix_gb300.build` "
                    "(there is no non-CUDA implementation of this path)")
            L = ctypes.CDLL(path)
            vp, sz, i, f, d = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float, ctypes.c_double
            G = ctypes.POINTER(_Geom)
            L.cart_write_to_cache.argtypes = [vp, vp, i, i, i, vp, vp, ctypes.c_longlong, i, i, vp]
            L.cart_attn_fwd_workspace_size.argtypes = [G, i, i]
            L.cart_attn_fwd_workspace_size.restype = sz
            L.cart_attn_fwd.argtypes = [G, i, i, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            L.cart_attn_bwd_workspace_size.argtypes = [G, i, i]
            L.cart_attn_bwd_workspace_size.restype = sz
            L.cart_attn_bwd.argtypes = [G, i, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                        i, vp, sz, vp]
            L.cart_attn_bwd_parts.argtypes = [G, i, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                              vp, vp, vp, ctypes.POINTER(ctypes.c_int), i, i, vp,
                                              sz, vp]
            L.cart_attn_bwd_reuse_workspace_size.argtypes = [G, i, i]
            L.cart_attn_bwd_reuse_workspace_size.restype = sz
            L.cart_attn_bwd_reuse.argtypes = [G, i, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                              vp, vp, vp, i, vp, sz, vp, sz, vp]
            L.cart_attn_decode_workspace_size.argtypes = [i, i, i, i, i, i]
            L.cart_attn_decode_workspace_size.restype = sz
            L.cart_attn_decode.argtypes = [i, i, i, i, i, f, d, vp, vp, vp, vp, vp, vp, vp, i, vp,
                                           vp, vp, sz, vp]
            L.cart_attn_decode_span_workspace_size.argtypes = [i, i, i, i, i, i, i]
            L.cart_attn_decode_span_workspace_size.restype = sz
            L.cart_attn_decode_span.argtypes = [i, i, i, i, i, i, i, f, d, vp, vp, vp, vp, vp, vp,
                                                vp, i, vp, vp, vp, sz, vp]
            L.cart_attn_fwd_packed_workspace_size.argtypes = [G, i, i, i]
            L.cart_attn_fwd_packed_workspace_size.restype = sz
            L.cart_attn_fwd_packed.argtypes = [G, i, vp, i, i, vp, vp, vp, vp, vp, vp, vp, vp,
                                               sz, vp]
            L.cart_attn_bwd_packed_workspace_size.argtypes = [G, i, i, i]
            L.cart_attn_bwd_packed_workspace_size.restype = sz
            L.cart_attn_bwd_packed.argtypes = [G, i, vp, i, i, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                               vp, vp, vp, vp, ctypes.POINTER(ctypes.c_int), i, i,
                                               vp, sz, vp]
            L.cart_attn_decode_tree_workspace_size.argtypes = [i] * 8
            L.cart_attn_decode_tree_workspace_size.restype = sz
            L.cart_attn_decode_tree.argtypes = [i, i, i, i, i, i, i, f, d, vp, vp, vp, vp, vp, vp,
                                                vp, i, i, vp, i, vp, vp, vp, vp, sz, vp]
            L.cart_pages_fork.argtypes = [i, vp, i, vp, vp, i, i, vp, vp, vp, i, vp, vp]
            L.cart_pages_workspace_size.argtypes = [i, i, i]
            L.cart_pages_workspace_size.restype = sz
            L.cart_pages_reserve.argtypes = [i, i, i, i, i, vp, vp, i, i, vp, i, vp, vp, vp, vp,
                                             vp, sz, vp]
            L.cart_pages_accept.argtypes = [i, i, i, i, i, i, vp, vp, i, i, vp, i, vp, vp, vp, vp,
                                            vp]
            L.cart_pages_compact.argtypes = [i, i, i, i, i, vp, vp, i, i, vp, i, vp, vp, vp, vp,
                                             sz, vp]
            L.cart_status_string.argtypes = [i]
            L.cart_status_string.restype = ctypes.c_char_p
            L.cart_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), i]
            L.cart_trace_enable.argtypes = [i]
            L.cart_release.argtypes = []
            L.cart_release.restype = ctypes.c_int
            L.cart_trace_count.argtypes = []
            L.cart_trace_get.argtypes = [i, ctypes.c_char_p, i, ctypes.POINTER(ctypes.c_float)]
            for name in ("cart_write_to_cache", "cart_attn_fwd", "cart_attn_bwd", "cart_attn_bwd_parts",
                         "cart_attn_bwd_reuse",
                         "cart_attn_fwd_packed", "cart_attn_bwd_packed",
                         "cart_attn_decode", "cart_attn_decode_span", "cart_device_status",
                         "cart_attn_decode_tree", "cart_pages_fork", "cart_pages_reserve",
                         "cart_pages_accept", "cart_pages_compact",
                         "cart_trace_enable",
                         "cart_trace_count", "cart_trace_get"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
        return _lib


EXPORTS = ("cart_write_to_cache", "cart_attn_fwd_workspace_size", "cart_attn_fwd",
           "cart_attn_bwd_workspace_size", "cart_attn_bwd", "cart_attn_bwd_parts",
           "cart_attn_bwd_reuse_workspace_size", "cart_attn_bwd_reuse",
           "cart_attn_decode_workspace_size",
           "cart_attn_decode", "cart_status_string", "cart_device_status", "cart_trace_enable",
           "cart_trace_count", "cart_trace_get", "cart_attn_decode_noalloc",
           "cart_attn_decode_span_workspace_size", "cart_attn_decode_span",
           "cart_attn_fwd_packed_workspace_size", "cart_attn_fwd_packed",
           "cart_attn_bwd_packed_workspace_size", "cart_attn_bwd_packed", "cart_release",
           "cart_attn_decode_tree_workspace_size", "cart_attn_decode_tree", "cart_pages_fork",
           "cart_pages_workspace_size", "cart_pages_reserve", "cart_pages_accept",
           "cart_pages_compact")


def _check(fn: str, rc: int):
    if rc != 0:
        raise CartError(fn, rc)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return CART_BF16
    if t.dtype == torch.float32:
        return CART_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, device) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def geom(B, n, Hq, Hkv, d, p, frozen_prefix=1, scale=None, theta=1.0e6, window=0) -> _Geom:
    """Training geometry; ``window`` > 0 is a sliding window in keys (the
    query at position P sees keys P - window + 1 .. P), 0 none."""
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    return _Geom(B, n, Hq, Hkv, d, p, frozen_prefix, float(scale), float(theta), int(window))


def _make(stream, make, *args, returned=True, **kwargs):
    """``make(*args, **kwargs)``, a tensor that a call on ``stream`` (None: the
    current one) works on: allocated, and filled, on that stream, since the
    current stream's memory could be a block that it has freed and is still
    working on; and one that the call returns is kept for the current stream
    too, which reads it."""
    if stream is None:
        return make(*args, **kwargs)
    with torch.cuda.stream(stream):
        t = make(*args, **kwargs)
    if returned:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor], stream) -> torch.Tensor:
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        return workspace
    return _make(stream, torch.empty, max(nbytes, 16), dtype=torch.uint8, device=device,
                 returned=False)


# ------------------------------------------------------------------ calls ----
def cart_write_to_cache(kc: torch.Tensor, vc: torch.Tensor, k_dst: torch.Tensor,
                        v_dst: torch.Tensor, dst_row0: int = 0, stream=None):
    """Write f32 cartridge rows ``[p, Hkv, d]`` into ``k_dst``/``v_dst``
    (``[rows, Hkv, d]`` bf16 or f32) starting at row ``dst_row0``."""
    p, Hkv, d = kc.shape
    row_stride = k_dst.stride(0)
    rc = lib().cart_write_to_cache(_ptr(kc), _ptr(vc), p, Hkv, d, _ptr(k_dst), _ptr(v_dst),
                                   row_stride, dst_row0, _dt(k_dst), _stream(stream, kc.device))
    _check("cart_write_to_cache", rc)
    return k_dst, v_dst


def fwd_workspace_size(g: _Geom, in_dtype: int, cart_dtype: int) -> int:
    return int(lib().cart_attn_fwd_workspace_size(ctypes.byref(g), in_dtype, cart_dtype))


def bwd_workspace_size(g: _Geom, in_dtype: int, cart_dtype: int) -> int:
    return int(lib().cart_attn_bwd_workspace_size(ctypes.byref(g), in_dtype, cart_dtype))


def cart_attn_fwd(q, k, v, kc, vc, *, frozen_prefix=1, scale=None, theta=1.0e6, o=None, lse=None,
                  workspace=None, stream=None, window=0):
    """Training forward.  q ``[B, n, Hq, d]``, k/v ``[B, n, Hkv, d]`` (not
    rotated), kc/vc ``[p, Hkv, d]`` (bf16 shadow or f32 leaves).  Returns
    ``(o, lse)`` with o like q and lse ``[B, Hq, n]`` f32.  ``window`` > 0:
    sliding window in keys over the concatenated sequence (see ``geom``)."""
    B, n, Hq, d = q.shape
    Hkv = k.shape[2]
    p = kc.shape[0]
    g = geom(B, n, Hq, Hkv, d, p, min(frozen_prefix, p), scale, theta, window)
    dt, cd = _dt(q), _dt(kc)
    if o is None:
        o = _make(stream, torch.empty_like, q)
    if lse is None:
        lse = _make(stream, torch.empty, (B, Hq, n), dtype=torch.float32, device=q.device)
    ws = _workspace(fwd_workspace_size(g, dt, cd), q.device, workspace, stream)
    rc = lib().cart_attn_fwd(ctypes.byref(g), dt, cd, _ptr(q), _ptr(k), _ptr(v), _ptr(kc),
                             _ptr(vc), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                             _stream(stream, q.device))
    _check("cart_attn_fwd", rc)
    return o, lse


def cart_attn_bwd(q, k, v, kc, vc, o, lse, dout, *, frozen_prefix=1, scale=None, theta=1.0e6,
                  accumulate=False, dq=None, dk=None, dv=None, dkc=None, dvc=None,
                  workspace=None, stream=None, frozen_rows=None, window=0,
                  fwd_workspace=None):
    """Backward.  Returns ``(dq, dk, dv, dkc, dvc)``; dkc/dvc are f32
    ``[p, Hkv, d]`` summed over the batch, rows < frozen_prefix and the rows
    listed in ``frozen_rows`` (a composed cartridge's part sinks) exactly 0.
    ``window`` must match the forward's.  ``fwd_workspace``: the workspace
    the forward of these inputs used (cart_attn_bwd_reuse: its rotated
    queries and keys are read instead of recomputed); not with
    ``frozen_rows``."""
    B, n, Hq, d = q.shape
    Hkv = k.shape[2]
    p = kc.shape[0]
    g = geom(B, n, Hq, Hkv, d, p, frozen_prefix, scale, theta, window)
    dt, cd = _dt(q), _dt(kc)
    dq = _make(stream, torch.empty_like, q) if dq is None else dq
    dk = _make(stream, torch.empty_like, k) if dk is None else dk
    dv = _make(stream, torch.empty_like, v) if dv is None else dv
    if dkc is None:
        dkc = _make(stream, torch.zeros if accumulate else torch.empty, (max(p, 1), Hkv, d),
                    dtype=torch.float32, device=q.device)
    if dvc is None:
        dvc = _make(stream, torch.zeros if accumulate else torch.empty, (max(p, 1), Hkv, d),
                    dtype=torch.float32, device=q.device)
    if fwd_workspace is not None:
        if frozen_rows is not None:
            raise ValueError("fwd_workspace does not combine with frozen_rows")
        ws = _workspace(int(lib().cart_attn_bwd_reuse_workspace_size(ctypes.byref(g), dt, cd)),
                        q.device, workspace, stream)
        rc = lib().cart_attn_bwd_reuse(ctypes.byref(g), dt, cd, _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(kc), _ptr(vc), _ptr(o), _ptr(lse), _ptr(dout),
                                       _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dkc), _ptr(dvc),
                                       1 if accumulate else 0, _ptr(fwd_workspace),
                                       fwd_workspace.numel(), _ptr(ws), ws.numel(),
                                       _stream(stream, q.device))
        _check("cart_attn_bwd_reuse", rc)
        return dq, dk, dv, dkc[:p], dvc[:p]
    ws = _workspace(bwd_workspace_size(g, dt, cd), q.device, workspace, stream)
    if frozen_rows is None:
        rc = lib().cart_attn_bwd(ctypes.byref(g), dt, cd, _ptr(q), _ptr(k), _ptr(v), _ptr(kc),
                                 _ptr(vc), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                                 _ptr(dv), _ptr(dkc), _ptr(dvc), 1 if accumulate else 0, _ptr(ws),
                                 ws.numel(), _stream(stream, q.device))
        _check("cart_attn_bwd", rc)
    else:
        rows = list(frozen_rows)
        arr = (ctypes.c_int * max(len(rows), 1))(*rows)
        rc = lib().cart_attn_bwd_parts(ctypes.byref(g), dt, cd, _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(kc), _ptr(vc), _ptr(o), _ptr(lse), _ptr(dout),
                                       _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dkc), _ptr(dvc), arr,
                                       len(rows), 1 if accumulate else 0, _ptr(ws), ws.numel(),
                                       _stream(stream, q.device))
        _check("cart_attn_bwd_parts", rc)
    return dq, dk, dv, dkc[:p], dvc[:p]


def bwd_reuse_workspace_size(g: _Geom, in_dtype: int, cart_dtype: int) -> int:
    return int(lib().cart_attn_bwd_reuse_workspace_size(ctypes.byref(g), in_dtype, cart_dtype))


def fwd_packed_workspace_size(g: _Geom, total: int, in_dtype: int, cart_dtype: int) -> int:
    return int(lib().cart_attn_fwd_packed_workspace_size(ctypes.byref(g), total, in_dtype,
                                                         cart_dtype))


def bwd_packed_workspace_size(g: _Geom, total: int, in_dtype: int, cart_dtype: int) -> int:
    return int(lib().cart_attn_bwd_packed_workspace_size(ctypes.byref(g), total, in_dtype,
                                                         cart_dtype))


def _packing(cu_seqlens, max_seqlen, q):
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.device != q.device:
        raise TypeError("cu_seqlens must be int32 on the tensors' device")
    return cu_seqlens.numel() - 1, int(max_seqlen), q.shape[0]


def cart_attn_fwd_packed(q, k, v, kc, vc, cu_seqlens, max_seqlen, *, frozen_prefix=1,
                         scale=None, theta=1.0e6, o=None, lse=None, workspace=None, stream=None,
                         window=0):
    """Training forward on packed segments.  q ``[T, Hq, d]``, k/v
    ``[T, Hkv, d]`` (not rotated), segment s = tokens cu_seqlens[s] ..
    cu_seqlens[s+1]-1 (int32 on the device), none longer than max_seqlen.
    Returns ``(o [T, Hq, d], lse [Hq, T] f32)``."""
    S, n, T = _packing(cu_seqlens, max_seqlen, q)
    Hq, d = q.shape[1], q.shape[2]
    Hkv = k.shape[1]
    p = kc.shape[0]
    g = geom(S, n, Hq, Hkv, d, p, min(frozen_prefix, p), scale, theta, window)
    dt, cd = _dt(q), _dt(kc)
    if o is None:
        o = _make(stream, torch.empty_like, q)
    if lse is None:
        lse = _make(stream, torch.empty, (Hq, T), dtype=torch.float32, device=q.device)
    ws = _workspace(fwd_packed_workspace_size(g, T, dt, cd), q.device, workspace, stream)
    rc = lib().cart_attn_fwd_packed(ctypes.byref(g), T, _ptr(cu_seqlens), dt, cd, _ptr(q),
                                    _ptr(k), _ptr(v), _ptr(kc), _ptr(vc), _ptr(o), _ptr(lse),
                                    _ptr(ws), ws.numel(), _stream(stream, q.device))
    _check("cart_attn_fwd_packed", rc)
    return o, lse


def cart_attn_bwd_packed(q, k, v, kc, vc, o, lse, dout, cu_seqlens, max_seqlen, *,
                         frozen_prefix=1, scale=None, theta=1.0e6, accumulate=False, dq=None,
                         dk=None, dv=None, dkc=None, dvc=None, workspace=None, stream=None,
                         frozen_rows=(), window=0):
    """Backward on packed segments (layouts of cart_attn_fwd_packed).
    Returns ``(dq, dk, dv, dkc, dvc)``; dkc/dvc f32 ``[p, Hkv, d]`` summed
    over the segments, frozen rows exactly 0."""
    S, n, T = _packing(cu_seqlens, max_seqlen, q)
    Hq, d = q.shape[1], q.shape[2]
    Hkv = k.shape[1]
    p = kc.shape[0]
    g = geom(S, n, Hq, Hkv, d, p, frozen_prefix, scale, theta, window)
    dt, cd = _dt(q), _dt(kc)
    dq = _make(stream, torch.empty_like, q) if dq is None else dq
    dk = _make(stream, torch.empty_like, k) if dk is None else dk
    dv = _make(stream, torch.empty_like, v) if dv is None else dv
    if dkc is None:
        dkc = _make(stream, torch.zeros if accumulate else torch.empty, (max(p, 1), Hkv, d),
                    dtype=torch.float32, device=q.device)
    if dvc is None:
        dvc = _make(stream, torch.zeros if accumulate else torch.empty, (max(p, 1), Hkv, d),
                    dtype=torch.float32, device=q.device)
    ws = _workspace(bwd_packed_workspace_size(g, T, dt, cd), q.device, workspace, stream)
    rows = list(frozen_rows)
    arr = (ctypes.c_int * max(len(rows), 1))(*rows)
    rc = lib().cart_attn_bwd_packed(ctypes.byref(g), T, _ptr(cu_seqlens), dt, cd, _ptr(q),
                                    _ptr(k), _ptr(v), _ptr(kc), _ptr(vc), _ptr(o), _ptr(lse),
                                    _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dkc),
                                    _ptr(dvc), arr, len(rows), 1 if accumulate else 0, _ptr(ws),
                                    ws.numel(), _stream(stream, q.device))
    _check("cart_attn_bwd_packed", rc)
    return dq, dk, dv, dkc[:p], dvc[:p]


def decode_workspace_size(B, Hq, Hkv, d, p, rows) -> int:
    return int(lib().cart_attn_decode_workspace_size(B, Hq, Hkv, d, p, rows))


def cart_attn_decode(q, k_new, v_new, kc, vc, k_cache, v_cache, lens, *, scale=None, theta=1.0e6,
                     o=None, workspace=None, stream=None):
    """One decode step.  q ``[B, Hq, d]``, k_new/v_new ``[B, Hkv, d]`` (bf16,
    not rotated), kc/vc ``[p, Hkv, d]`` bf16 shared cartridge, caches
    ``[B, rows, Hkv, d]`` bf16 (modified: row lens[b] receives the new token),
    lens ``[B]`` int32 on the device.  Returns o ``[B, Hq, d]`` bf16."""
    B, Hq, d = q.shape
    Hkv = k_new.shape[1]
    p = kc.shape[0]
    rows = k_cache.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if lens.dtype != torch.int32:
        raise TypeError("lens must be int32")
    if o is None:
        o = _make(stream, torch.empty_like, q)
    ws = _workspace(decode_workspace_size(B, Hq, Hkv, d, p, rows), q.device, workspace, stream)
    rc = lib().cart_attn_decode(B, Hq, Hkv, d, p, float(scale), float(theta), _ptr(q),
                                _ptr(k_new), _ptr(v_new), _ptr(kc), _ptr(vc), _ptr(k_cache),
                                _ptr(v_cache), rows, _ptr(lens), _ptr(o), _ptr(ws), ws.numel(),
                                _stream(stream, q.device))
    _check("cart_attn_decode", rc)
    return o


def decode_span_workspace_size(B, span, Hq, Hkv, d, p, rows) -> int:
    return int(lib().cart_attn_decode_span_workspace_size(B, span, Hq, Hkv, d, p, rows))


def cart_attn_decode_span(q, k_new, v_new, kc, vc, k_cache, v_cache, lens, *, scale=None,
                          theta=1.0e6, o=None, workspace=None, stream=None, window=0):
    """Span verify: ``span`` new tokens per conversation in one step.  q
    ``[B, span, Hq, d]``, k_new/v_new ``[B, span, Hkv, d]`` (bf16, not
    rotated); the caches receive the span's rows lens[b] .. lens[b]+span-1.
    Returns o ``[B, span, Hq, d]`` bf16.  ``window`` > 0: token t sees the
    keys at positions p + lens[b] + t - window + 1 .. p + lens[b] + t."""
    B, span, Hq, d = q.shape
    Hkv = k_new.shape[2]
    p = kc.shape[0]
    rows = k_cache.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if lens.dtype != torch.int32:
        raise TypeError("lens must be int32")
    if o is None:
        o = _make(stream, torch.empty_like, q)
    ws = _workspace(decode_span_workspace_size(B, span, Hq, Hkv, d, p, rows), q.device, workspace,
                    stream)
    rc = lib().cart_attn_decode_span(B, span, int(window), Hq, Hkv, d, p, float(scale),
                                     float(theta), _ptr(q),
                                     _ptr(k_new), _ptr(v_new), _ptr(kc), _ptr(vc),
                                     _ptr(k_cache), _ptr(v_cache), rows, _ptr(lens), _ptr(o),
                                     _ptr(ws), ws.numel(), _stream(stream, q.device))
    _check("cart_attn_decode_span", rc)
    return o


# ------------------------------------------------- paged private caches ----
# The calls below are a few microseconds of GPU time for a small batch, so
# their bindings keep to a few checks per tensor.
_raw_stream = torch._C._cuda_getCurrentRawStream


class _On:
    """Where a call on a paged cache runs: on ``device``, made current while
    it is not, and on ``stream`` or the device's current one."""

    __slots__ = ("device", "guard", "stream", "handle")

    def __init__(self, device, stream):
        self.device = device
        self.guard = None
        index = device.index
        if device.type != "cuda":
            raise ValueError(f"tensors must be on a GPU, not on {device}")
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream must be one of {device}, not of {stream.device}")
        if index != torch.cuda.current_device():
            self.guard = torch.cuda.device(device)
            self.guard.__enter__()
        self.handle = _raw_stream(index)
        self.stream = None
        if stream is not None and stream.cuda_stream != self.handle:
            self.stream, self.handle = stream, stream.cuda_stream

    def empty(self, shape, dtype, returned=True):
        """Memory of the stream that the call's kernels run on (see _make)."""
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        return _make(self.stream, torch.empty, shape, dtype=dtype, device=self.device,
                     returned=returned)

    def close(self):
        if self.guard is not None:
            self.guard.__exit__(None, None, None)


def _arg(name, t, dtype, shape, device):
    """Data pointer of a contiguous tensor that has to have this dtype, shape
    and device."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, not on {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _fits(**sizes):
    """Refuses a number that the library's 32 bits would take for another
    (those that fit are its own to refuse)."""
    for name, n in sizes.items():
        if not -1 << 31 <= n < 1 << 31:
            raise ValueError(f"{name}: {n} does not fit 32 bits")


def _scratch(on, workspace, need):
    """(tensor, pointer, bytes) of the caller's workspace, or of a new one."""
    if workspace is None:
        need = max(need, 16)
        workspace = on.empty((need,), torch.uint8, returned=False)
        return workspace, workspace.data_ptr(), need
    if workspace.device != on.device or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be contiguous and on {on.device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _pools(k_pages, v_pages):
    """(layers, pages, rows, Hkv, d, dtype code, k pointer, v pointer, device)
    of a pair of pools ``[layers, pages, rows, Hkv, d]`` or one layer of it."""
    shape = k_pages.shape
    if len(shape) not in (4, 5):
        raise ValueError("pools are [layers, pages, rows, Hkv, d] or one layer of it")
    dev, dt = k_pages.device, k_pages.dtype
    return (shape[0] if len(shape) == 5 else 1, *shape[-4:], _dt(k_pages),
            _arg("k_pages", k_pages, dt, shape, dev), _arg("v_pages", v_pages, dt, shape, dev), dev)


@functools.lru_cache(maxsize=1024)  # (a function of the sizes alone; the call costs 2 us)
def decode_tree_workspace_size(B, nodes, Hq, Hkv, d, p, page_rows, max_pages) -> int:
    return int(lib().cart_attn_decode_tree_workspace_size(B, nodes, Hq, Hkv, d, p, page_rows,
                                                          max_pages))


def cart_attn_decode_tree(q, k_new, v_new, kc, vc, k_pages, v_pages, table, lens, parents=None, *,
                          scale=None, theta=1.0e6, window=0, o=None, workspace=None, stream=None):
    """One step over a tree of drafted tokens per conversation, its private
    rows in pages.  q ``[B, nodes, Hq, d]``, k_new/v_new ``[B, nodes, Hkv,
    d]`` (bf16, not rotated), kc/vc ``[p, Hkv, d]`` bf16 shared cartridge
    (``[0, Hkv, d]``: none), k_pages/v_pages ``[pages, page_rows, Hkv, d]``
    bf16 pools (the rows lens[b] + t of the used nodes t are written), table
    ``[B, max_pages]`` and lens ``[B]`` int32.  parents ``[B, nodes]`` int32: the node that each
    node follows, an earlier one, -1 for the cached rows, -2 for an unused
    node; None: chains.  Returns o ``[B, nodes, Hq, d]`` bf16, 0 for unused
    nodes.  ``window`` as in ``cart_attn_decode_span``."""
    B, T, Hq, d = q.shape
    Hkv, p = k_new.shape[2], kc.shape[0]
    N, P = k_pages.shape[0], k_pages.shape[1]
    M, dev, bf, i32 = table.shape[-1], q.device, torch.bfloat16, torch.int32
    if (B | M | N | window) >> 31:
        _fits(conversations=B, max_pages=M, pages=N, window=window)
    new = (B, T, Hkv, d)
    args = (_arg("q", q, bf, q.shape, dev),
            _arg("k_new", k_new, bf, new, dev), _arg("v_new", v_new, bf, new, dev),
            _arg("kc", kc, bf, (p, Hkv, d), dev), _arg("vc", vc, bf, (p, Hkv, d), dev),
            _arg("k_pages", k_pages, bf, (N, P, Hkv, d), dev),
            _arg("v_pages", v_pages, bf, (N, P, Hkv, d), dev), N, P,
            _arg("table", table, i32, (B, M), dev), M,
            _arg("lens", lens, i32, (B,), dev),
            None if parents is None else _arg("parents", parents, i32, (B, T), dev))
    on = _On(dev, stream)
    try:
        if o is None:
            o = torch.empty_like(q) if on.stream is None else on.empty(q.shape, bf)
            op = o.data_ptr()
        else:
            op = _arg("o", o, bf, q.shape, dev)
        ws, wp, wn = _scratch(on, workspace,
                              decode_tree_workspace_size(B, T, Hq, Hkv, d, p, P, M))
        rc = (_lib or lib()).cart_attn_decode_tree(
            B, T, window, Hq, Hkv, d, p, d ** -0.5 if scale is None else scale, theta, *args, op,
            wp, wn, on.handle)
    finally:
        on.close()
    _check("cart_attn_decode_tree", rc)
    return o


@functools.lru_cache(maxsize=1024)
def pages_workspace_size(B, max_pages, n_pages) -> int:
    return int(lib().cart_pages_workspace_size(B, max_pages, n_pages))


def cart_pages_fork(table, lens, refs, src, dst, rows=None, *, page_rows, done=None, stream=None):
    """Conversation dst[f] becomes the first rows[f] (None: all) rows of
    conversation src[f], sharing its pages.  table ``[B, max_pages]``, lens
    ``[B]`` and refs ``[pages]`` int32 are updated; src, dst, rows
    ``[forks]`` int32, all on the device.  Returns done ``[forks]`` int32: 0
    for a fork that was left out (dst also named by another fork)."""
    B, M = table.shape
    F, N = src.shape[0], refs.shape[0]
    if (B | M | F | N | page_rows) >> 31:
        _fits(conversations=B, max_pages=M, forks=F, pages=N, page_rows=page_rows)
    dev, i32 = table.device, torch.int32
    args = (B, _arg("table", table, i32, (B, M), dev), M, _arg("lens", lens, i32, (B,), dev),
            _arg("refs", refs, i32, (N,), dev), N, page_rows, _arg("src", src, i32, (F,), dev),
            _arg("dst", dst, i32, (F,), dev),
            None if rows is None else _arg("rows", rows, i32, (F,), dev), F)
    on = _On(dev, stream)
    try:
        if done is None:
            done = on.empty((F,), i32)
        rc = (_lib or lib()).cart_pages_fork(*args, _arg("done", done, i32, (F,), dev), on.handle)
    finally:
        on.close()
    _check("cart_pages_fork", rc)
    return done


def cart_pages_reserve(k_pages, v_pages, table, lens, refs, rows, *, done=None, workspace=None,
                       stream=None):
    """Room for rows[b] rows in all of every conversation: pages behind them
    are given back, and those of rows lens[b] .. rows[b] - 1 come to be b's
    alone (a shared one is copied in every layer; one that is missing is taken
    as it is).  rows ``[B]`` int32 on the device, < 0: left as it is, 0:
    everything is given back, at most lens[b]: nothing is to be appended (see
    the header).
    Pools ``[layers, pages, page_rows, Hkv, d]`` (bf16 or f32); table, lens
    and refs are updated.  Returns done ``[B]`` int32: 1 where there is
    room; a conversation without it must not append (its next row may lie in
    a shared page): ``lens`` -1 for it in the step's other calls, its real
    one kept apart."""
    layers, N, P, Hkv, d, dt, kp, vp, dev = _pools(k_pages, v_pages)
    B, M = table.shape
    if (B | M | N) >> 31:
        _fits(conversations=B, max_pages=M, pages=N)
    i32 = torch.int32
    args = (B, layers, Hkv, d, dt, kp, vp, N, P, _arg("table", table, i32, (B, M), dev), M,
            _arg("lens", lens, i32, (B,), dev), _arg("refs", refs, i32, (N,), dev),
            _arg("rows", rows, i32, (B,), dev))
    on = _On(dev, stream)
    try:
        if done is None:
            done = on.empty((B,), i32)
        ws, wp, wn = _scratch(on, workspace, pages_workspace_size(B, M, N))
        rc = (_lib or lib()).cart_pages_reserve(*args, _arg("done", done, i32, (B,), dev), wp, wn,
                                                on.handle)
    finally:
        on.close()
    _check("cart_pages_reserve", rc)
    return done


def cart_pages_accept(k_pages, v_pages, table, lens, parents, node, *, new_lens=None, stream=None):
    """Keeps the path to node[b] (``[B]`` int32; -1: nothing) of each
    conversation's tree: its rows are moved to lens[b], lens[b] + 1, ... in
    every layer.  parents as in ``cart_attn_decode_tree`` (a tensor, or the
    number of nodes of chains).  Returns new_lens ``[B]`` int32."""
    layers, N, P, Hkv, d, dt, kp, vp, dev = _pools(k_pages, v_pages)
    B, M = table.shape
    i32 = torch.int32
    chains = isinstance(parents, int)
    T = parents if chains else parents.shape[-1]
    if (B | M | N | T) >> 31:
        _fits(conversations=B, max_pages=M, pages=N, nodes=T)
    args = (B, T, layers, Hkv, d, dt, kp, vp, N, P, _arg("table", table, i32, (B, M), dev), M,
            _arg("lens", lens, i32, (B,), dev),
            None if chains else _arg("parents", parents, i32, (B, T), dev),
            _arg("node", node, i32, (B,), dev))
    on = _On(dev, stream)
    try:
        if new_lens is None:
            new_lens = on.empty((B,), i32)
        rc = (_lib or lib()).cart_pages_accept(
            *args, _arg("new_lens", new_lens, i32, (B,), dev), on.handle)
    finally:
        on.close()
    _check("cart_pages_accept", rc)
    return new_lens


def cart_pages_compact(k_pages, v_pages, table, refs, *, moved=None, live=None, workspace=None,
                       stream=None):
    """Moves the pool's live pages to its front, in every layer; table and
    refs are updated.  Returns ``(moved [pages], live [1])`` int32: each
    page's new number (-1: it was free) and the number of live pages."""
    layers, N, P, Hkv, d, dt, kp, vp, dev = _pools(k_pages, v_pages)
    B, M = table.shape
    if (B | M | N) >> 31:
        _fits(conversations=B, max_pages=M, pages=N)
    i32 = torch.int32
    args = (B, layers, Hkv, d, dt, kp, vp, N, P, _arg("table", table, i32, (B, M), dev), M,
            _arg("refs", refs, i32, (N,), dev))
    on = _On(dev, stream)
    try:
        if moved is None:
            moved = on.empty((N,), i32)
        if live is None:
            live = on.empty((1,), i32)
        ws, wp, wn = _scratch(on, workspace, pages_workspace_size(B, M, N))
        rc = (_lib or lib()).cart_pages_compact(*args, _arg("moved", moved, i32, (N,), dev),
                                                _arg("live", live, i32, (1,), dev), wp, wn,
                                                on.handle)
    finally:
        on.close()
    _check("cart_pages_compact", rc)
    return moved, live


def release() -> None:
    """Destroy this device's helper stream and events (recreated on use)."""
    _check("cart_release", lib().cart_release())


def device_status(clear: bool = True) -> int:
    """Bits set by kernels whose bounded waits gave up (0 = none)."""
    bits = ctypes.c_uint(0)
    rc = lib().cart_device_status(ctypes.byref(bits), 1 if clear else 0)
    if rc not in (0, -7):
        raise CartError("cart_device_status", rc)
    return int(bits.value)


def trace_enable(on: bool = True):
    """Start (clearing earlier records) or stop recording per-launch events."""
    lib().cart_trace_enable(1 if on else 0)


def trace_read(with_times: bool = True):
    """List of (kernel name, device ms or None) for the recorded launches."""
    L = lib()
    out = []
    buf = ctypes.create_string_buffer(32)
    for i in range(L.cart_trace_count()):
        ms = ctypes.c_float(-1.0)
        rc = L.cart_trace_get(i, buf, 32, ctypes.byref(ms) if with_times else None)
        if rc != 0 and with_times:
            raise CartError("cart_trace_get", rc)
        out.append((buf.value.decode(), float(ms.value) if with_times else None))
    return out
