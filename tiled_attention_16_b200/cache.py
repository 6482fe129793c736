"""A K/V cache at 16 or 8 bits and decoding over it: the binding of
include/fa_cache.h (argument marshalling only).

The cache is plain tensors that the caller owns: k_cache and v_cache
[B, Hkv, capacity, D], whose dtype is the format (``torch.bfloat16``,
``torch.float8_e4m3fn`` or ``torch.int8``), and for the 8-bit formats
k_scale and v_scale, fp32 [B, Hkv, capacity] (a code stands for code * scale).
``make_cache`` allocates the four.  Lengths and slots are int32 tensors on the
device, so captured calls follow them.  There is no fallback: if the library
is missing or the device is not a B200 the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from .attention import FA_OK, FAError, _check, _same_device, _stream_ptr, lib, symbols_in
from .rope import FaRows, _ptr, check_rows

HEADER_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fa_cache.h")

FORMATS = {torch.bfloat16: 0, torch.float8_e4m3fn: 1, torch.int8: 2}   # FA_CACHE_BF16, _E4M3, _INT8


class FaCacheShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hkv", ctypes.c_int), ("capacity", ctypes.c_int), ("D", ctypes.c_int),
                ("format", ctypes.c_int)]


class FaCacheDecodeShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("Nq", ctypes.c_int),
                ("capacity", ctypes.c_int), ("n_prefix", ctypes.c_int), ("D", ctypes.c_int), ("format", ctypes.c_int),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int)]


_lib = None


def _cache_lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = lib()
        vp, i = ctypes.c_void_p, ctypes.c_int
        shp, dshp, rows = ctypes.POINTER(FaCacheShape), ctypes.POINTER(FaCacheDecodeShape), ctypes.POINTER(FaRows)
        L.fa_cache_write.argtypes = [shp, i, rows, rows, vp, vp, vp, vp, vp, vp, vp]
        L.fa_cache_write.restype = i
        L.fa_cache_read.argtypes = [shp, i, vp, vp, vp, vp, vp, vp, vp, vp]
        L.fa_cache_read.restype = i
        L.fa_decode_cache_workspace_bytes.argtypes = [dshp]
        L.fa_decode_cache_workspace_bytes.restype = ctypes.c_size_t
        L.fa_decode_cache.argtypes = [dshp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.fa_decode_cache.restype = i
        _lib = L
    return _lib


def declared_symbols() -> list[str]:
    """Entry points declared in include/fa_cache.h (FA_API functions)."""
    return symbols_in(HEADER_PATH)


def make_cache(B: int, Hkv: int, capacity: int, D: int, dtype=torch.bfloat16, device="cuda"):
    """(k_cache, v_cache, k_scale, v_scale) on `device`, contents undefined;
    the scales are None for bf16."""
    if dtype not in FORMATS:
        raise TypeError(f"cache dtype must be one of {list(FORMATS)}, got {dtype}")
    k, v = (torch.empty((B, Hkv, capacity, D), device=device, dtype=dtype) for _ in range(2))
    if dtype == torch.bfloat16:
        return k, v, None, None
    ks, vs = (torch.empty((B, Hkv, capacity), device=device, dtype=torch.float32) for _ in range(2))
    return k, v, ks, vs


def _check_cache(k_cache, v_cache, k_scale, v_scale) -> int:
    """The caches' format, after checks of the four tensors."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [B, Hkv, capacity, D]")
    dt = k_cache.dtype
    if dt not in FORMATS:
        raise TypeError(f"k_cache must be one of {list(FORMATS)}, got {dt}")
    shape = k_cache.shape
    _check(k_cache, "k_cache", shape, dt)
    _check(v_cache, "v_cache", shape, dt)
    if dt == torch.bfloat16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
    else:
        if k_scale is None or v_scale is None:
            raise ValueError(f"a {dt} cache needs k_scale and v_scale")
        _check(k_scale, "k_scale", shape[:3], torch.float32)
        _check(v_scale, "v_scale", shape[:3], torch.float32)
    return FORMATS[dt]


def cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, start: torch.Tensor,
                count: torch.Tensor | None = None, k_scale: torch.Tensor | None = None,
                v_scale: torch.Tensor | None = None) -> None:
    """Write row n of k, v [B,Hkv,N,D] (bf16 views) into slot start[b] + n of
    sequence b, for n < count[b] (int32 [B] tensors; default count: N),
    quantised row by row where the cache holds 8 bits.  Rows whose slot is
    outside the cache are dropped; all other slots stay as they are."""
    fmt = _check_cache(k_cache, v_cache, k_scale, v_scale)
    B, Hkv, cap, D = k_cache.shape
    if k.dim() != 4:
        raise ValueError("k must be [B, Hkv, N, D]")
    N = k.shape[2]
    kr, vr = check_rows(k, "k", (B, Hkv, N, D)), check_rows(v, "v", (B, Hkv, N, D))
    _check(start, "start", (B,), torch.int32)
    if count is not None:
        _check(count, "count", (B,), torch.int32)
    if N == 0:
        return
    dev = _same_device(k, v, k_cache, v_cache, start, count, k_scale, v_scale)
    shp = FaCacheShape(B, Hkv, cap, D, fmt)
    with torch.cuda.device(dev):
        st = _cache_lib().fa_cache_write(ctypes.byref(shp), N, ctypes.byref(kr), ctypes.byref(vr), start.data_ptr(),
                                         _ptr(count), k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scale),
                                         _ptr(v_scale), _stream_ptr(dev))
    if st != FA_OK:
        raise FAError(st, "fa_cache_write")


def cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, n: int | None = None, lens: torch.Tensor | None = None,
               k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
               out_k: torch.Tensor | None = None, out_v: torch.Tensor | None = None):
    """The first n slots (default: all) of every sequence as bf16
    (k [B,Hkv,n,D], v); rows at or behind lens[b] (int32 [B]) are 0."""
    fmt = _check_cache(k_cache, v_cache, k_scale, v_scale)
    B, Hkv, cap, D = k_cache.shape
    n = cap if n is None else int(n)
    if lens is not None:
        _check(lens, "lens", (B,), torch.int32)
    shape = (B, Hkv, n, D)
    out_k = torch.empty(shape, device=k_cache.device, dtype=torch.bfloat16) if out_k is None else out_k
    out_v = torch.empty(shape, device=k_cache.device, dtype=torch.bfloat16) if out_v is None else out_v
    _check(out_k, "out_k", shape)
    _check(out_v, "out_v", shape)
    dev = _same_device(k_cache, v_cache, lens, k_scale, v_scale, out_k, out_v)
    shp = FaCacheShape(B, Hkv, cap, D, fmt)
    with torch.cuda.device(dev):
        st = _cache_lib().fa_cache_read(ctypes.byref(shp), n, _ptr(lens), k_cache.data_ptr(), v_cache.data_ptr(),
                                        _ptr(k_scale), _ptr(v_scale), out_k.data_ptr(), out_v.data_ptr(),
                                        _stream_ptr(dev))
    if st != FA_OK:
        raise FAError(st, "fa_cache_read")
    return out_k, out_v


def decode_cache_workspace_bytes(B, Hq, Hkv, Nq, capacity, D, dtype=torch.bfloat16, n_prefix=0) -> int:
    """Bytes of decode_cache's workspace on the current device."""
    shp = FaCacheDecodeShape(int(B), int(Hq), int(Hkv), int(Nq), int(capacity), int(n_prefix), int(D), FORMATS[dtype],
                             1.0, 1)
    return int(_cache_lib().fa_decode_cache_workspace_bytes(ctypes.byref(shp)))


def decode_cache(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, lens: torch.Tensor,
                 k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                 prefix_k: torch.Tensor | None = None, prefix_v: torch.Tensor | None = None, causal: bool = True,
                 scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None):
    """Attention of Nq new queries q [B,Hq,Nq,D] of each sequence over its
    lens[b] cached slots (int32 [B]; the new tokens' own rows among them), and
    before those over prefix_k, prefix_v [Hkv,Np,D] (bf16), which all sequences
    share and which is read once for the batch.  Query i stands at slot
    lens[b] - Nq + i.  Returns (o [B,Hq,Nq,D] bf16, lse [B,Hq,Nq] fp32); a
    query that sees no key gets 0 and -inf."""
    if q.dim() != 4:
        raise ValueError("q must be [B, Hq, Nq, D]")
    fmt = _check_cache(k_cache, v_cache, k_scale, v_scale)
    _, Hkv, cap, D = k_cache.shape
    B, Hq, Nq, _ = q.shape
    _check(q, "q", (B, Hq, Nq, D))
    if k_cache.shape[0] != B:
        raise ValueError(f"k_cache has {k_cache.shape[0]} sequences, q has {B}")
    _check(lens, "lens", (B,), torch.int32)
    n_prefix = 0
    if prefix_k is not None or prefix_v is not None:
        if prefix_k is None or prefix_v is None:
            raise ValueError("prefix_k and prefix_v come together")
        if prefix_k.dim() != 3:
            raise ValueError("prefix_k must be [Hkv, Np, D]")
        n_prefix = prefix_k.shape[1]
        _check(prefix_k, "prefix_k", (Hkv, n_prefix, D))
        _check(prefix_v, "prefix_v", (Hkv, n_prefix, D))
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32) if lse is None else lse
    _check(out, "out", (B, Hq, Nq, D))
    _check(lse, "lse", (B, Hq, Nq), torch.float32)
    dev = _same_device(q, k_cache, v_cache, lens, k_scale, v_scale, prefix_k, prefix_v, out, lse, workspace)
    shp = FaCacheDecodeShape(B, Hq, Hkv, Nq, cap, n_prefix, D, fmt, scale, 1 if causal else 0)
    with torch.cuda.device(dev):
        L = _cache_lib()
        if workspace is None:
            nbytes = int(L.fa_decode_cache_workspace_bytes(ctypes.byref(shp)))
            workspace = torch.empty(max(nbytes, 256), device=dev, dtype=torch.uint8)
        st = L.fa_decode_cache(ctypes.byref(shp), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scale),
                               _ptr(v_scale), lens.data_ptr(), _ptr(prefix_k), _ptr(prefix_v), out.data_ptr(),
                               lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                               _stream_ptr(dev))
    if st != FA_OK:
        raise FAError(st, "fa_decode_cache")
    return out, lse
