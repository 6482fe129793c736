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
import functools
import math
import os

import torch

from ._args import on_device, raw_stream, want
from .attention import FA_OK, FAError, lib, symbols_in
from .rope import FaRows, check_rows

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


def _check_cache(k_cache, v_cache, k_scale, v_scale):
    """(format, address of k_scale, of v_scale) after checks of the four tensors."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [B, Hkv, capacity, D]")
    dt = k_cache.dtype
    fmt = FORMATS.get(dt)
    if fmt is None:
        raise TypeError(f"k_cache must be one of {list(FORMATS)}, got {dt}")
    shape = k_cache.shape
    want(k_cache, "k_cache", shape, dt, k_cache)
    want(v_cache, "v_cache", shape, dt, k_cache)
    if fmt == 0:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
        return 0, None, None
    if k_scale is None or v_scale is None:
        raise ValueError(f"a {dt} cache needs k_scale and v_scale")
    want(k_scale, "k_scale", shape[:3], torch.float32, k_cache)
    want(v_scale, "v_scale", shape[:3], torch.float32, k_cache)
    return fmt, k_scale.data_ptr(), v_scale.data_ptr()


def cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, start: torch.Tensor,
                count: torch.Tensor | None = None, k_scale: torch.Tensor | None = None,
                v_scale: torch.Tensor | None = None) -> None:
    """Write row n of k, v [B,Hkv,N,D] (bf16 views) into slot start[b] + n of
    sequence b, for n < count[b] (int32 [B] tensors; default count: N),
    quantised row by row where the cache holds 8 bits.  Rows whose slot is
    outside the cache are dropped; all other slots stay as they are."""
    fmt, ks, vs = _check_cache(k_cache, v_cache, k_scale, v_scale)
    B, Hkv, cap, D = k_cache.shape
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be [B, Hkv, N, D]")
    N = k.shape[2]
    if N > 0x7FFFFFFF:       # (a broadcast view; more than the C side's int holds)
        raise ValueError(f"k has {N} rows a head, more than 2^31 - 1")
    shape = (B, Hkv, N, D)
    kr, vr = check_rows(k, "k", shape, k_cache), check_rows(v, "v", shape, k_cache)
    want(start, "start", (B,), torch.int32, k_cache)
    if count is not None:
        want(count, "count", (B,), torch.int32, k_cache)
    if N == 0:
        return
    index = k_cache.get_device()
    guard = on_device(index)
    if guard is not None:
        with guard:
            return cache_write(k, v, k_cache, v_cache, start, count, k_scale, v_scale)
    shp = FaCacheShape(B, Hkv, cap, D, fmt)
    st = _cache_lib().fa_cache_write(ctypes.byref(shp), N, ctypes.byref(kr), ctypes.byref(vr), start.data_ptr(),
                                     None if count is None else count.data_ptr(), k_cache.data_ptr(),
                                     v_cache.data_ptr(), ks, vs, raw_stream(index))
    if st != FA_OK:
        raise FAError(st, "fa_cache_write")


def cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, n: int | None = None, lens: torch.Tensor | None = None,
               k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
               out_k: torch.Tensor | None = None, out_v: torch.Tensor | None = None):
    """The first n slots (default: all) of every sequence as bf16
    (k [B,Hkv,n,D], v); rows at or behind lens[b] (int32 [B]) are 0."""
    fmt, ks, vs = _check_cache(k_cache, v_cache, k_scale, v_scale)
    B, Hkv, cap, D = k_cache.shape
    n = cap if n is None else int(n)
    if lens is not None:
        want(lens, "lens", (B,), torch.int32, k_cache)
    shape = (B, Hkv, n, D)
    index = k_cache.get_device()
    guard = on_device(index)
    if guard is not None:
        with guard:
            return cache_read(k_cache, v_cache, n, lens, k_scale, v_scale, out_k, out_v)
    if out_k is None:
        out_k = torch.empty(shape, dtype=torch.bfloat16, device=k_cache.device)
    else:
        want(out_k, "out_k", shape, torch.bfloat16, k_cache)
    if out_v is None:
        out_v = torch.empty(shape, dtype=torch.bfloat16, device=k_cache.device)
    else:
        want(out_v, "out_v", shape, torch.bfloat16, k_cache)
    if n == 0:
        return out_k, out_v
    shp = FaCacheShape(B, Hkv, cap, D, fmt)
    st = _cache_lib().fa_cache_read(ctypes.byref(shp), n, None if lens is None else lens.data_ptr(),
                                    k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, out_k.data_ptr(),
                                    out_v.data_ptr(), raw_stream(index))
    if st != FA_OK:
        raise FAError(st, "fa_cache_read")
    return out_k, out_v


@functools.lru_cache(maxsize=1024)
def _decode_shape(index, *fields):
    """The C shape and its workspace on device `index`."""
    shp = FaCacheDecodeShape(*fields)
    return shp, int(_cache_lib().fa_decode_cache_workspace_bytes(ctypes.byref(shp)))


def decode_cache_workspace_bytes(B, Hq, Hkv, Nq, capacity, D, dtype=torch.bfloat16, n_prefix=0) -> int:
    """Bytes of decode_cache's workspace on the current device (0: none needed)."""
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
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [B, Hq, Nq, D]")
    fmt, ks, vs = _check_cache(k_cache, v_cache, k_scale, v_scale)
    _, Hkv, cap, D = k_cache.shape
    B, Hq, Nq, _ = q.shape
    want(q, "q", (B, Hq, Nq, D), torch.bfloat16, k_cache)
    if k_cache.shape[0] != B:
        raise ValueError(f"k_cache has {k_cache.shape[0]} sequences, q has {B}")
    want(lens, "lens", (B,), torch.int32, k_cache)
    n_prefix, pk, pv = 0, None, None
    if prefix_k is not None or prefix_v is not None:
        if prefix_k is None or prefix_v is None:
            raise ValueError("prefix_k and prefix_v come together")
        if not isinstance(prefix_k, torch.Tensor) or prefix_k.dim() != 3:
            raise ValueError("prefix_k must be [Hkv, Np, D]")
        n_prefix = prefix_k.shape[1]
        want(prefix_k, "prefix_k", (Hkv, n_prefix, D), torch.bfloat16, k_cache)
        want(prefix_v, "prefix_v", (Hkv, n_prefix, D), torch.bfloat16, k_cache)
        pk, pv = prefix_k.data_ptr(), prefix_v.data_ptr()
    index = k_cache.get_device()
    guard = on_device(index)
    if guard is not None:
        with guard:
            return decode_cache(q, k_cache, v_cache, lens, k_scale, v_scale, prefix_k, prefix_v, causal, scale, out,
                                lse, workspace)
    if out is None:
        out = torch.empty_like(q)
    else:
        want(out, "out", (B, Hq, Nq, D), torch.bfloat16, k_cache)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    else:
        want(lse, "lse", (B, Hq, Nq), torch.float32, k_cache)
    shp, nbytes = _decode_shape(index, B, Hq, Hkv, Nq, cap, n_prefix, D, fmt,
                                1.0 / math.sqrt(D) if scale is None else float(scale), 1 if causal else 0)
    ws = None
    if workspace is None:
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    else:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous buffer on {q.device}")
        nbytes = workspace.numel() * workspace.element_size()
        ws = workspace.data_ptr()
    st = _cache_lib().fa_decode_cache(ctypes.byref(shp), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ks, vs,
                                      lens.data_ptr(), pk, pv, out.data_ptr(), lse.data_ptr(), ws, nbytes,
                                      raw_stream(index))
    if st != FA_OK:
        raise FAError(st, "fa_decode_cache")
    return out, lse
