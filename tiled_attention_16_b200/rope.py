"""Per-head norm of queries and keys with the position rotation, in one pass:
the binding of include/fa_rope.h (argument marshalling only).

The rows come from the projection as strided views, usually
``qkv.view(B, N, Hq + 2 * Hkv, D)[:, :, :Hq].transpose(1, 2)``, and leave in
the contiguous [B, H, N, D] layout that ``attention.fwd``, ``attention.decode``
and ``cache.cache_write`` take.  There is no fallback: if the library is
missing or the device is not a B200 the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from ._args import on_device, raw_stream, want
from .attention import FA_OK, FAError, lib, symbols_in

HEADER_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fa_rope.h")


class FaRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_longlong), ("stride_h", ctypes.c_longlong),
                ("stride_n", ctypes.c_longlong)]


class FaRopeShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("N", ctypes.c_int),
                ("D", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("eps", ctypes.c_float), ("weight_bf16", ctypes.c_int)]


_lib = None


def _rope_lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = lib()
        vp = ctypes.c_void_p
        shp, rows = ctypes.POINTER(FaRopeShape), ctypes.POINTER(FaRows)
        L.fa_qk_norm_rope.argtypes = [shp, rows, rows, vp, vp, vp, vp, vp, vp, vp]
        L.fa_qk_norm_rope.restype = ctypes.c_int
        L.fa_qk_norm_rope_bwd_workspace_bytes.argtypes = [shp]
        L.fa_qk_norm_rope_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.fa_qk_norm_rope_bwd.argtypes = [shp, vp, vp, rows, rows, vp, vp, vp, vp, rows, rows, vp, vp, vp,
                                          ctypes.c_size_t, vp]
        L.fa_qk_norm_rope_bwd.restype = ctypes.c_int
        _lib = L
    return _lib


def declared_symbols() -> list[str]:
    """Entry points declared in include/fa_rope.h (FA_API functions)."""
    return symbols_in(HEADER_PATH)


def check_rows(t: torch.Tensor, name: str, shape, first: torch.Tensor | None = None) -> FaRows:
    """A bf16 CUDA view [B, H, N, D] whose rows of D values are contiguous, on
    the device of `first`, as the C side takes it (which checks alignment,
    strides and, for views that are written, overlap)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU path)")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if first is not None and t.get_device() != first.get_device():
        raise ValueError(f"all tensors must be on one device: got {first.device} and {t.device}")
    sb, sh, sn, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must have contiguous rows (last stride 1, got {sd})")
    return FaRows(t.data_ptr(), sb, sh, sn)


def _common(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved):
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor) or q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, H, N, D]")
    B, Hq, N, D = q.shape
    Hkv = k.shape[1]
    qr, kr = check_rows(q, "q", (B, Hq, N, D)), check_rows(k, "k", (B, Hkv, N, D), q)
    wt = getattr(q_weight, "dtype", None)
    if wt != torch.float32 and wt != torch.bfloat16:
        raise TypeError(f"q_weight must be torch.bfloat16 or torch.float32, got {wt}")
    want(q_weight, "q_weight", (D,), wt, q)
    want(k_weight, "k_weight", (D,), wt, q)
    rot = 0
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor):
            raise TypeError("inv_freq must be a torch.Tensor")
        rot = 2 * inv_freq.numel()
        want(inv_freq, "inv_freq", (rot // 2,), torch.float32, q)
    if positions is not None:
        want(positions, "positions", (B, N), torch.int32, q)
    return (FaRopeShape(B, Hq, Hkv, N, D, rot, 1 if interleaved else 0, eps, 1 if wt == torch.bfloat16 else 0), qr, kr,
            q_weight.data_ptr(), k_weight.data_ptr(), inv_freq.data_ptr() if rot else None,
            None if positions is None else positions.data_ptr())


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                 inv_freq: torch.Tensor | None, positions: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, out_q: torch.Tensor | None = None, out_k: torch.Tensor | None = None):
    """RMS norm of every head of q [B,Hq,N,D] and k [B,Hkv,N,D] (bf16 views),
    times its weight [D] (bf16 or fp32), rotated by the angles
    positions[b, n] * inv_freq[i] (fp32, half as many as the values that
    rotate; None: no rotation).  positions: int32 [B,N], default 0 .. N-1.
    Pairs are (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved.
    Returns contiguous (q_out, k_out), bf16."""
    shp, qr, kr, qw, kw, freq, pos = _common(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved)
    if out_q is None:
        out_q = q.new_empty(q.shape)
    else:
        want(out_q, "out_q", q.shape, torch.bfloat16, q)
    if out_k is None:
        out_k = k.new_empty(k.shape)
    else:
        want(out_k, "out_k", k.shape, torch.bfloat16, q)
    index = q.get_device()
    guard = on_device(index)
    if guard is not None:
        with guard:
            return qk_norm_rope(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, out_q, out_k)
    st = _rope_lib().fa_qk_norm_rope(ctypes.byref(shp), ctypes.byref(qr), ctypes.byref(kr), qw, kw, freq, pos,
                                     out_q.data_ptr(), out_k.data_ptr(), raw_stream(index))
    if st != FA_OK:
        raise FAError(st, "fa_qk_norm_rope")
    return out_q, out_k


def qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                     q_weight: torch.Tensor, k_weight: torch.Tensor, inv_freq: torch.Tensor | None,
                     positions: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                     dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None):
    """Gradients of qk_norm_rope: dq_out, dk_out are those of its outputs
    (contiguous, as attention.bwd returns them).  Returns (dq, dk, dq_weight,
    dk_weight): dq, dk bf16 [B,H,N,D] views, token-major in memory unless views
    are given (of a packed gradient, for instance); the weights' gradients
    fp32 [D], summed in a fixed order."""
    shp, qr, kr, qw, kw, freq, pos = _common(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved)
    want(dq_out, "dq_out", q.shape, torch.bfloat16, q)
    want(dk_out, "dk_out", k.shape, torch.bfloat16, q)
    D, dev = q.shape[3], q.device
    if dq is None:
        dq = _token_major(q.shape, dev)
    if dk is None:
        dk = _token_major(k.shape, dev)
    dqr, dkr = check_rows(dq, "dq", q.shape, q), check_rows(dk, "dk", k.shape, q)
    index = q.get_device()
    guard = on_device(index)
    if guard is not None:
        with guard:
            return qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved,
                                    dq, dk, workspace)
    L = _rope_lib()
    dqw = torch.empty(D, dtype=torch.float32, device=dev)
    dkw = torch.empty(D, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(_bwd_workspace(D, index), dtype=torch.uint8, device=dev)
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous buffer on {q.device}")
    st = L.fa_qk_norm_rope_bwd(ctypes.byref(shp), dq_out.data_ptr(), dk_out.data_ptr(), ctypes.byref(qr),
                               ctypes.byref(kr), qw, kw, freq, pos, ctypes.byref(dqr), ctypes.byref(dkr),
                               dqw.data_ptr(), dkw.data_ptr(), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), raw_stream(index))
    if st != FA_OK:
        raise FAError(st, "fa_qk_norm_rope_bwd")
    return dq, dk, dqw, dkw


def _token_major(shape, device) -> torch.Tensor:
    """A [B, H, N, D] view with the tokens' heads side by side in memory."""
    B, H, N, D = shape
    return torch.empty_strided((B, H, N, D), (N * H * D, D, H * D, 1), dtype=torch.bfloat16, device=device)


@functools.lru_cache(maxsize=None)
def _bwd_workspace(D: int, index: int) -> int:
    """At least 256, so that a refused head dimension is the library's to report."""
    return max(qk_norm_rope_bwd_workspace_bytes(D), 256)


def qk_norm_rope_bwd_workspace_bytes(D: int) -> int:
    """Bytes of the backward's workspace on the current device (any B, N, heads)."""
    shp = FaRopeShape(1, 1, 1, 1, int(D), 0, 0, 1e-6, 0)
    return int(_rope_lib().fa_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(shp)))
