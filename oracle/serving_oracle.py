"""fp64 definitions of the operators around the attention: per-head norm with
rotation, quantised cache rows, decoding over a cache with a shared prefix.
Test infrastructure only, plain NumPy, one row or one sequence at a time where
that is the plainest."""
from __future__ import annotations

import numpy as np

from .attention_oracle import _f64


def rope_angles(positions, inv_freq):
    """[..., rotary_dim / 2] angles."""
    return np.asarray(positions, dtype=np.float64)[..., None] * _f64(inv_freq)


def reduced_angles(positions, inv_freq):
    """rope_angles modulo a turn, in [-pi, pi], for products of any size: the
    turns are formed in integers of 2^-400."""
    one = 1 << 400

    def arctan_inverse(x):   # Machin: pi = 16 arctan(1/5) - 4 arctan(1/239)
        term, total, n = one // x, 0, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    out = np.zeros(np.shape(positions) + (len(inv_freq),))
    for i, f in enumerate(np.asarray(inv_freq, dtype=np.float64).tolist()):
        num, den = f.as_integer_ratio()
        rate = one * one * num // (2 * pi * den)
        for at in np.ndindex(*np.shape(positions)):
            turn = rate * int(positions[at]) % one
            out[at + (i,)] = 2 * np.pi * ((turn - one if 2 * turn >= one else turn) / one)
    return out


def rotate(u, ang, interleaved: bool, inverse: bool = False):
    """Rows u [..., D] with the pairs of the first 2 * ang.shape[-1] values turned by ang [..., R / 2]."""
    y = np.array(u, dtype=np.float64)
    half = ang.shape[-1]
    lo = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    hi = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    c, s = np.cos(ang), np.sin(ang) * (-1.0 if inverse else 1.0)
    a, b = y[..., lo].copy(), y[..., hi].copy()
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    return y


def norm_rope(x, w, inv_freq, positions, eps: float, interleaved: bool, angles=rope_angles):
    """x [B,H,N,D], w [D], positions [B,N] -> (y, u): rotated and unrotated normed rows."""
    x, w = _f64(x), _f64(w)
    u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rotate(u, angles(positions, inv_freq)[:, None], interleaved), u


def norm_rope_backward(dy, x, w, inv_freq, positions, eps: float, interleaved: bool, angles=rope_angles):
    """(dx, dw, size_dx, size_dw): gradients and, for error bounds, the sums of
    magnitudes that they come from."""
    dy, x, w = _f64(dy), _f64(x), _f64(w)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    ang = angles(positions, inv_freq)[:, None]
    g = rotate(dy, ang, interleaved, inverse=True)
    dw = (g * xh).sum((0, 1, 2))
    h = g * w
    dx = r * (h - xh * (h * xh).mean(-1, keepdims=True))
    gmag = np.abs(rotate(np.abs(dy), np.zeros_like(ang), interleaved))
    half = ang.shape[-1]
    lo = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    hi = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    both = gmag[..., lo] + gmag[..., hi]
    gmag[..., lo], gmag[..., hi] = both, both.copy()
    hm = gmag * np.abs(w)
    size_dx = r * (hm + np.abs(xh) * (hm * np.abs(xh)).mean(-1, keepdims=True))
    return dx, dw, size_dx, (gmag * np.abs(xh)).sum((0, 1, 2))


def round_e4m3(y):
    """Nearest e4m3 value (ties to even), |y| <= 448."""
    mag = np.abs(y)
    e = np.floor(np.log2(np.maximum(mag, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.rint(y / step) * step


def quantise_rows(x, fmt: str):
    """(codes as values, scale [...]) of rows x [..., D]; fmt "e4m3" or "int8"."""
    x = _f64(x)
    amax = np.abs(x).max(-1)
    bad = ~np.isfinite(amax)
    safe = np.where(bad, 0.0, amax)
    if fmt == "int8":
        scale = np.maximum((safe.astype(np.float32) / np.float32(127.0)).astype(np.float64), 2.0 ** -120)
    else:
        scale = 2.0 ** np.full(safe.shape, -120.0)
        for e in range(-119, 121):
            scale = np.where(safe > 448.0 * scale, 2.0 ** e, scale)
    xs = np.where(bad[..., None], 0.0, x) / scale[..., None]
    codes = np.rint(xs) if fmt == "int8" else round_e4m3(xs)
    return codes, np.where(bad, np.nan, scale)


def decode_rows(q, keys, values, scale: float, visible):
    """One query row q [D] over keys [n, D], values [n, D] that are visible
    (bool [n]).  Returns (o, lse, sum_j p_j |v_j|, max_j sum_d |q_d k_jd| * scale)."""
    k, v = keys[visible], values[visible]
    if k.shape[0] == 0:
        return np.zeros_like(q), -np.inf, np.zeros_like(q), 0.0
    s = (k @ q) * scale
    m = s.max()
    e = np.exp(s - m)
    p = e / e.sum()
    return p @ v, m + np.log(e.sum()), p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * scale)


def decode_cache(q, k, v, lens, scale: float, causal: bool, prefix_k=None, prefix_v=None):
    """q [B,Hq,Nq,D] over the first lens[b] rows of k, v [B,Hkv,cap,D] behind
    prefix_k, prefix_v [Hkv,Np,D].  Returns (o, lse, weight, size): as
    decode_rows, for every query."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Hq, Nq, D = q.shape
    Hkv, cap = k.shape[1], k.shape[2]
    pk = _f64(prefix_k) if prefix_k is not None else np.zeros((Hkv, 0, D))
    pv = _f64(prefix_v) if prefix_v is not None else np.zeros((Hkv, 0, D))
    o, wt = np.zeros_like(q), np.zeros_like(q)
    lse, size = np.zeros((B, Hq, Nq)), np.zeros((B, Hq, Nq))
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            keys = np.concatenate([pk[g], k[b, g, :n]])
            vals = np.concatenate([pv[g], v[b, g, :n]])
            for i in range(Nq):
                own = np.arange(n) <= (n - Nq + i if causal else n - 1)
                visible = np.concatenate([np.ones(pk.shape[1], dtype=bool), own])
                o[b, h, i], lse[b, h, i], wt[b, h, i], size[b, h, i] = decode_rows(q[b, h, i], keys, vals, scale, visible)
    return o, lse, wt, size
