"""Token-sequence operators in float64 numpy: per-head RMS norm with the rotary
position, attention of packed sequences, and the paged cache with its 8-bit rows.

Plain loops over sequences and heads, from the formulas; no code shared with the
library."""
from __future__ import annotations

import numpy as np


def norm_rope(x, gain=None, eps=1e-6, positions=None, inv_freq=None, interleaved=False, mscale=1.0):
    """``x[T,H,D]`` -> normalised and rotated heads."""
    y = np.array(x, np.float64)
    if gain is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    if inv_freq is None:
        return y
    half = len(inv_freq)
    ang = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang)[:, None] * mscale, np.sin(ang)[:, None] * mscale
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    out = y.copy()
    out[..., ia] = y[..., ia] * c - y[..., ib] * s
    out[..., ib] = y[..., ia] * s + y[..., ib] * c
    return out


def attention(q, k, v, causal, scale):
    """One sequence: ``q[n,Hq,D]``, ``k, v [m,Hk,D]`` -> out ``[n,Hq,D]``, log of the sums ``[n,Hq]``."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, Hq, D = q.shape
    m, Hk = k.shape[:2]
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    for i in range(n):
        seen = min(m, max(0, m - n + i + 1)) if causal else m
        if seen == 0:
            continue
        for h in range(Hq):
            kv = h // (Hq // Hk)
            s = k[:seen, kv] @ q[i, h] * scale
            top = s.max()
            p = np.exp(s - top)
            out[i, h] = p @ v[:seen, kv] / p.sum()
            lse[i, h] = top + np.log(p.sum())
    return out, lse


def packed(q, k, v, cu_q, cu_k, causal, scale):
    """Sequences packed by offsets; rows outside them NaN."""
    out = np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    for b in range(len(cu_q) - 1):
        rows = slice(cu_q[b], cu_q[b + 1])
        out[rows], lse[rows] = attention(q[rows], k[cu_k[b]:cu_k[b + 1]], v[cu_k[b]:cu_k[b + 1]], causal, scale)
    return out, lse


# ----------------------------------------------------------------- 8-bit rows

def _e4m3_values():
    """The 128 non-negative codes' values (code 127 is NaN): exponent bias 7, 3 fraction bits."""
    v = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(128)])
    v[127] = np.nan
    return v


E4M3 = _e4m3_values()


def e4m3_decode(codes):
    c = np.asarray(codes, np.uint8)
    return np.where(c & 128, -1.0, 1.0) * E4M3[c & 127]


def e4m3_encode(x):
    """Nearest code, ties to the even one (the codes are ordered, so evenness is the code's)."""
    a = np.abs(np.asarray(x, np.float64))
    hi = np.clip(np.searchsorted(E4M3[:127], a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    c = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (a >= E4M3[126]), hi, lo).astype(np.uint8)
    c = np.where(np.isnan(a), 127, c).astype(np.uint8)
    return c | np.where(np.signbit(x), 128, 0).astype(np.uint8)


def quantise_row(x):
    """Codes and scale byte of one row: the smallest e in [-100, 119] with max |x| <= 448 2^e (0 for a zero row)."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    m = np.abs(x[fin]).max() if fin.any() else 0.0
    e = -100
    if m == 0:
        e = 0
    while e < 119 and m > 448 * 2.0 ** e:
        e += 1
    return e4m3_encode(np.where(fin, x * 2.0 ** -e, np.nan)), e + 127


def quantise(x):
    """``x[..., D]`` -> (codes, scale bytes)."""
    flat = np.asarray(x, np.float64).reshape(-1, np.shape(x)[-1])
    rows = [quantise_row(r) for r in flat]
    return (np.array([r[0] for r in rows], np.uint8).reshape(np.shape(x)),
            np.array([r[1] for r in rows], np.uint8).reshape(np.shape(x)[:-1]))


def dequantise(codes, scales):
    return e4m3_decode(codes) * 2.0 ** (np.asarray(scales, np.float64)[..., None] - 127)
