"""Float64 references of the scored routing, the MX rows and the residual RMS
norm (numpy; shares no code with the kernels).

MX rows here are element values and scale exponents; `pack` gives the stored
bytes.  Element tables are enumerated from the formats' definitions (sign,
exponent and mantissa fields of the OCP Microscaling element types), and
rounding is a search for the nearest table entry, ties to the even code.
"""
from __future__ import annotations

import numpy as np

E4M3, E2M1 = 1, 2


def _table(ebits: int, mbits: int, bias: int, n: int) -> np.ndarray:
    out = []
    for c in range(n):
        e, m = c >> mbits, c & ((1 << mbits) - 1)
        f = m / (1 << mbits)
        out.append((1 + f) * 2.0 ** (e - bias) if e else f * 2.0 ** (1 - bias))
    return np.array(out)


TABLE = {E4M3: _table(4, 3, 7, 127), E2M1: _table(2, 1, 1, 8)}  # magnitudes by code (0x7f of e4m3 is NaN)
TOP = {E4M3: 448.0, E2M1: 6.0}


def nearest_code(a: np.ndarray, fmt: int) -> np.ndarray:
    """Code of the nearest magnitude of a >= 0, ties to the even code."""
    t = TABLE[fmt]
    hi = np.clip(np.searchsorted(t, a), 1, len(t) - 1)
    lo = hi - 1
    dl, dh = a - t[lo], t[hi] - a
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def scale_exponent(m: np.ndarray, fmt: int) -> np.ndarray:
    """Smallest p >= -126 with m <= TOP * 2^p (finite m >= 0)."""
    f, e = np.frexp(m / TOP[fmt])  # m / TOP = f * 2^e, 0.5 <= f < 1 (division of a float32 by 448 or 6 in float64)
    p = np.where(f == 0.5, e - 1, e)
    # the quotient may round onto a power of two: settle by exact products
    p = np.where(TOP[fmt] * np.exp2(p.astype(np.float64)) < m, p + 1, p)
    p = np.where(TOP[fmt] * np.exp2(p.astype(np.float64) - 1) >= m, p - 1, p)
    return np.where(m == 0, -126, np.maximum(p, -126)).astype(np.int64)


def quantize(x: np.ndarray, fmt: int):
    """x [..., K] -> (codes [..., K] with sign bit, scale bytes [..., K/32])."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    p = scale_exponent(np.abs(b).max(-1), fmt)
    u = b / np.exp2(p.astype(np.float64))[..., None]
    sign = np.signbit(u) & ~bad[..., None]
    codes = nearest_code(np.abs(u), fmt) | (sign.astype(np.int64) << (7 if fmt == E4M3 else 3))
    return codes.reshape(x.shape), np.where(bad, 255, p + 127)


def values(codes: np.ndarray, scales: np.ndarray, fmt: int) -> np.ndarray:
    bit = 7 if fmt == E4M3 else 3
    codes = np.asarray(codes, np.int64)
    mag = codes & ((1 << bit) - 1)
    t = np.append(TABLE[fmt], np.nan) if fmt == E4M3 else TABLE[fmt]
    el = t[mag] * np.where(codes >> bit, -1.0, 1.0)
    s = np.where(np.asarray(scales) == 255, np.nan, np.exp2(np.asarray(scales, np.float64) - 127))
    return el * np.repeat(s, 32, -1)


def pack(codes: np.ndarray, fmt: int) -> np.ndarray:
    c = np.asarray(codes, np.uint8)
    return c if fmt == E4M3 else c[..., 0::2] | (c[..., 1::2] << 4)


def unpack(b: np.ndarray, fmt: int) -> np.ndarray:
    b = np.asarray(b, np.uint8)
    return b.astype(np.int64) if fmt == E4M3 else np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1).astype(np.int64)


def rmsnorm(v: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    """v [..., H] float64 (the rounded sum) -> v / sqrt(mean v^2 + eps) * weight."""
    v = np.asarray(v, np.float64)
    return v / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def route_scored(logits, k, sigmoid=False, bias=None, n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
    """ids int64 [T][k] (-1: no eligible expert left), weights float64 [T][k]; one token at a time."""
    logits = np.asarray(logits, np.float32)
    T, E = logits.shape
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        barred = np.isnan(logits[t]) | np.isneginf(logits[t])
        x = np.where(barred, 0.0, np.minimum(logits[t], np.finfo(np.float32).max).astype(np.float64))
        if sigmoid:
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-x))
        else:
            top = x[~barred].max() if (~barred).any() else 0.0
            e = np.where(barred, 0.0, np.exp(np.where(barred, -1.0, x - top)))
            s = e / e.sum() if e.sum() > 0 else e
        s = np.where(barred, 0.0, s)
        c = s + (np.asarray(bias, np.float64) if bias is not None else 0.0)
        barred = barred | np.isnan(c) | np.isneginf(c)
        c = np.where(barred, -np.inf, c)
        if n_group > 1:
            by = c.reshape(n_group, -1)
            gs = np.array([np.sum(np.sort(g[g > -np.inf])[::-1][:group_top]) if (g > -np.inf).any() else -np.inf for g in by])
            order = sorted(range(n_group), key=lambda g: (-gs[g], g))[:topk_group]
            for g in range(n_group):
                if g not in order:
                    by[g] = -np.inf
        order = sorted((e for e in range(E) if c[e] > -np.inf), key=lambda e: (-c[e], e))[:k]
        ids[t, : len(order)] = order
        w[t, : len(order)] = s[order]
        total = w[t].sum() if renorm else 1.0
        w[t] = w[t] / total * scale if total > 0 else 0.0
    return ids, w
