"""Plain 64-bit forms of the operators around selection (``include/sel.h``):
the 4-bit output head, sampling of 16-bit rows with a policy per row, and the
embedding lookup. Inputs are numpy arrays that hold the 16-bit values exactly
(float64), so nothing is rounded here; written from the definitions, with no
code of the kernels."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

INVALID = 0xFFFFFFFF


def dequantise(q, scales, zeros, group):
    """[V, H] float64 entries s * (q - z): byte i of a row holds column 2 i in
    its low nibble and 2 i + 1 in its high one; z is a byte's low four bits."""
    V, half = q.shape
    w = np.empty((V, 2 * half))
    w[:, 0::2] = q & 15
    w[:, 1::2] = q >> 4
    z = np.full(scales.shape, 8.0) if zeros is None else (zeros & 15).astype(np.float64)
    return (w - np.repeat(z, group, axis=1)) * np.repeat(scales, group, axis=1)


def head_w4(x, q, scales, zeros, group):
    """(logits, sum of the terms' magnitudes), both [rows, V] float64."""
    w = dequantise(q, scales, zeros, group)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def embed(ids, table, scale):
    out = np.zeros((ids.size, table.shape[1]))
    ok = ids < table.shape[0]
    out[ok] = table[ids[ok]] * scale
    return out


def sample16_row(x, T, top_k, top_p, min_p, u):
    """(id, probability) of one row by sorting it; INVALID and NaN when the
    row, its policy or its uniform is out of range."""
    bad = INVALID, np.nan
    if not (T >= 0 and np.isfinite(T) and 0 < top_p <= 1 and 0 <= min_p < 1 and 0 <= u < 1):
        return bad
    if np.isnan(x).any() or (x == np.inf).any() or not np.isfinite(x).any():
        return bad
    order = np.lexsort((np.arange(x.size), -x))
    order = order[np.isfinite(x[order])]
    if T == 0:
        return int(order[0]), 1.0
    z = x[order]
    with np.errstate(over="ignore"):
        w = np.exp((z - z[0]) / T)
    n = min(top_k, order.size) if top_k else order.size
    cum = np.cumsum(w.astype(np.longdouble))
    Z = cum[n - 1]
    cut = n
    if top_p < 1:
        cut = min(cut, int(np.sum(cum < np.longdouble(top_p) * Z)) + 1)
    cut = min(cut, int(np.sum(w >= min_p)))
    Zs = cum[cut - 1]
    i = min(int(np.sum(cum <= np.longdouble(u) * Zs)), cut - 1)
    return int(order[i]), float(w[i] / Zs)


def sample16(x, T, top_k, top_p, min_p, u):
    got = [sample16_row(x[r], float(T[r]), int(top_k[r]), float(top_p[r]), float(min_p[r]), float(u[r]))
           for r in range(len(x))]
    return np.array([g[0] for g in got], dtype=np.uint32), np.array([g[1] for g in got])


def sample16_row_exact(x, top_k, top_p, u):
    """sample16_row for rows whose finite logits are all equal (every weight is
    1), in rationals: the borders of the cuts and of the draw fall exactly on ids."""
    ids = np.flatnonzero(np.isfinite(x))
    n = min(top_k, ids.size) if top_k else ids.size
    keep = -((-Fraction(top_p) * n) // 1)  # smallest whole number reaching top_p * n
    n = min(n, max(1, int(keep)))
    return int(ids[min(n - 1, int((Fraction(u) * n) // 1))]), 1.0 / n
