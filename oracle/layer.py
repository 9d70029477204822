"""Oracle of the operators between the quantised products, in numpy float64:
norms around a block, rotary positions, row quantisation and attention of
drafted tokens over cached rows.  Written from the formulas of the header's
comments, one row or one query at a time; nothing is shared with the kernels.
"""
from __future__ import annotations

import numpy as np


def norm_rows(t, weight, bias, kind, eps, offset=0.0):
    t = np.asarray(t, np.float64)
    if kind == "layer":
        t = t - t.mean(axis=1, keepdims=True)
    t = t / np.sqrt((t * t).mean(axis=1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + offset)
    return t if bias is None else t + bias


def block_norm(residual, x, *, weight=None, bias=None, kind="rms", post_weight=None, post_bias=None, gate=None,
               block_scale=1.0, residual_scale=1.0, eps=1e-6, weight_offset=0.0):
    """(h, y); y is None without a weight."""
    h = 0.0
    if x is not None:
        b = np.asarray(x, np.float64)
        if post_weight is not None:
            b = norm_rows(b, post_weight, post_bias, kind, eps, weight_offset)
        h = block_scale * (b if gate is None else b * np.asarray(gate, np.float64))
    if residual is not None:
        h = h + residual_scale * np.asarray(residual, np.float64)
    return h, None if weight is None else norm_rows(h, weight, bias, kind, eps, weight_offset)


def rotate(x, positions, frequency, interleaved, magnitude=1.0):
    """x [T, H, D], its first 2 len(frequency) channels rotated, one pair at a time."""
    x = np.array(x, np.float64)
    out = x.copy()
    half = len(frequency)
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        angle = np.asarray(positions, np.float64) * frequency[j]
        c, s = np.cos(angle)[:, None] * magnitude, np.sin(angle)[:, None] * magnitude
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def row_scales(x, top):
    """amax / top over the last axis; 1 for a zero row, NaN for one with a NaN or an infinity."""
    amax = np.abs(x).max(axis=-1)
    s = np.where(amax > 0, amax / top, 1.0)
    return np.where(np.isfinite(x).all(axis=-1), s, np.nan)


def visible(n, length, i, mask_row=None):
    """Which of `length` positions drafted token i of n sees; mask_row: truth values over drafted tokens."""
    see = np.zeros(length, bool)
    for p in range(length):
        j = p - (length - n)
        if j < 0:
            see[p] = True
        elif mask_row is None:
            see[p] = j <= i
        else:
            see[p] = j < len(mask_row) and bool(mask_row[j])
    return see


def attend_one(q, k, v, scale, see):
    """One query [D] over keys and values [L, D]: (out, lse, sum of p |v|)."""
    if not see.any():
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1])
    k, v = k[see], v[see]
    z = scale * (k @ q)
    top = z.max()
    p = np.exp(z - top)
    total = p.sum()
    return (p @ v) / total, top + np.log(total), (p @ np.abs(v)) / total
