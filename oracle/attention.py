"""Attention-layer operators in fp64 (oracle).

TEST INFRASTRUCTURE (see the package docstring).

The formulas of include/dg.h's dg_qk_norm_rope, dg_cache_write, dg_cache_read
and dg_cache_attention, one token and one head at a time, on numpy arrays. A
paged cache is a dict {(page, head, offset): row}, a batch the lists past[b],
new[b] and the page table.
"""
from __future__ import annotations

import numpy as np

from . import fp8

EXP_MIN, EXP_MAX = -100, 119


def norm_rope(x, weight, positions, inv_freq, interleaved=False, eps=1e-6, offset=0.0):
    """x [tokens, heads, D] normed per head and rotated; also |a| + |b| of each element's pair."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    y = x / np.sqrt((x * x).sum(-1, keepdims=True) / D + eps)
    y = y * ((1.0 if weight is None else np.asarray(weight, np.float64)) + offset)
    out, size = y.copy(), np.abs(y)
    n = len(inv_freq)
    # extended precision: an fp64 product loses 2^-22 radians at positions near 2^31
    t = np.asarray(positions).astype(np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)
    c, s = np.cos(t).astype(np.float64), np.sin(t).astype(np.float64)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        out[..., a] = y[..., a] * c[:, None, i] - y[..., b] * s[:, None, i]
        out[..., b] = y[..., b] * c[:, None, i] + y[..., a] * s[:, None, i]
        size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, size


def quantise(row):
    """(code values, biased exponent) of one row: power-of-two scale from the largest finite
    magnitude, infinities and NaN as NaN."""
    row = np.asarray(row, np.float64)
    fine = np.isfinite(row)
    amax = np.abs(row[fine]).max() if fine.any() else 0.0
    e = int(np.clip(fp8.row_scale_exponent(np.array([amax]))[0], EXP_MIN, EXP_MAX))
    codes = np.full(row.shape, np.nan)
    codes[fine] = fp8.fp8_round(np.ldexp(row[fine], -e), "e4m3")
    return codes, e + 127


def dequantise(codes, exp):
    return np.ldexp(np.asarray(codes, np.float64), int(exp) - 127)


def attend(Q, K, V, seen, scale):
    """Query rows Q [R, D] over the positions each sees (bool [R, L]): (out [R, D], lse [R],
    sum p |v| [R, D], largest sum |q k| scale of each row [R], root of the sum of (p v)^2 over
    keys and columns [R]). What a row does not see is left out of its sums, not multiplied by zero."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        z = np.where(seen, Q @ K.T * scale, -np.inf)
        m = z.max(1, initial=-np.inf)
        p = np.where(seen, np.exp(z - np.where(np.isneginf(m), 0.0, m)[:, None]), 0.0)
        l = p.sum(1)
        p /= np.where(l == 0, 1.0, l)[:, None]
        fine = np.isfinite(V)
        out = p @ np.where(fine, V, 0.0)
        for j in np.flatnonzero(~fine.all(1)):
            out += np.where(seen[:, j, None], p[:, j, None] * np.where(fine[j], 0.0, V[j]), 0.0)
        size = p @ np.abs(np.where(fine, V, 0.0))
        logit = np.where(seen, np.abs(Q) @ np.abs(np.where(np.isfinite(K), K, 0.0)).T * scale, 0.0)
        spread = np.sqrt((p * p) @ (np.where(fine, V, 0.0) ** 2).sum(1))
        return out, m + np.log(l), size, logit.max(1, initial=0.0), spread


def seen_by(i, past, new, mask, words=None):
    """Which of the past + new positions new token i sees."""
    seen = np.ones(past + new, bool)
    node = np.arange(new)
    if mask == "causal":
        seen[past:] = node <= i
    elif mask == "tree":
        for j in node:
            seen[past + j] = j // 32 < len(words) and (int(words[j // 32]) >> (j % 32)) & 1
    return seen
