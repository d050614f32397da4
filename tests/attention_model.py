"""Attention, norm + rotation and eviction in float64 numpy, written from their
definitions, with the error bounds that the GPU tests hold the kernels to.

Bounds (u: unit roundoff of the 16-bit type, 2^-8 for bfloat16 and 2^-11 for
float16; e = 2^-24 that of binary32).  A score sums d exact products in
binary32, in any order: |ds| <= 2 (d + 8) e scale sum |q| A, where A bounds the
magnitudes that are multiplied: |k| for 16-bit rows; for packed rows, whose
codes may be multiplied as integers with an offset and scaled afterwards, four
times the row's range more.  Taking a score to an exponent's argument costs
|s| 2^-22 more.  A weight is then off by a factor exp(2 ds), and is rounded to
the 16-bit type before it meets the values: u sum w B with B = |v| (plus the
row's range for packed rows, whose scale is rounded with the weight), and
2^-24 sum B for float16 weights that fall below its normal range.  The result
is rounded once more: u |o|.
"""
from __future__ import annotations

import numpy as np

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
E = 2.0 ** -24


def visible(p, nk, window, sinks):
    """Which of nk keys a query at place p sees."""
    j = np.arange(nk)
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def attend(q, k, v, see, scale, dtype, k_range=0.0, v_range=0.0):
    """q [d], k, v [n, d], see [n] -> (o, o's bound, lse, lse's bound, w, w's
    bound); rows that are not seen play no part.  *_range: [n] or 0, the ranges
    of packed rows."""
    d = q.shape[0]
    n = k.shape[0]
    w, wb = np.zeros(n), np.zeros(n)
    if not see.any():
        return np.zeros(d), np.zeros(d), -np.inf, 0.0, w, wb
    k, v, q = k[see].astype(np.float64), v[see].astype(np.float64), q.astype(np.float64)
    kr = np.broadcast_to(np.asarray(k_range, np.float64), (n,))[see]
    vr = np.broadcast_to(np.asarray(v_range, np.float64), (n,))[see]
    s = (k @ q) * scale
    ds = 2 * (d + 8) * E * abs(scale) * (np.abs(k) @ np.abs(q) + 4 * kr * np.abs(q).sum())
    ds = ds.max() + 2.0 ** -22 * (np.abs(s).max() + 1)
    m = s.max()
    p = np.exp(s - m)
    ws = p / p.sum()
    rel = np.expm1(2 * ds) + 2.0 ** -20
    b = np.abs(v) + vr[:, None]
    o = ws @ v
    bound = U[dtype] * np.abs(o) + (U[dtype] + rel) * (ws @ b) * (1 + U[dtype]) + 1e-30
    if dtype == "fp16":
        bound += 2.0 ** -24 * b.sum(0) + 2.0 ** -24  # weights and results below the normal range
    w[see], wb[see] = ws, ws * rel + 1e-37
    return o, bound, m + np.log(p.sum()), ds + 2.0 ** -21 * (1 + abs(m)), w, wb


def unpack_rows(rows, dim, bits):
    """Packed rows [.., stride] uint8 -> (values float64 [.., dim], range [..])."""
    n = dim * bits // 8
    par = np.ascontiguousarray(rows[..., n:n + 4]).view(np.float16).astype(np.float64)
    codes = rows[..., :n]
    if bits == 4:
        codes = np.stack((codes & 15, codes >> 4), -1).reshape(rows.shape[:-1] + (dim,))
    return par[..., :1] * codes + par[..., 1:], par[..., 0] * (2 ** bits - 1)


def norm_rope(x, weight, cos, sin, eps, interleaved):
    """x [tokens, heads, d] float64, weight [d], cos / sin [tokens, R / 2]."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    r = cos.shape[1]
    z = y.copy()
    for i in range(r):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        z[..., a] = y[..., a] * cos[:, None, i] - y[..., b] * sin[:, None, i]
        z[..., b] = y[..., b] * cos[:, None, i] + y[..., a] * sin[:, None, i]
    return z


def evict_ids(mass, n, keep, sinks, recent):
    """The slots kept of one sequence and head."""
    if n <= keep:
        return list(range(n))
    m = np.where(np.isnan(mass[:n]), -np.inf, mass[:n])
    middle = sorted(range(sinks, n - recent), key=lambda i: (-m[i], i))[: keep - sinks - recent]
    return list(range(sinks)) + sorted(middle) + list(range(n - recent, n))
