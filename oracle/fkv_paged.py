"""Float64 restatement of the paged-cache operators, from their definitions.

numpy, one query row at a time; shares no code with the CUDA library.  Besides
each result, the attention returns what a rounding analysis needs: the mean of
|v| under the same weights, and a bound on the fp32 error of a score.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24  # largest relative rounding error of one fp32 operation


def norm_rope(x, *, weight=None, eps=1e-6, norm=True, omega=(), positions=None, axis_pairs=None,
              style="interleaved"):
    """Rows x [tokens][heads][D] normed and rotated.  Returns (y, mag): mag is
    |y_a| + |y_b| of the pair before the turn (|y| elsewhere), the scale of the
    fp32 errors."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    if norm:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps)
        if weight is not None:
            y = y * np.asarray(weight, dtype=np.float64)
    mag = np.abs(y)
    out = y.copy()
    n = len(omega)
    axis = np.repeat(np.arange(len(axis_pairs)), axis_pairs) if axis_pairs is not None else np.zeros(n, int)
    for i in range(n):
        a, b = (i, i + n) if style == "half" else (2 * i, 2 * i + 1)
        ang = np.asarray(positions[axis[i]], dtype=np.float64) * float(omega[i])
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., a] * s + y[..., b] * c
        mag[..., a] = mag[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, mag


def cache_rows(cache, table_row, n):
    """Positions 0..n-1 of a sequence: [heads][n][D] from [pages][heads][rows][D]."""
    ps = cache.shape[2]
    if n == 0:
        return np.zeros((cache.shape[1], 0, cache.shape[3]))
    return np.concatenate([cache[int(table_row[p])] for p in range((n + ps - 1) // ps)], axis=1)[:, :n]


def visible(kv, pos, *, causal, window, prefix):
    j = np.arange(kv)
    near = np.ones(kv, bool)
    if causal:
        near &= j <= pos
    if window:
        near &= j > pos - window
    return near | (j < prefix)


def attend_row(q, k, v, pos, *, scale, cap=0.0, slope=0.0, causal=True, window=0, prefix=0):
    """One query row over k, v [n][D].  Returns (out, lse, mean |v|, score
    error bound, visible keys)."""
    see = np.nonzero(visible(len(k), pos, causal=causal, window=window, prefix=prefix))[0]
    D = k.shape[-1] if k.ndim == 2 else 0
    if len(see) == 0:
        z = np.zeros(v.shape[-1])
        return z, -np.inf, z, 0.0, 0
    k, v = k[see].astype(np.float64), v[see].astype(np.float64)
    q = q.astype(np.float64)
    raw = k @ q * scale
    z = cap * np.tanh(raw / cap) if cap else raw
    dist = slope * (see - pos)
    # fp32: the D products and sums of q.k, its scaling; the cap, relative to the
    # smaller of c and the score (the tanh within 9 roundings, the factors that
    # enclose it and a shared reciprocal within 10; 3 in fp32); the distance term and
    # the sum; log2 e
    dz = (D + 4) * U32 * np.max(np.abs(k) @ np.abs(q)) * scale
    dz += 32 * U32 * min(cap, np.max(np.abs(raw))) if cap else 8 * U32 * np.max(np.abs(raw))
    dz += 4 * U32 * np.max(np.abs(dist)) + 4 * U32 * np.max(np.abs(z + dist))
    z = z + dist
    m = z.max()
    e = np.exp(z - m)
    p = e / e.sum()
    return p @ v, m + np.log(e.sum()), p @ np.abs(v), dz, len(see)
