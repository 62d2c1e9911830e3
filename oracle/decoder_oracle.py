"""CPU oracle of the operators between a decoder's linear layers -- TEST
INFRASTRUCTURE ONLY (see the package docstring; no code is shared with the HIP
path). Float64 from the formulas: causal attention of new tokens over cached
ones, rotary positions, the root-mean-square norm with the residual's addition.
"""

from __future__ import annotations

import numpy as np


def attention(q, k, v, scale: float, window: int = 0):
    """One sequence: q [n][Hq][D] are its last n tokens' queries, k, v
    [L][Hk][D] all its tokens. Returns (o [n][Hq][D], weight [n][Hq][D], total
    [n][Hq]): the output, sum_t p_t |v_t| with the softmax weights p_t, and
    sum_t exp(score_t - max score), the last two for error bounds. Rows that
    see no token are zero."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, Hq, D = q.shape
    L, Hk = k.shape[0], k.shape[1]
    o = np.zeros((n, Hq, D))
    wt = np.zeros((n, Hq, D))
    total = np.zeros((n, Hq))
    for i in range(n):
        p = L - n + i
        lo = max(0, p - window + 1) if window > 0 else 0
        if p < lo:
            continue
        for h in range(Hq):
            c = h // (Hq // Hk)
            s = (k[lo:p + 1, c] @ q[i, h]) * scale
            e = np.exp(s - s.max())
            total[i, h] = e.sum()
            w = e / e.sum()
            o[i, h] = w @ v[lo:p + 1, c]
            wt[i, h] = w @ np.abs(v[lo:p + 1, c])
    return o, wt, total


def rope(x, positions, table, rot_dim: int, interleaved: bool):
    """x [T][H][D], table [P][rot_dim / 2][2] of (cos, sin): float64 result."""
    y = np.array(x, np.float64)
    c = np.asarray(table, np.float64)[np.asarray(positions), :, 0][:, None, :]
    s = np.asarray(table, np.float64)[np.asarray(positions), :, 1][:, None, :]
    i = np.arange(rot_dim // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)
    xa, xb = y[..., a].copy(), y[..., b].copy()
    y[..., a] = xa * c - xb * s
    y[..., b] = xb * c + xa * s
    return y


def rope_frequencies(rot_dim: int, base: float) -> np.ndarray:
    """Angle per position of pair i: base^(-2 i / rot_dim)."""
    return np.array([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)])


def rms_norm(x, weight, eps: float, residual=None):
    """(y float64, h float16): h = RNE_fp16(x + residual), y from h."""
    x = np.asarray(x, np.float16)
    h = x if residual is None else (x.astype(np.float64) + np.asarray(residual, np.float64)).astype(np.float16)
    hf = h.astype(np.float64)
    y = hf / np.sqrt((hf * hf).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return y, h
