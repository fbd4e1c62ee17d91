"""Plain numpy forms, in float64, of the serving operators: per-head norm and position rotation, the 8-bit row
format, and attention of drafted tokens over a cache.  Test infrastructure only; shares no code with the GPU path.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100


def e4m3_table() -> np.ndarray:
    """The values of the 256 e4m3 codes (bias 7, no infinities, two NaN codes)."""
    out = np.empty(256)
    for code in range(256):
        sign = -1.0 if code & 0x80 else 1.0
        e, m = (code >> 3) & 0xF, code & 7
        if e == 15 and m == 7:
            out[code] = np.nan
        else:
            out[code] = sign * (2.0 ** -6 * m / 8 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8))
    return out


TABLE = e4m3_table()


def norm(x: np.ndarray, w, eps: float) -> np.ndarray:
    """x * w / sqrt(mean(x^2) + eps) over the last axis."""
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return y if w is None else y * w


def rotate(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [..., T, h, d] turned pair by pair by positions[..., T] * inv_freq."""
    rot = 2 * len(inv_freq)
    out = x.copy()
    for i, f in enumerate(inv_freq):
        a = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        angle = positions.astype(np.float64) * float(f)
        c, s = np.cos(angle)[..., None], np.sin(angle)[..., None]
        out[..., a[0]] = x[..., a[0]] * c - x[..., a[1]] * s
        out[..., a[1]] = x[..., a[1]] * c + x[..., a[0]] * s
    return out


def row_scale(x: np.ndarray) -> np.ndarray:
    """max(amax, 2^-100) / 448 of every row (last axis)."""
    return np.maximum(np.abs(x).max(axis=-1), AMAX_FLOOR) / E4M3_MAX


def attend(q, K, V, prefix: int, n: int, masks, tau=None):
    """One batch row.  q [T, h_q, d], K [h_k, cap, d], V [h_v, cap, d]; masks: T integers or None (u <= t).
    Returns out [n, h_q, d] and the smallest distance of any visible score from its threshold (inf without)."""
    T, h_q, d = q.shape
    h_k, h_v = K.shape[0], V.shape[0]
    out = np.zeros((n, h_q, d))
    border = np.inf
    for t in range(n):
        word = (1 << (t + 1)) - 1 if masks is None else int(masks[t])
        rows = list(range(prefix)) + [prefix + u for u in range(n) if word >> u & 1]
        if not rows:
            continue
        for j in range(h_q):
            a = K[j * h_k // h_q, rows] @ q[t, j] / np.sqrt(d)
            keep = np.ones(len(rows), bool)
            if tau is not None:
                keep = a >= tau[j]
                if np.isfinite(tau[j]):
                    border = min(border, float(np.abs(a - tau[j]).min()))
            if keep.any():
                p = np.exp(a[keep] - a[keep].max())
                out[t, j] = (p / p.sum()) @ V[j * h_v // h_q, rows][keep]
    return out, border
