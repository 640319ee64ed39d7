"""RMS norm of the query and key heads with the position rotation, and its
gradient, in float64 (numpy).

TEST INFRASTRUCTURE ONLY.  Shares no code with ``ref`` or the CUDA path.

    n = v / sqrt(mean v^2 + eps) * w, then the pairs (a, b) of n's first rot
    channels become (a cos - b sin, b cos + a sin) at angle positions * freqs,
    paired (i, i + rot/2) or, interleaved, (2i, 2i+1).
"""
from __future__ import annotations

import numpy as np

from .scan import U, f64


def matrix(position, freqs, d, interleaved):
    """The rotation of one position as a d x d matrix."""
    R = np.eye(d)
    half = len(freqs)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(position * freqs[i]), np.sin(position * freqs[i])
        R[a, a], R[a, b], R[b, a], R[b, b] = c, -s, s, c
    return R


def forward(v, positions, freqs, w=None, eps=1e-6, interleaved=False, ulps=32):
    """(out, bound on a float32 evaluation's error), v [T, H, d]."""
    v, freqs, pos = f64(v), f64(freqs), f64(positions)
    w = np.ones(v.shape[-1]) if w is None else f64(w)
    n = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * w
    out, bound = np.zeros_like(n), np.zeros_like(n)
    for t in range(v.shape[0]):
        R = matrix(pos[t], freqs, v.shape[-1], interleaved)
        out[t] = n[t] @ R.T
        bound[t] = ulps * U * (np.abs(n[t]) @ (R != 0).T.astype(float))
    return out, bound


def backward(v, dout, positions, freqs, w=None, eps=1e-6, interleaved=False, ulps=32):
    """(dv, dweight, bound of dv, bound of dweight)."""
    v, dout, freqs, pos = f64(v), f64(dout), f64(freqs), f64(positions)
    d = v.shape[-1]
    w = np.ones(d) if w is None else f64(w)
    r = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    b, e_b = np.zeros_like(dout), np.zeros_like(dout)
    for t in range(v.shape[0]):
        R = matrix(pos[t], freqs, d, interleaved)
        b[t] = dout[t] @ R
        e_b[t] = ulps * U * (np.abs(dout[t]) @ (R != 0).astype(float))
    c, e_c = b * w, e_b * np.abs(w)
    dv = r * (c - v * r * r * (c * v).mean(-1, keepdims=True))
    e_dv = r * (e_c + ulps * U * np.abs(c) + np.abs(v) * r * r *
                (e_c * np.abs(v) + 2 * ulps * U * np.abs(c * v)).mean(-1, keepdims=True))
    dw = (b * v * r).sum((0, 1))
    e_dw = ((e_b + 2 * ulps * U * np.abs(b)) * np.abs(v) * r).sum((0, 1))
    return dv, dw, e_dv, e_dw
