"""Gated linear recurrence, its gradients, and the gradient of the input
prologue, in float64 (numpy).

TEST INFRASTRUCTURE ONLY.  Shares no code with ``ref`` or the CUDA path.

Per channel c of each packed sequence (s = sigmoid(e^A z)):

    z:  a = exp(-5 s),  h_t = a_t h_{t-1} + (1 - a_t) x_t
    g:  a = exp(g),     h_t = a_t h_{t-1} + x_t

Every function also returns, next to each value, a bound on the error of a
float32 evaluation: ``ulps`` units of 2^-24 relative to the magnitude of the
terms of every operation, carried through the recurrence by the recurrence
itself (an error of h_{t-1} reaches h_t times a_t).
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def f64(x):
    if hasattr(x, "detach"):
        x = x.detach().cpu().double().numpy()
    return np.asarray(x, np.float64)


def sigmoid(u):
    e = np.exp(-np.abs(u))
    return np.where(u >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def gate(z=None, A=None, g=None):
    """(a, input scale, sigmoid or None)."""
    if g is not None:
        a = np.exp(f64(g))
        return a, np.ones_like(a), None
    s = sigmoid(np.exp(f64(A)) * f64(z))
    return np.exp(-5.0 * s), -np.expm1(-5.0 * s), s


def forward(x, cu, *, z=None, A=None, g=None, h0=None, ulps=32):
    """dict of y (unrounded), h_final, prev (the state before each token), and
    of their bounds e_y, e_h_final, e_prev."""
    x = f64(x)
    T, C = x.shape
    N = len(cu) - 1
    a, m, _ = gate(z, A, g)
    h0 = np.zeros((N, C)) if h0 is None else f64(h0)
    y, prev, e_y, e_prev = (np.zeros((T, C)) for _ in range(4))
    h_final, e_final = h0.copy(), np.zeros((N, C))
    for n in range(N):
        h, e = h0[n], np.zeros(C)
        for t in range(cu[n], cu[n + 1]):
            prev[t], e_prev[t] = h, e
            e = a[t] * e + ulps * U * (a[t] * np.abs(h) + m[t] * np.abs(x[t]))
            h = a[t] * h + m[t] * x[t]
            y[t], e_y[t] = h, e
        h_final[n], e_final[n] = h, e
    return dict(y=y, h_final=h_final, prev=prev, e_y=e_y, e_h_final=e_final, e_prev=e_prev)


def backward(x, cu, dy, *, z=None, A=None, g=None, h0=None, dh_final=None, ulps=32):
    """dict of dx, dz and dA (or dg), dh0, and of their bounds e_*."""
    f = forward(x, cu, z=z, A=A, g=g, h0=h0, ulps=ulps)
    x, dy = f64(x), f64(dy)
    T, C = x.shape
    N = len(cu) - 1
    a, m, s = gate(z, A, g)
    dh = np.zeros((N, C)) if dh_final is None else f64(dh_final)
    lam, e_lam = np.zeros((T, C)), np.zeros((T, C))
    dh0, e_dh0 = dh.copy(), np.zeros((N, C))
    for n in range(N):
        back, e = dh[n], np.zeros(C)
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            lam[t] = dy[t] + back
            e_lam[t] = e + ulps * U * (np.abs(dy[t]) + np.abs(back))
            back, e = a[t] * lam[t], a[t] * e_lam[t]
        dh0[n], e_dh0[n] = back, e + ulps * U * np.abs(back)
    out = dict(dh0=dh0, e_dh0=e_dh0, dx=m * lam, e_dx=m * (e_lam + ulps * U * np.abs(lam)))
    if g is not None:
        out.update(dg=lam * a * f["prev"],
                   e_dg=a * (e_lam * np.abs(f["prev"]) + np.abs(lam) * f["e_prev"] +
                             ulps * U * np.abs(lam * f["prev"])))
        return out
    # 1 - s as sigmoid(-u): the difference is 0 from u = 37 on, where e^-u is not
    slope = 5.0 * s * sigmoid(-np.exp(f64(A)) * f64(z)) * np.exp(f64(A))
    d = f["prev"] - x
    dz = -lam * a * d * slope
    e_dz = a * slope * (e_lam * np.abs(d) +
                        np.abs(lam) * (f["e_prev"] +
                                       ulps * U * (np.abs(f["prev"]) + np.abs(x))))
    zz = f64(z)
    out.update(dz=dz, e_dz=e_dz, dA=(dz * zz).sum(0),
               e_dA=(e_dz * np.abs(zz)).sum(0) + 2 * ulps * U * np.abs(dz * zz).sum(0))
    return out


def conv_backward(x, w, cu, dy, ulps=32):
    """dict of dx, dw of the input prologue and of their bounds."""
    x, w, dy = f64(x), f64(w), f64(dy)
    T, C = x.shape
    W = w.shape[1]
    dx, e_dx, dw, e_dw = np.zeros((T, C)), np.zeros((T, C)), np.zeros((C, W)), np.zeros((C, W))
    for n in range(len(cu) - 1):
        lo, hi = cu[n], cu[n + 1]
        for t in range(lo, hi):
            taps = [j for j in range(W) if t - j >= lo]      # x[t-j] under w[W-1-j]
            u = sum(w[:, W - 1 - j] * x[t - j] for j in taps)
            e_u = ulps * U * sum(np.abs(w[:, W - 1 - j] * x[t - j]) for j in taps)
            p = sigmoid(u)
            du = dy[t] * p * (1.0 + u * (1.0 - p))
            # |d/du (p (1 + u (1 - p)))| <= 1/2
            e_du = np.abs(dy[t]) * (0.5 * e_u + ulps * U * p * (1.0 + np.abs(u) * (1.0 - p)))
            for j in taps:
                dx[t - j] += w[:, W - 1 - j] * du
                e_dx[t - j] += np.abs(w[:, W - 1 - j]) * (e_du + ulps * U * np.abs(du))
                dw[:, W - 1 - j] += du * x[t - j]
                e_dw[:, W - 1 - j] += np.abs(x[t - j]) * (e_du + 2 * ulps * U * np.abs(du))
    return dict(dx=dx, dw=dw, e_dx=e_dx, e_dw=e_dw)
