"""Float64 references of the experts in 16 bits, their gradients and the
low-rank adapters (numpy; shares no code with the kernels).  Every function
also gives the sum of magnitudes behind each result, which bounds what a
32-bit accumulation in any order may be off by.
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def segments(offsets):
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]


def product(w, a, offsets):
    """w [E][N][K], grouped rows a [M][K] -> y [M][N], magnitudes."""
    y = np.zeros((a.shape[0], w.shape[1]))
    m = np.zeros_like(y)
    for e, s0, s1 in segments(offsets):
        y[s0:s1] = a[s0:s1] @ w[e].T
        m[s0:s1] = np.abs(a[s0:s1]) @ np.abs(w[e]).T
    return y, m


def swiglu(y):
    g, u = np.split(y, 2, axis=1)
    return g * sigmoid(g) * u


def grad_rows(w, dy, offsets):
    """w [E][N][K], dy [M][N] -> da [M][K], magnitudes."""
    return product(np.swapaxes(w, 1, 2), dy, offsets)


def swiglu_grad(dh, pre):
    """Gradient by what enters the SwiGLU from the one by its output."""
    g, u = np.split(pre, 2, axis=1)
    s = sigmoid(g)
    return np.concatenate([dh * u * (s + g * s * (1 - s)), dh * g * s], axis=1)


def grad_weights(dy, a, offsets):
    """dy [M][N], grouped rows a [M][K] -> dw [E][N][K], magnitudes."""
    E = len(offsets) - 1
    dw = np.zeros((E, dy.shape[1], a.shape[1]))
    m = np.zeros_like(dw)
    for e, s0, s1 in segments(offsets):
        dw[e] = dy[s0:s1].T @ a[s0:s1]
        m[e] = np.abs(dy[s0:s1]).T @ np.abs(a[s0:s1])
    return dw, m


def combine_grad(dout, y, pos, w, n_valid, ids=None, E=0):
    """dout [T][H], y [P][H], pos and w [T][k] -> (dy, dw, magnitudes of dw, dlogits)."""
    T, k = pos.shape
    dy, dw, m = np.zeros(y.shape), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = pos[t, j]
            if 0 <= p < n_valid:
                dy[p] = w[t, j] * dout[t]
                dw[t, j] = y[p] @ dout[t]
                m[t, j] = np.abs(y[p]) @ np.abs(dout[t])
    dl = None
    if ids is not None:
        dl = np.zeros((T, E))
        for t in range(T):
            for j in range(k):
                if 0 <= pos[t, j] < n_valid and 0 <= ids[t, j] < E:
                    dl[t, ids[t, j]] += w[t, j] * (dw[t, j] - w[t] @ dw[t])
    return dy, dw, m, dl


def adapters(y, x, A, B, ids, scale):
    """Tokens' adapters ids [T] (outside [0, n): none) -> out [T][N], magnitudes of v = A x and of B v, |scale| included."""
    out, mag = y.copy(), np.zeros_like(y)
    for t, a in enumerate(ids):
        if 0 <= a < A.shape[0]:
            out[t] = y[t] + scale[a] * (B[a] @ (A[a] @ x[t]))
            mag[t] = abs(scale[a]) * (np.abs(B[a]) @ (np.abs(A[a]) @ np.abs(x[t])))
    return out, mag
