"""Float64 oracle of low-rank adapters: y_t = base_t + scale_a B_a^T A_a x_t for token t of adapter a = ids[t] (-1: none)."""
import numpy as np


def forward(x, A, B, ids, scale, base):
    """y and u."""
    y, u = base.copy(), np.zeros((x.shape[0], A.shape[1]))
    for t, a in enumerate(ids):
        if a >= 0:
            u[t] = A[a] @ x[t]
            y[t] += scale[a] * (u[t] @ B[a])
    return y, u


def backward(dy, x, u, A, B, ids, scale, base):
    """dx, dA, dB."""
    dx, dA, dB = base.copy(), np.zeros_like(A), np.zeros_like(B)
    for a in range(A.shape[0]):
        rows = np.flatnonzero(np.asarray(ids) == a)
        v = scale[a] * (dy[rows] @ B[a].T)
        dx[rows] += v @ A[a]
        dA[a] = v.T @ x[rows]
        dB[a] = scale[a] * (u[rows].T @ dy[rows])
    return dx, dA, dB
