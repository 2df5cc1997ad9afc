"""Oracle: layer normalisation and its RMS form, forward and backward, per row in float64 (test
infrastructure only).  The backward is written as the row's Jacobian product, not as the closed form:

  y_i = n_i gamma_i + beta_i,   n = (s - mu) / sigma,   sigma = sqrt(mean((s - mu)^2) + eps)
  dn_i / ds_j = (delta_ij - [mean] 1/H - n_i n_j / H) / sigma
"""
from __future__ import annotations

import numpy as np

LAYER, RMS = 0, 1


def _stats(s, kind, eps):
    mu = s.mean() if kind == LAYER else 0.0
    return mu, np.sqrt(np.mean((s - mu) ** 2) + eps)


def forward(x, gamma, beta, eps, kind=LAYER):
    """(y, mean, rstd) of rows x [T, H]."""
    x = np.asarray(x, dtype=np.float64)
    y, mean, rstd = np.empty_like(x), np.empty(len(x)), np.empty(len(x))
    for t, s in enumerate(x):
        mu, sigma = _stats(s, kind, eps)
        y[t] = (s - mu) / sigma * gamma + (0.0 if beta is None else beta)
        mean[t], rstd[t] = mu, 1.0 / sigma
    return y, mean, rstd


def backward(dy, x, gamma, eps, kind=LAYER, dres=None):
    """(dx, dgamma, dbeta) for the loss <dy, y> plus <dres, x>."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    H = x.shape[1]
    dx, dgamma = np.zeros_like(x), np.zeros(H)
    for t, s in enumerate(x):
        mu, sigma = _stats(s, kind, eps)
        n = (s - mu) / sigma
        J = (np.eye(H) - (1.0 / H if kind == LAYER else 0.0) - np.outer(n, n) / H) / sigma   # J[i, j] = dn_i / ds_j
        dx[t] = J.T @ (dy[t] * gamma)
        dgamma += dy[t] * n
    if dres is not None:
        dx = dx + dres
    return dx, dgamma, dy.sum(0)
