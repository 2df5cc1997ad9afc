"""Oracle: router top-K with the load-balance and z losses and the losses' gradient, token by token in
float64 (test infrastructure only).

Selection: descending by value, equal values by ascending expert, NaN above every number, a masked expert
(-inf) takes no slot (id -1, score 0).  Losses, over sequences s of n_s tokens (n in all):

  balance = alpha sum_s (n_s / n) sum_e f_se P_se,   f_se = E c_se / (K n_s),   P_se = 1 / n_s sum_t p_te
  z       = beta / n sum_t logsumexp(l_t)^2

The gradient is the Jacobian product of each token's softmax with the loss's partial derivatives, the counts
being constants.
"""
from __future__ import annotations

import numpy as np

SOFTMAX_OVER_TOPK, TOPK_OVER_SOFTMAX, TOPK = 0, 1, 2


def _softmax(v):
    """Softmax and logsumexp; all zeros and -inf where every entry is -inf."""
    m = np.max(v)
    if m == -np.inf:
        return np.zeros_like(v), -np.inf
    e = np.exp(v - m)
    return e / e.sum(), m + np.log(e.sum())


def _sequences(T, seg):
    seg = [0, T] if seg is None else [int(i) for i in seg]
    owner = np.full(T, -1)
    for s in range(len(seg) - 1):
        owner[seg[s]:seg[s + 1]] = s
    return owner, len(seg) - 1


def topk(logits, K, seg=None):
    """ids [T, K] (-1: unused slot)."""
    T, E = logits.shape
    owner, _ = _sequences(T, seg)
    ids = np.full((T, K), -1, dtype=np.int32)
    for t in range(T):
        if owner[t] < 0:
            continue
        rank = sorted(range(E), key=lambda e: (not np.isnan(logits[t, e]),
                                               0.0 if np.isnan(logits[t, e]) else -logits[t, e], e))
        for k, e in enumerate(rank[:K]):
            if logits[t, e] != -np.inf:
                ids[t, k] = e
    return ids


def scores(mode, logits, ids, renorm=False):
    lg = np.asarray(logits, dtype=np.float64)
    out = np.zeros(ids.shape)
    for t in range(len(lg)):
        ok = ids[t] >= 0
        sel = ids[t, ok]
        if mode == TOPK:
            out[t, ok] = lg[t, sel]
        elif mode == TOPK_OVER_SOFTMAX and not renorm:
            out[t, ok] = _softmax(lg[t])[0][sel]
        elif ok.any():
            out[t, ok] = _softmax(lg[t, sel])[0]
    return out


def losses(logits, ids, alpha, beta, seg=None):
    """dict(lse, counts, prob_sum, loss)."""
    lg = np.asarray(logits, dtype=np.float64)
    T, E = lg.shape
    K = ids.shape[1]
    owner, S = _sequences(T, seg)
    counts, prob, lse = np.zeros((S, E), dtype=np.int64), np.zeros((S, E)), np.full(T, -np.inf)
    length = np.array([(owner == s).sum() for s in range(S)])
    n = max(1, int(length.sum()))
    z = 0.0
    for t in range(T):
        if owner[t] < 0:
            continue
        p, lse[t] = _softmax(lg[t])
        prob[owner[t]] += p
        if lse[t] != -np.inf:
            z += lse[t] ** 2
        for e in ids[t]:
            if 0 <= e < E:
                counts[owner[t], e] += 1
    bal = 0.0
    for s in range(S):
        if length[s]:
            bal += length[s] / n * np.sum(E * counts[s] / (K * length[s]) * prob[s] / length[s])
    return dict(lse=lse, counts=counts, prob_sum=prob, loss=np.array([alpha * bal, beta / n * z]))


def gradient(logits, counts, K, alpha, beta, dloss=(1.0, 1.0), seg=None, add=None):
    lg = np.asarray(logits, dtype=np.float64)
    T, E = lg.shape
    owner, S = _sequences(T, seg)
    length = np.array([(owner == s).sum() for s in range(S)])
    n = max(1, int(length.sum()))
    out = np.zeros((T, E)) if add is None else np.array(add, dtype=np.float64)
    for t in range(T):
        s = owner[t]
        if s < 0 or np.all(lg[t] == -np.inf):
            continue
        p, lse = _softmax(lg[t])
        J = np.diag(p) - np.outer(p, p)
        out[t] += dloss[0] * alpha * E / (K * n * length[s]) * (J @ counts[s])
        out[t] += dloss[1] * beta / n * 2 * lse * p
    return out
