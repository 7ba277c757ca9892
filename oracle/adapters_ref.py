"""Float64 reference of the adapter products, their gradients and the
distillation loss.  Test infrastructure only, as the rest of the package.

Rows are activations: X [n, d], dY [n, m]; W_hat [m, d]; adapters A
[L, rank, d], B [L, m, rank], alpha [L]; ids [n], outside [0, L) for rows
without an adapter.
"""

from __future__ import annotations

import numpy as np

__all__ = ["lora_matmul", "lora_backward", "distill", "distill_targets"]


def _rows_of(ids, count):
    ids = np.asarray(ids)
    return [np.nonzero(ids == a)[0] for a in range(count)]


def lora_matmul(X, W_hat, A, B, alpha, ids):
    """(Y, H): Y = X W_hat^T + alpha_a H B_a^T, H = X A_a^T."""
    X, W_hat, A, B = (np.asarray(v, dtype=np.float64) for v in (X, W_hat, A, B))
    Y = X @ W_hat.T
    H = np.zeros((X.shape[0], A.shape[1]))
    for a, rows in enumerate(_rows_of(ids, A.shape[0])):
        H[rows] = X[rows] @ A[a].T
        Y[rows] += float(alpha[a]) * (H[rows] @ B[a].T)
    return Y, H


def lora_backward(dY, X, H, W_hat, A, B, alpha, ids):
    """(dX, dA, dB) of sum(dY * Y); H as the forward pass kept it."""
    dY, X, H, W_hat, A, B = (np.asarray(v, dtype=np.float64) for v in (dY, X, H, W_hat, A, B))
    dX = dY @ W_hat
    dA, dB = np.zeros_like(A), np.zeros_like(B)
    for a, rows in enumerate(_rows_of(ids, A.shape[0])):
        G = float(alpha[a]) * (dY[rows] @ B[a])
        dX[rows] += G @ A[a]
        dA[a] = G.T @ X[rows]
        dB[a] = float(alpha[a]) * (dY[rows].T @ H[rows])
    return dX, dA, dB


def distill_targets(ids, t_logits, vocab, temperature, t_lse=None):
    """One row's known ids (distinct, sorted), the teacher's probability of
    each, and what is left for the rest (0 without t_lse)."""
    ids = np.asarray(ids)
    ok = (ids >= 0) & (ids < vocab)
    ids, t = ids[ok], np.asarray(t_logits, dtype=np.float64)[ok] / temperature
    if t_lse is not None:
        p = np.exp(t - float(t_lse))
        rest = max(0.0, 1.0 - p.sum())
    else:
        top = t.max() if len(t) else 0.0
        e = np.exp(t - top) if np.isfinite(top) else np.zeros_like(t)
        p = e / e.sum() if e.sum() > 0 else e
        rest = 0.0
    known = np.unique(ids)
    return known, np.array([p[ids == v].sum() for v in known]), rest, p, ids


def _lse(z):
    top = z.max() if z.size else -np.inf
    return top + np.log(np.exp(z - top).sum()) if np.isfinite(top) else top


def distill(logits, t_idx, t_logits, temperature=1.0, t_lse=None, weight=None):
    """(loss [n], d sum(loss) / d logits [n, vocab]), the definition row by row:
    T^2 sum p (log p - log q) over the known ids and, with t_lse, the class
    of all others (unless the student has no mass there)."""
    logits = np.asarray(logits, dtype=np.float64)
    n, vocab = logits.shape
    loss, grad = np.zeros(n), np.zeros((n, vocab))
    for k in range(n):
        w = 1.0 if weight is None else float(weight[k])
        if w == 0.0:
            continue
        z = logits[k] / temperature
        known, p_of, rest, p, ids = distill_targets(t_idx[k], t_logits[k], vocab, temperature,
                                                    None if t_lse is None else t_lse[k])
        if t_lse is None and p.sum() == 0.0:
            continue
        lse = _lse(z)
        q = np.exp(z - lse)
        with np.errstate(divide="ignore"):
            terms = [pi * (np.log(pi) - (z[v] - lse)) for pi, v in zip(p, ids) if pi > 0]
        value = float(np.sum(terms))
        out = np.ones(vocab, dtype=bool)
        out[known] = False
        lse_rest = _lse(z[out])
        # what the target's probabilities add up to: 1, but for a class left out
        mass = 1.0
        if t_lse is not None and not (rest > 0 and np.isfinite(lse_rest)):
            rest, mass = 0.0, p.sum()
        d = mass * q
        if t_lse is not None and np.isfinite(lse_rest):
            q_rest = np.exp(lse_rest - lse)
            if rest > 0:
                value += rest * (np.log(rest) - (lse_rest - lse))
            d[out] = np.exp(z[out] - lse_rest) * (mass * q_rest - rest)
        d[known] -= p_of
        loss[k] = w * temperature ** 2 * value
        grad[k] = w * temperature * d
    return loss, grad
