"""Float64 oracle of the losses at the output head: cross entropy and distillation
from a teacher's top logits, with their gradients.  Plain numpy, shares no code with
the CUDA library."""

import numpy as np


def entries(indices, logits, vocab, tau):
    """(there, p, log p) of [T][K] entries: p the softmax of logits / tau over the row's
    entries that are there (indices in the vocabulary, logits above -inf)."""
    there = (indices >= 0) & (indices < vocab) & ~(logits == -np.inf)
    s = np.where(there, logits, -np.inf)
    top = np.max(s, 1, keepdims=True)
    d = np.where(there, (s - np.where(there.any(1, keepdims=True), top, 0.0)) / tau, -np.inf)
    total = np.exp(d).sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        log_p = np.where(there, d - np.log(total), 0.0)
    return there, np.where(there, np.exp(log_p), 0.0), log_p


def head_loss(x, W, indices, logits, weights, tau):
    """(loss, total, dx, dW, more): indices [T][K]; more: what error bounds need."""
    T, V = x.shape[0], W.shape[0]
    there, p, log_p = entries(indices, logits, V, tau)
    on = there.any(1)
    rows = np.flatnonzero(on)
    w = np.zeros(T)
    w[rows] = weights[rows] if weights is not None else 1.0 / max(1, len(rows))
    loss, dx, dW = np.zeros(T), np.zeros(x.shape), np.zeros(W.shape)
    u = x[rows] @ W.T / tau
    top = u.max(1, keepdims=True) if len(rows) else np.zeros((0, 1))
    lse = top + np.log(np.exp(u - top).sum(1, keepdims=True))
    q = np.exp(u - lse)
    P = np.zeros(u.shape)
    for n, t in enumerate(rows):
        k = np.flatnonzero(there[t])
        i = indices[t, k]
        np.add.at(P[n], i, p[t, k])
        loss[t] = tau ** 2 * np.sum(p[t, k] * (log_p[t, k] - u[n, i] + lse[n, 0]))
    dz = (w[rows] * tau)[:, None] * (q - P)
    dx[rows] = dz @ W
    dW += dz.T @ x[rows]
    return loss, float(np.sum(w * loss)), dx, dW, dict(rows=rows, w=w, u=u, q=q, P=P, dz=dz, p=p,
                                                       log_p=log_p, there=there)


def cross_entropy(x, W, targets, weights):
    return head_loss(x, W, targets[:, None], np.zeros((len(targets), 1)), weights, 1.0)
