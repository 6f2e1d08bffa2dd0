"""fp64 reference of the output head's cross entropy and its gradients, from the
formulas in include/moe.h (test infrastructure only; shares no code with the kernels)."""
from __future__ import annotations

import numpy as np


def logits(x, w):
    return np.asarray(x, np.float64) @ np.asarray(w, np.float64).T


def takes_part(target, vocab):
    t = np.asarray(target, np.int64)
    return (t >= 0) & (t < vocab)


def forward(x, w, target):
    """(loss, lse), zero for rows that take no part."""
    vocab = len(w)
    on = takes_part(target, vocab)
    loss, lse = np.zeros(len(x)), np.zeros(len(x))
    if on.any():
        z = logits(np.asarray(x)[on], w)
        top = z.max(1)
        s = top + np.log(np.exp(z - top[:, None]).sum(1))
        lse[on] = s
        loss[on] = s - z[np.arange(len(z)), np.asarray(target)[on]]
    return loss, lse


def probs(x, w, target, lse, dloss):
    """P [rows, vocab]: the logits' gradient of sum(dloss loss)."""
    vocab = len(w)
    on = takes_part(target, vocab)
    p = np.zeros((len(x), vocab))
    if on.any():
        q = np.exp(logits(np.asarray(x)[on], w) - np.asarray(lse, np.float64)[on][:, None])
        q[np.arange(len(q)), np.asarray(target)[on]] -= 1.0
        p[on] = q * np.asarray(dloss, np.float64)[on][:, None]
    return p


def backward(x, w, target, lse, dloss):
    """(dx, dw)."""
    p = probs(x, w, target, lse, dloss)
    x = np.where(takes_part(target, len(w))[:, None], np.asarray(x, np.float64), 0.0)
    return p @ np.asarray(w, np.float64), p.T @ x
