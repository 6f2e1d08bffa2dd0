"""fp64 reference of the two ends of a training step: the pre-norm with its
backward pass, and the orthogonalised update of a weight matrix.

Written from the formulas in include/moe.h; shares no code with the kernels.
"""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

A, B, C = 3.4445, -4.7750, 2.0315


def norm_forward(kind: str, s: np.ndarray, gamma=None, beta=None, eps: float = 1e-6):
    """(y, mean, rstd) of the rows of s (the sum with the residual, where there is one)."""
    s = np.asarray(s, np.float64)
    mean = s.mean(1) if kind == "layer" else np.zeros(s.shape[0])
    c = s - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + float(np.float32(eps)))
    y = c * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    if beta is not None:
        y = y + np.asarray(beta, np.float64)
    return y, mean, rstd


def norm_backward(kind: str, dy, s, gamma, mean, rstd, dsum=None):
    """(ds, dgamma, dbeta) from the statistics of the forward pass."""
    dy, s = np.asarray(dy, np.float64), np.asarray(s, np.float64)
    h = (s - (np.asarray(mean, np.float64)[:, None] if kind == "layer" else 0.0)) * np.asarray(rstd, np.float64)[:, None]
    t = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    ds = t - h * (t * h).mean(1, keepdims=True)
    if kind == "layer":
        ds = ds - t.mean(1, keepdims=True)
    ds = ds * np.asarray(rstd, np.float64)[:, None]
    if dsum is not None:
        ds = ds + np.asarray(dsum, np.float64)
    return ds, (dy * h).sum(0), dy.sum(0)


def update_of(g, momentum=None, mu: float = 0.0, nesterov: bool = True) -> Tuple[np.ndarray, Optional[np.ndarray]]:
    """The update before it is orthogonalised, and the momentum after it."""
    g = np.asarray(g, np.float64)
    if momentum is None:
        return g, None
    mu = float(np.float32(mu))
    m = mu * np.asarray(momentum, np.float64) + g
    return (g + mu * m if nesterov else m), m


def orthogonalize(u, steps: int = 5, eps: float = 1e-7, scale: float = 1.0) -> np.ndarray:
    """Newton-Schulz steps on one matrix [rows, cols]."""
    u = np.asarray(u, np.float64)
    n = np.sqrt((u * u).sum()) + float(np.float32(eps))
    x = u / n if n > 0 else np.zeros_like(u)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for _ in range(steps):
        r = x @ x.T
        x = A * x + (B * r + C * (r @ r)) @ x
    return scale * (x.T if tall else x)
