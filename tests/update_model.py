"""The roundings of the orthogonalised update, in NumPy: what its error against
64 bits comes from, and so what a test of it may allow.

Every product runs on fp16 operands with wider sums.  Rounded to fp16 are x (the
low part, rounded again, enters the elementwise part only), and R, Q and the
products of a pair off their diagonals.  The last rounding, of the output to
bf16, is 1.66e-3 of the norm by itself (its half step 2^-8 times 0.43, the rms
of a uniform rounding of normally distributed values).

CASES are the inputs whose tolerance is pinned: `bound` is 1.15 to 1.3 times
what the model gives, less than what it gives without the choices that the
kernels make for accuracy (see test_update_model_cpu.py).
"""
from dataclasses import dataclass

import numpy as np

from oracle import update_oracle as U

A, B, C = np.float32(U.A), np.float32(U.B), np.float32(U.C)


@dataclass(frozen=True)
class Case:
    count: int
    rows: int
    cols: int
    rank: int
    bound: float
    steps: int = 5
    noise: float = 0.0
    decay: float = 0.0          # the outer products' weights go down to 10^-decay
    dtype: str = "bf16"
    pair: bool = False          # the first two steps share one product

    @property
    def name(self):
        return f"{self.count}x{self.rows}x{self.cols} rank {self.rank} steps {self.steps}" + (" noise" if self.noise else "") + f" {self.dtype}"


CASES = [
    # a weight gradient of 128 tokens; nearly rank one; few tokens on small, middle and large matrices
    Case(1, 1024, 2048, 128, 2.3e-3, decay=1.5, pair=True),
    Case(64, 256, 1024, 1, 2.3e-3, noise=1e-3, dtype="f32", pair=True),
    Case(1, 256, 1024, 1, 2.3e-3, noise=1e-3, dtype="f32"),
    Case(64, 32, 32, 16, 2.6e-3),
    Case(64, 8, 8, 4, 3.1e-3),
    Case(64, 16, 200, 8, 2.7e-3),
    Case(64, 200, 16, 8, 2.7e-3),
    Case(64, 64, 64, 64, 2.4e-3),
    Case(8, 128, 128, 64, 2.4e-3),
    Case(16, 190, 200, 100, 2.3e-3),
    Case(16, 220, 161, 60, 2.4e-3, dtype="f32"),
    Case(2, 333, 1001, 100, 2.3e-3),
    Case(2, 1001, 333, 100, 2.3e-3, dtype="f32"),
    Case(3, 700, 520, 64, 2.4e-3),
    Case(9, 1100, 1300, 200, 2.3e-3),
    # more steps amplify what lies outside the gradient's span further
    Case(64, 32, 32, 16, 3.0e-3, steps=8),
    Case(64, 32, 32, 16, 5.5e-3, steps=16),
    Case(2, 333, 1001, 100, 2.3e-3, steps=8),
    Case(2, 333, 1001, 100, 3.6e-3, steps=16),
    Case(2, 1001, 333, 100, 2.4e-3, steps=6),
    # exactly of low rank, but for the rounding to fp32: any step that left the span would show
    Case(64, 16, 200, 8, 3.0e-3, steps=7, dtype="f32"),
    Case(64, 32, 32, 16, 3.4e-3, steps=8, dtype="f32"),
    Case(2, 333, 1001, 100, 2.7e-3, steps=8, dtype="f32"),
    Case(2, 2048, 256, 64, 2.6e-3, steps=8, dtype="f32"),
]


def gradients(case: Case, count=None) -> np.ndarray:
    rng = np.random.default_rng(case.rows * 131 + case.cols + case.rank)
    n = case.count if count is None else count
    w = np.logspace(0, -case.decay, case.rank) / np.sqrt(case.rank)
    g = np.stack([(rng.normal(size=(case.rows, case.rank)) * w) @ rng.normal(size=(case.rank, case.cols)) for _ in range(n)])
    if case.noise:
        g = g + case.noise * rng.normal(size=g.shape)
    g = g.astype(np.float32)
    return to_bf16(g) if case.dtype == "bf16" else g


def to_bf16(v: np.ndarray) -> np.ndarray:
    bits = np.ascontiguousarray(v, np.float32).view(np.uint32).astype(np.uint64)
    return ((bits + 0x7fff + ((bits >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)


def half(v, scale):
    """v in fp16, stored times a power of two."""
    return (v * np.float32(scale)).astype(np.float16).astype(np.float32) / np.float32(scale)


class Sym:
    """A symmetric matrix: its diagonal apart, the rest (and what the diagonal's rounding leaves) in fp16."""

    def __init__(self, full, scale):
        self.d = half(full.diagonal(), scale)
        self.m = half(full - np.diag(self.d), scale)

    def __matmul__(self, o):
        return self.m @ o.m + self.d[:, None] * o.m + self.m * o.d[None, :] + np.diag(self.d * o.d)


def modelled(g, steps=5, pair=False, low_by_diagonal=False, lows=1):
    """One matrix through the kernels' roundings.  low_by_diagonal: the low part is
    always taken by the diagonal; lows: steps before whose x there is no low part."""
    x = np.asarray(g, np.float32)
    x = x.T if x.shape[0] > x.shape[1] else x
    x = x * np.float32(1.0 / (np.sqrt((x.astype(np.float64) ** 2).sum()) + 1e-7))
    hi = half(x, 4096)
    lo = half(x - hi, 4096)
    left = steps
    while left > 0:
        k = 2 if pair and left == steps and steps > 1 else 1
        r, p = Sym(hi @ hi.T, 4096), None
        for i in range(k):
            q = r @ r
            q = C * q + B * (r.m + np.diag(r.d)) + A * np.eye(len(q), dtype=np.float32)
            q = Sym(q, 256)
            p = q if p is None else Sym(q @ p, 256)
            if i + 1 < k:
                r = Sym(Sym(q @ r, 4096) @ q, 4096)
        left -= k
        e = A ** k - p.d
        kappa = B * B / (4 * C) * A ** (k - 1)
        w = 0 if low_by_diagonal or left < 2 else 1 if left > 2 else np.maximum(1 - e / kappa, 0)
        gain = (p.d + e * w)[:, None]
        x = p.m @ hi + p.d[:, None] * hi + gain * lo
        hi = half(x, 4096)
        lo = half(x - hi, 4096) if left > lows else np.zeros_like(x)
    x = to_bf16(x)
    return x.T if g.shape[0] > g.shape[1] else x


def relative(got, want) -> float:
    return float(np.linalg.norm(np.asarray(got, np.float64) - want) / np.linalg.norm(want))
