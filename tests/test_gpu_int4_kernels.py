"""Each kernel of the 4-bit products (tests/int4_kernels.py) in every group, both products,
on both sides of the rule that chooses it, over reductions whose scales come in several
runs: elementwise within the bound of tests/test_gpu_int4_exact.py, and as a whole no
further off than the output's rounding."""
import numpy as np
import pytest
import torch

from tests.gpu_common import say, to_f64
from tests.int4_kernels import E, K, KERNELS, batch
from tests.test_gpu_int4 import Case, b16, u32
from tests.test_gpu_int4_exact import groups_of

pytestmark = pytest.mark.gpu


def check(c, what, rows, codes, scales, got):
    y, tot, mag = groups_of(codes, rows, scales, c.group)
    d = u32 * (64 * mag + 70 * tot)
    want, tol = y, d + b16 * np.abs(y)
    if c.mode == "gate_up":
        n = y.shape[1] // 2
        gate, up, dg, du = y[:, :n], y[:, n:], d[:, :n], d[:, n:]
        want = gate / (1 + np.exp(-gate)) * up
        tol = 1.1 * np.abs(up) * dg + np.abs(gate) * du + dg * du + (2.0 ** -20 * (1 + np.abs(gate)) + b16) * np.abs(want)
    off = np.abs(got - want)
    assert (off <= tol).all(), f"{what}: worst {(off / tol).max():.2f}"
    # half a step of bf16 is 2^-8 of a value at most: 2^-8 / sqrt 3 of it on average, a tenth
    # more for what 256 values a row vary by
    assert np.linalg.norm(off) <= 1.1 * b16 / 3 ** 0.5 * np.linalg.norm(want), what


@pytest.mark.parametrize("mode,group,mean", KERNELS)
def test_kernel(mode, group, mean):
    say(f"int4 {mode}, groups of {group}, {mean} rows an expert: {KERNELS[mode, group, mean]}")
    T, D, F, Fs = batch(mode, mean)
    rng = np.random.default_rng(mean)
    counts = list(rng.multinomial(T * K, [0.4, 0.1, 0.3, 0.2]))
    c = Case(mode, T, D, F, Fs, group, counts, K, seed=group + mean)
    c.run()
    torch.cuda.synchronize()
    a, got, s = to_f64(c.a), to_f64(c.out), to_f64(c.s)
    width, n = (c.F, c.S * c.F) if mode == "gate_up" else (c.D, c.S * c.D)
    routed = got[:n].reshape(c.S, width)
    for e in range(E):
        lo, hi = c.offsets[e], c.offsets[e + 1]
        if hi == lo:
            continue
        rows = a.reshape(T, D)[c.sorted_token[lo:hi]] if mode == "gate_up" else a[: c.S * F].reshape(c.S, F)[lo:hi]
        check(c, f"expert {e}", rows, c.w[e], s[e], routed[lo:hi])
    if mode == "gate_up":
        rows, shared = a.reshape(T, D), got[n:].reshape(T, Fs)
    else:
        rows, shared = a[c.S * F:].reshape(T, Fs), to_f64(c.out_shared).reshape(T, D)
    check(c, "shared expert", rows, c.ws[0], to_f64(c.ss)[0], shared)
