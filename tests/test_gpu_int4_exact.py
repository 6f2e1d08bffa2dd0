"""What 4-bit codes contribute to a product is exact: a code of 0 nothing at all,
whatever its activation, and the rest as in an fp32 sum of the terms themselves.

Tolerance.  u = 2^-24 is half a step of fp32, b = 2^-8 of bf16.  A group's sum is at most
4 MFMAs of 32 exact products each, added in at most 8 levels with an error of a step
(2 u) each, of sums that M_g = sum |q a| bounds: 64 u M_g.  Then as elsewhere the scale's
product, the sum over groups (at most 64) and waves' parts: 70 u of the sum of |s_g y_g|.
  d = u (64 sum_g |s_g| M_g + 70 sum_g |s_g y_g|);  down: d + b |y|
gate_up: 1.1 |u| dg + |g| du + dg du + (2^-20 (1 + |g|) + b) |h|
"""
import numpy as np
import pytest
import torch

from mixture_experts_transformer_moe_amd import binding as M
from tests.gpu_common import say, to_f64
from tests.test_gpu_int4 import b16, bf16, u32, Case

pytestmark = pytest.mark.gpu

# rows an expert in the kernel of 16 rows, of 32, and in the tile kernel (both directions)
ROWS = [3, 15, 45]


def groups_of(w, a, scales, group):
    """(y, sum |s y_g|, sum |s| M_g) of rows a by codes w [N, K]."""
    y, tot, mag = (np.zeros((len(a), len(w))) for _ in range(3))
    for i in range(scales.shape[1]):
        c, x, s = w[:, i * group:(i + 1) * group].astype(np.float64), a[:, i * group:(i + 1) * group], scales[:, i]
        part = (x @ c.T) * s
        y += part
        tot += np.abs(part)
        mag += (np.abs(x) @ np.abs(c).T) * np.abs(s)
    return y, tot, mag


def outputs(c, e):
    """(activations, outputs) of expert e's rows, in float64."""
    width = c.F if c.mode == "gate_up" else c.D
    lo, hi = c.offsets[e], c.offsets[e + 1]
    got = to_f64(c.out)[: c.S * width].reshape(c.S, width)[lo:hi]
    if c.mode == "gate_up":
        return to_f64(c.a).reshape(c.T, c.D)[c.sorted_token[lo:hi]], got
    return to_f64(c.a)[: c.S * c.F].reshape(c.S, c.F)[lo:hi], got


def check_tight(c):
    """Every routed output within the bound above."""
    scales = to_f64(c.s)
    for e in range(c.E):
        rows, got = outputs(c, e)
        y, tot, mag = groups_of(c.w[e], rows, scales[e], c.group)
        d = u32 * (64 * mag + 70 * tot)
        want, tol = y, d + b16 * np.abs(y)
        if c.mode == "gate_up":
            n = y.shape[1] // 2
            gate, up, dg, du = y[:, :n], y[:, n:], d[:, :n], d[:, n:]
            want = gate / (1 + np.exp(-gate)) * up
            tol = 1.1 * np.abs(up) * dg + np.abs(gate) * du + dg * du + (2.0 ** -20 * (1 + np.abs(gate)) + b16) * np.abs(want)
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= tol + 1e-37).all(), f"expert {e}: worst {(np.abs(got - want) / (tol + 1e-37)).max():.2f}"


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("mode", ["gate_up", "down"])
def test_codes_of_zero_add_nothing(mode, rows, group):
    """channels of 10^8 and 2^120 under codes of 0: the outputs are those of the other channels"""
    say(f"int4 {mode}, {rows} rows an expert, groups of {group}: large channels under codes of 0")
    counts = [rows - 1, rows, rows + 1]
    c = Case(mode, 3 * rows, 512, 512, 0, group, counts, 1, seed=rows + group)
    K = 512
    big = [5, 77, 300]
    c.w[:, :, big] = 0
    from oracle import int4_oracle as I
    c.pw = M.pack_int4(torch.from_numpy(I.two_a_byte(c.w)).cuda())
    c.a.view(-1, K)[:, 5] = 1e8
    c.a.view(-1, K)[1::2, 77] = -1e8
    c.a.view(-1, K)[0::3, 300] = 2.0 ** 120
    c.run()
    torch.cuda.synchronize()
    check_tight(c)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("mode", ["gate_up", "down"])
def test_zero_weights_give_zero(mode, rows, group):
    """rows of zeros, and groups of zeros beside groups of 10^-6, through the quantiser, with outlier channels"""
    say(f"int4 {mode}, {rows} rows an expert, groups of {group}: zero weights")
    c = Case(mode, 3 * rows, 512, 512, 0, group, [rows] * 3, 1, seed=rows + 1)
    rng = np.random.default_rng(rows + group)
    E, N, K = c.w.shape
    w = rng.normal(size=(E, N, K)) * 0.02
    w[:, 1::4] = 0.0                                     # whole rows (of gate and of up)
    w[:, 2::4] *= 5e-5
    w[:, 2::4, : K // 2] = 0.0                           # half of the groups of a row of small weights
    bits = bf16(w)
    c.pw, c.s = M.quantize_int4(bits, group)
    from oracle import int4_oracle as I
    c.w = I.unpack(c.pw.cpu().numpy(), E, N, K)
    assert (c.w[:, 1::4] == 0).all()
    a = rng.normal(size=(c.a.numel() // K, K))
    a[:, :8] *= 50.0
    c.a.copy_(bf16(a).view(-1))
    c.run()
    torch.cuda.synchronize()
    for e in range(E):
        assert (outputs(c, e)[1][:, 1::4] == 0).all()
    check_tight(c)
