"""Every property of the orthogonalised update on each path that a size can take:
matrices one workgroup holds, tiles of 32 and 64 (few of them), of 128 and of
256, with and without the first two steps under one product, wide and tall.

The tolerances are those of tests/test_gpu_update.py, and in norm what
the model of tests/update_model.py leaves: it gives at most 2.16e-3 for gradients
of full rank of these sizes and 1 to 6 steps, a quarter less than the 2.6e-3 here.
"""
import numpy as np
import pytest
import torch

from mixture_experts_transformer_moe_amd import binding as M
from oracle import update_oracle as U
from tests.gpu_common import say, to_f64
from tests.test_gpu_update import DT, check_update, dev, gradient, orth, u32

pytestmark = pytest.mark.gpu

# path of the last product, (count, rows, cols); the workspace tells a matrix that
# one workgroup holds (256 bytes) from the others
PATHS = {
    "one workgroup": (2, 150, 260), "one workgroup, 161 rows": (3, 161, 224), "one workgroup, 192 rows": (2, 192, 200),
    "tiles of 32": (2, 260, 400), "tiles of 64, long rows": (2, 40, 3900),
    "tiles of 64, pair": (2, 520, 800), "tiles of 128": (20, 260, 520), "tiles of 128, odd": (25, 333, 401),
    "tiles of 256": (9, 1100, 1300), "tiles of 256, pair": (8, 1024, 1600),
}
SMALL = [k for k in PATHS if np.prod(PATHS[k]) < 4_000_000]


def shape_of(path, tall=False):
    n, r, c = PATHS[path]
    small = M.moe_orthogonalize_workspace_bytes(n, r, c) == 256
    assert small == path.startswith("one workgroup"), f"{path}: {PATHS[path]} takes another path now"
    return (n, c, r) if tall else (n, r, c)


def grads(shape, dtype, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(DT[dtype])


def check(out, want, where, bound=2.6e-3):
    check_update(out, want, where)
    n = np.linalg.norm(want)
    assert np.linalg.norm(to_f64(out) - want) <= bound * n, where


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6])
@pytest.mark.parametrize("tall", [False, True], ids=["wide", "tall"])
@pytest.mark.parametrize("path", list(PATHS))
def test_steps(path, tall, steps):
    say(f"orthogonalize {path} {'tall' if tall else 'wide'} steps {steps}")
    shape = shape_of(path, tall)
    g = grads(shape, "bf16" if steps % 2 else "f32", seed=steps)
    out = orth(g, steps=steps, scale=0.2 * max(shape[1:]) ** 0.5)
    for i in {0, shape[0] - 1}:
        check(out[i], U.orthogonalize(to_f64(g[i]), steps, scale=0.2 * max(shape[1:]) ** 0.5), f"{path} {i}")


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tall", [False, True], ids=["wide", "tall"])
@pytest.mark.parametrize("path", SMALL)
def test_momentum(path, tall, dtype, nesterov):
    say(f"orthogonalize {path} {'tall' if tall else 'wide'} momentum {dtype} nesterov={nesterov}")
    n, rows, cols = shape_of(path, tall)
    m = grads((n, rows, cols), "f32", 3, 1e-2)
    m64 = to_f64(m)
    for step in range(2):                               # the state carries over
        g = grads((n, rows, cols), dtype, 10 + step, 3e-3)
        u, m64 = U.update_of(to_f64(g), m64, 0.95, nesterov)
        out = orth(g, m, 0.95, nesterov)
        # one fused multiply-add a step, each off by u of its result, which the
        # first step's may exceed by 1 / 0.95
        assert (np.abs(to_f64(m) - m64) <= 3 * u32 * np.abs(m64).max()).all()
        for i in {0, n - 1}:
            check(out[i], U.orthogonalize(u[i]), f"{path} step {step} {i}")


@pytest.mark.parametrize("path", list(PATHS))
def test_zero_and_nonfinite_matrices_keep_to_themselves(path):
    shape = shape_of(path)
    n, rows, cols = shape
    say(f"orthogonalize {path}, one matrix zero or not finite")
    g = grads(shape, "f32", 5)
    clean = orth(g)
    for bad, (i, j) in ((0.0, (0, 0)), (float("nan"), (rows - 1, 9)), (float("-inf"), (7, cols - 1))):
        h = g.clone()
        if bad == 0.0:
            h[n - 1] = 0.0
        else:
            h[n - 1, i, j] = bad
        for eps in (1e-7, 0.0):
            out = orth(h, eps=eps)
            assert (out[n - 1] == 0).all() if bad == 0.0 else torch.isnan(out[n - 1]).all()
        out = orth(h)
        assert torch.equal(out[: n - 1], clean[: n - 1])


@pytest.mark.parametrize("path", SMALL)
def test_nonfinite_momentum(path):
    # an infinity in the state makes that matrix NaN, and no other
    shape = shape_of(path)
    n, rows, cols = shape
    say(f"orthogonalize {path}, momentum not finite")
    g, m = grads(shape, "bf16", 6), grads(shape, "f32", 7)
    m0, m1 = m.clone(), m.clone()
    clean = orth(g, m0)
    m1[n - 1, rows - 1, 0] = float("inf")
    out = orth(g, m1)
    assert torch.isnan(out[n - 1]).all() and torch.isinf(m1[n - 1, rows - 1, 0])
    assert torch.equal(out[: n - 1], clean[: n - 1]) and torch.equal(m1[: n - 1], m0[: n - 1])


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e4, 1e30])
@pytest.mark.parametrize("path", [p for p in SMALL if p.startswith("tiles")] + ["one workgroup, 192 rows"])
def test_does_not_depend_on_the_gradients_scale(path, scale):
    # squares of these leave fp32's range; eps below the norm's rounding
    shape = shape_of(path)
    say(f"orthogonalize {path} scale {scale}")
    for dtype in ("bf16", "f32"):
        g = grads(shape, dtype, 8, scale)
        out = orth(g, eps=0.0)
        for i in {0, shape[0] - 1}:
            check(out[i], U.orthogonalize(to_f64(g[i]), eps=0.0), f"{path} {dtype} {i}")


@pytest.mark.parametrize("path", [p for p in SMALL if p.startswith("tiles")])
def test_tiny_against_eps(path):
    # a gradient as small as eps is not blown up
    shape = shape_of(path)
    g = grads(shape, "f32", 9, 1e-7 / (shape[1] * shape[2]) ** 0.5)
    say(f"orthogonalize {path} tiny against eps")
    out = orth(g, eps=1e-7)
    check(out[0], U.orthogonalize(to_f64(g[0]), eps=1e-7), path)


@pytest.mark.parametrize("path", SMALL)
def test_in_place_and_rows_behind(path):
    # out is g itself, inside a longer buffer whose rest stays as it was
    n, rows, cols = shape_of(path)
    say(f"orthogonalize {path} in place")
    g = grads((n, rows, cols), "bf16", 12)
    want = orth(g)
    buf = torch.full((n * rows * cols + 4096,), 9.0, dtype=torch.bfloat16, device="cuda")
    h = buf[: n * rows * cols].view(n, rows, cols)
    h.copy_(g)
    orth(h, out=h)
    assert torch.equal(h, want) and (buf[n * rows * cols:] == 9.0).all()


@pytest.mark.parametrize("path", ["one workgroup, 161 rows", "tiles of 32", "tiles of 128, odd"])
def test_momentum_keeps_what_lies_behind_it(path):
    n, rows, cols = shape_of(path)
    g = grads((n, rows, cols), "f32", 13)
    buf = torch.full((n * rows * cols + 4096,), 9.0, dtype=torch.float32, device="cuda")
    m = buf[: n * rows * cols].view(n, rows, cols)
    m.zero_()
    say(f"orthogonalize {path} momentum in a longer buffer")
    orth(g, m, 0.9)
    assert torch.equal(m, g) and (buf[n * rows * cols:] == 9.0).all()
