"""GPU parity of the pre-norm, its backward pass and the orthogonalised update
against the fp64 oracle (oracle/update_oracle.py), through the C ABI.

Tolerances.  u = 2^-24 is half a step of fp32, b = 2^-8 half a step of bf16.
  * norm, fp32: a row's statistics come from sums of at most 64 values a thread
    and 10 levels of a tree, each addition off by u of a partial sum that the
    sum of magnitudes bounds; with the few roundings after them 128 u of the
    largest magnitude that enters an element.  bf16 adds b of the value.
  * dgamma, dbeta: each thread adds at most rows / 1 values in turn (tests keep
    that below 128), then at most 4 + 64 partial sums: 256 u of the sum of
    magnitudes.
  * update: the output's rounding is at most b of the value.  Inside, the
    largest error is that of x after the third step, held to 2^-11 (half a step
    of fp16, rms 2^-11 / sqrt 3) in the products that follow, which amplify it
    by at most a^2 = 11.9: 3.4e-3 < b of the matrix' norm.  Together 2 b in
    norm.  Every product is P x with the short side inside, so with d the
    roundings of P and e those of x an element is off by sum_k d_ik x_kj and
    sum_k P_ik e_kj, |e_kj| <= 2^-12 |x_kj|: terms of random sign whose sum of
    squares is that of column j of x.  So beside an element's own rounding 8
    standard deviations, b each, of its column along the short side (not of the
    whole matrix: the columns of a matrix of rank one differ like their entries).
"""
import numpy as np
import pytest
import torch

from mixture_experts_transformer_moe_amd import binding as M, configs
from mixture_experts_transformer_moe_amd.inputs import LayerInputs, dout_encoded, token_mask
from oracle import update_oracle as U
from tests.gpu_common import StackedInputs, say, to_f64

pytestmark = pytest.mark.gpu

u32, b16 = 2.0 ** -24, 2.0 ** -8
KIND = {"layer": M.MOE_NORM_LAYER, "rms": M.MOE_NORM_RMS}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, dt):
    return torch.from_numpy(np.asarray(a, np.float32)).to(dt).cuda()


def f32(n):
    return torch.full((n,), 7.0, dtype=torch.float32, device="cuda")


def norm_case(kind, rows, cols, dtype, residual=True, affine=True, seed=0, offset=0.25, scale=1.0):
    rng = np.random.default_rng(seed)
    dt = DT[dtype]
    x = dev((rng.normal(size=(rows, cols)) + offset) * scale, dt)
    r = dev(rng.normal(size=(rows, cols)) * scale, dt) if residual else None
    gamma = dev(1 + 0.2 * rng.normal(size=cols), torch.float32) if affine else None
    beta = dev(0.2 * rng.normal(size=cols), torch.float32) if affine else None
    return rng, dt, x, r, gamma, beta


def check_forward(kind, dtype, x, r, gamma, beta, eps, sum_, y, mean, rstd):
    s = to_f64(x)
    if r is not None:
        want = (x.float() + r.float()).to(x.dtype)       # one fp32 addition, rounded once
        assert torch.equal(sum_, want)
        s = to_f64(want)
    ry, rm, rr = U.norm_forward(kind, s, None if gamma is None else to_f64(gamma),
                                None if beta is None else to_f64(beta), eps)
    amax = np.abs(s).max(1, initial=0.0)
    if kind == "layer":
        assert (np.abs(to_f64(mean) - rm) <= 128 * u32 * amax).all()
    # rstd: half the relative error of the variance, whose terms carry the mean's
    dm = 128 * u32 * amax * rr
    assert (np.abs(to_f64(rstd) / rr - 1) <= 128 * u32 + dm).all()
    g = 1.0 if gamma is None else np.abs(to_f64(gamma))
    tol = 128 * u32 * ((amax * rr)[:, None] + np.abs(ry)) * (g + 0 * ry) + 4 * u32 * np.abs(ry) + 1e-300
    if beta is not None:
        tol = tol + 4 * u32 * np.abs(to_f64(beta))
    tol = tol + np.abs(ry) * dm[:, None]
    if dtype == "bf16":
        tol = tol + b16 * np.abs(ry)
    assert (np.abs(to_f64(y) - ry) <= tol).all()


NORM_SIZES = [(1, 1), (3, 5), (2, 64), (7, 255), (1, 511), (5, 513), (33, 1023), (2, 1025), (64, 2048), (3, 2049),
              (32, 4096), (5, 6000), (1, 8191), (3, 16384), (1030, 520), (1025, 1000), (1100, 2050), (1027, 7),
              (1024, 4100)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
def test_norm_forward(rows, cols, kind, dtype):
    residual, affine = (rows + cols) % 2 == 0, cols != 64
    say(f"norm forward {rows}x{cols} {kind} {dtype} residual={residual}")
    _, dt, x, r, gamma, beta = norm_case(kind, rows, cols, dtype, residual, affine, seed=rows * 7 + cols)
    y = torch.full_like(x, 9.0)
    s = torch.full_like(x, 9.0) if residual else None
    mean, rstd = f32(rows), f32(rows)
    M.moe_norm_forward(KIND[kind], x, r, gamma, beta, 1e-5, s, y, mean, rstd)
    torch.cuda.synchronize()
    check_forward(kind, dtype, x, r, gamma, beta, 1e-5, s, y, mean, rstd)
    if kind == "rms":
        assert (mean == 7.0).all()                      # not written


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
def test_norm_backward(rows, cols, kind, dtype):
    residual, affine = (rows + cols) % 2 == 1, cols != 64
    say(f"norm backward {rows}x{cols} {kind} {dtype} dsum={residual}")
    rng, dt, x, r, gamma, _ = norm_case(kind, rows, cols, dtype, residual, affine, seed=rows * 5 + cols)
    dy = dev(rng.normal(size=(rows, cols)) + 0.1, dt)
    _, m64, r64 = U.norm_forward(kind, to_f64(x), eps=1e-5)
    mean, rstd = dev(m64, torch.float32), dev(r64, torch.float32)
    dx, dg, db = torch.full_like(x, 9.0), f32(cols), f32(cols)
    with_beta = cols % 3 != 0
    ws = torch.full((M.moe_norm_workspace_bytes(rows, cols),), 255, dtype=torch.uint8, device="cuda")
    M.moe_norm_backward(KIND[kind], dy, x, gamma, mean if kind == "layer" else None, rstd, r, dx, dg,
                        db if with_beta else None, ws)
    torch.cuda.synchronize()
    args = (to_f64(dy), to_f64(x), None if gamma is None else to_f64(gamma), to_f64(mean), to_f64(rstd))
    rx, rg, rb = U.norm_backward(kind, *args, None if r is None else to_f64(r))
    h = np.abs((args[1] - (args[3][:, None] if kind == "layer" else 0)) * args[4][:, None])
    t = np.abs(args[0] * (1.0 if gamma is None else args[2]))
    top = (t.max(1) * (1 + h.max(1) * h.mean(1)) * args[4])[:, None]
    tol = 128 * u32 * (top + np.abs(rx)) + (b16 * np.abs(rx) if dtype == "bf16" else 0)
    # (x - mean) in fp32: u of |x| + |mean|, times rstd and what multiplies h
    tol = tol + 8 * u32 * ((np.abs(args[1]) + np.abs(args[3])[:, None]) * args[4][:, None] ** 2 * t.max(1)[:, None])
    assert (np.abs(to_f64(dx) - rx) <= tol).all()
    he = h + (np.abs(args[1]) + np.abs(args[3])[:, None]) * args[4][:, None]
    assert (np.abs(to_f64(dg) - rg) <= 256 * u32 * (np.abs(args[0]) * he).sum(0)).all()
    if with_beta:
        assert (np.abs(to_f64(db) - rb) <= 256 * u32 * np.abs(args[0]).sum(0)).all()
    else:
        assert (db == 7.0).all()


# rows that share a wave, ragged ends of every length, three vectors a thread
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1100, 60), (1100, 100), (1027, 250), (1030, 2100), (1030, 4101)] +
                         [(5, 8 + k) for k in range(1, 8)] + [(1025, 15 + k) for k in range(3)])
def test_norm_forms(rows, cols, dtype):
    test_norm_forward(rows, cols, "layer", dtype)
    test_norm_backward(rows, cols, "layer", dtype)


def test_norm_of_constant_and_huge_rows():
    # a constant row has no variance: y = beta; values near fp32's square-root range keep finite statistics
    x = torch.ones(4, 300, device="cuda") * torch.tensor([0.0, 3.0, 1e18, -1e-30], device="cuda")[:, None]
    beta = torch.linspace(-1, 1, 300, device="cuda")
    y, mean, rstd = torch.empty_like(x), f32(4), f32(4)
    M.moe_norm_forward(M.MOE_NORM_LAYER, x, None, None, beta, 1e-6, None, y, mean, rstd)
    torch.cuda.synchronize()
    # rows 0, 1, 3: the mean of equal values is off by 300 u of them at most
    for i, v in ((0, 0.0), (1, 3.0), (3, 1e-30)):
        assert (y[i] - beta).abs().max() <= 300 * u32 * v * 1e3 + 2 * u32
    assert torch.isfinite(y[2]).all() and torch.isfinite(rstd).all()


def test_norm_keeps_nan_to_its_row():
    x = torch.randn(6, 1000, device="cuda").bfloat16()
    clean = torch.empty_like(x)
    M.moe_norm_forward(M.MOE_NORM_RMS, x, None, None, None, 1e-6, None, clean, None, None)
    x[2, 5], x[4, 999] = float("nan"), float("inf")
    y = torch.empty_like(x)
    M.moe_norm_forward(M.MOE_NORM_RMS, x, None, None, None, 1e-6, None, y, None, None)
    torch.cuda.synchronize()
    for i in (0, 1, 3, 5):
        assert torch.equal(y[i], clean[i])
    assert torch.isnan(y[2]).all() and torch.isnan(y[4, 999])


def test_norm_in_place_and_no_rows():
    _, _, x, r, gamma, beta = norm_case("layer", 70, 770, "bf16", seed=3)
    y, s, mean, rstd = torch.empty_like(x), torch.empty_like(x), f32(70), f32(70)
    M.moe_norm_forward(M.MOE_NORM_LAYER, x, r, gamma, beta, 1e-6, s, y, mean, rstd)
    x2, r2 = x.clone(), r.clone()
    M.moe_norm_forward(M.MOE_NORM_LAYER, x2, r2, gamma, beta, 1e-6, r2, x2, mean, rstd)
    assert torch.equal(x2, y) and torch.equal(r2, s)
    dy = torch.randn_like(x)
    ws = torch.empty(M.moe_norm_workspace_bytes(70, 770), dtype=torch.uint8, device="cuda")
    dx, dg, db = torch.empty_like(x), f32(770), f32(770)
    M.moe_norm_backward(M.MOE_NORM_LAYER, dy, s, gamma, mean, rstd, r, dx, dg, db, ws)
    dy2 = dy.clone()
    M.moe_norm_backward(M.MOE_NORM_LAYER, dy2, s, gamma, mean, rstd, r, dy2, None, None, None)
    assert torch.equal(dy2, dx)
    # in place, the sums' workgroups may not read what dx overwrites
    for other in (dy.clone(), s.clone()):
        a, b = (other, s) if torch.equal(other, dy) else (dy, other)
        dg2, db2 = f32(770), f32(770)
        M.moe_norm_backward(M.MOE_NORM_LAYER, a, b, gamma, mean, rstd, r, other, dg2, db2, ws)
        assert torch.equal(other, dx)
        h = ((s.double() - mean.double()[:, None]) * rstd.double()[:, None]).abs()
        assert ((dg2 - dg).abs() <= 512 * u32 * ((dy.double().abs() * (h + 1)).sum(0))).all()
        assert ((db2 - db).abs() <= 512 * u32 * dy.double().abs().sum(0)).all()
    none = torch.empty(0, 770, dtype=torch.bfloat16, device="cuda")
    M.moe_norm_backward(M.MOE_NORM_LAYER, none, none, gamma, f32(0), f32(0), None, none.clone(), dg, db, None)
    torch.cuda.synchronize()
    assert (dg == 0).all() and (db == 0).all()


def test_norm_past_two_to_the_31_elements():
    # the last rows alone give the same bits (rows do not depend on each other)
    say("norm 140000x16384 bf16")
    rows, cols, last = 140000, 16384, 5
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    y, mean, rstd = torch.empty_like(x), f32(rows), f32(rows)
    M.moe_norm_forward(M.MOE_NORM_LAYER, x, None, None, None, 1e-6, None, y, mean, rstd)
    x1 = x[-last:].clone()
    y1, mean1, rstd1 = torch.empty_like(x1), f32(last), f32(last)
    M.moe_norm_forward(M.MOE_NORM_LAYER, x1, None, None, None, 1e-6, None, y1, mean1, rstd1)
    assert torch.equal(y[-last:], y1) and torch.equal(mean[-last:], mean1) and torch.equal(rstd[-last:], rstd1)
    dx, dx1 = torch.empty_like(x), torch.empty_like(x1)
    M.moe_norm_backward(M.MOE_NORM_LAYER, y, x, None, mean, rstd, None, dx, None, None, None)
    M.moe_norm_backward(M.MOE_NORM_LAYER, y1, x1, None, mean1, rstd1, None, dx1, None, None, None)
    torch.cuda.synchronize()
    assert torch.equal(dx[-last:], dx1)


# ---------------------------------------------------------------- the update

def gradient(rng, rows, cols, tokens):
    w = np.logspace(0, -1.5, tokens)
    return (rng.normal(size=(rows, tokens)) * w) @ rng.normal(size=(tokens, cols)) * 1e-3 / np.sqrt(tokens)


def check_update(out, want, where=""):
    want = np.asarray(want)
    got = to_f64(out)
    assert np.isfinite(got).all(), where
    n = np.linalg.norm(want)
    rms = n / np.sqrt(want.size)
    err = np.linalg.norm(got - want)
    say(f"update {where} {want.shape}: rel {err / max(n, 1e-300):.2e}, max {np.abs(got - want).max() / max(rms, 1e-300):.2e} rms")
    assert err <= 2 * b16 * n, where
    col = np.sqrt((want ** 2).mean(0 if want.shape[0] <= want.shape[1] else 1, keepdims=True))
    assert (np.abs(got - want) <= b16 * np.abs(want) + 8 * b16 * col).all(), where


def orth(g, momentum=None, mu=0.95, nesterov=True, steps=5, eps=1e-7, scale=1.0, out=None, stream=None):
    count = g.shape[0] if g.dim() == 3 else 1
    n = M.moe_orthogonalize_workspace_bytes(count, g.shape[-2], g.shape[-1])
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")      # fp16 and fp32 NaN
    if out is None:
        out = torch.full(g.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    M.moe_orthogonalize(g, momentum, mu, nesterov, steps, eps, scale, out, ws, stream)
    torch.cuda.synchronize()
    return out


ORTH_SIZES = [(1, 1, 1), (2, 1, 7), (1, 9, 1), (3, 32, 32), (2, 33, 31), (5, 64, 200), (2, 127, 129), (1, 130, 513),
              (3, 333, 101), (2, 256, 256), (1, 300, 2000), (2, 1000, 257), (1, 520, 1030), (20, 260, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("count,rows,cols", ORTH_SIZES)
def test_orthogonalize(count, rows, cols, dtype):
    say(f"orthogonalize {count}x{rows}x{cols} {dtype}")
    rng = np.random.default_rng(rows + 3 * cols)
    g = dev(np.stack([gradient(rng, rows, cols, max(1, min(rows, cols) // 2)) for _ in range(count)]), DT[dtype])
    out = orth(g)
    for i in range(count):
        check_update(out[i], U.orthogonalize(to_f64(g[i])), f"{i}")


@pytest.mark.parametrize("count,rows,cols", [(40, 1024, 512), (70, 512, 700), (9, 1100, 1300)])
def test_orthogonalize_many_tiles(count, rows, cols):
    # enough tiles for the 256-wide ones, several a workgroup
    rng = np.random.default_rng(7)
    g = torch.randn(count, rows, cols, device="cuda").bfloat16()
    out = orth(g)
    for i in (0, 1, count // 2, count - 1):
        check_update(out[i], U.orthogonalize(to_f64(g[i])), f"{i}")


def test_orthogonalize_past_two_to_the_31_elements():
    # (24 GB of workspace; the last matrices against the oracle)
    count, rows, cols = 2100, 512, 2048
    say(f"orthogonalize {count}x{rows}x{cols} bf16")
    g = torch.empty(count, rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    out = orth(g)
    for i in (0, count - 1):
        check_update(out[i], U.orthogonalize(to_f64(g[i])), f"{i}")


@pytest.mark.parametrize("rows,cols", [(4000, 20000), (20000, 4000)])
def test_orthogonalize_large_matrix(rows, cols):
    # against the formula in 64 bits on the device (Q commutes with R, so R' = Q R Q)
    say(f"orthogonalize {rows}x{cols} f32")
    g = torch.empty(rows, cols, device="cuda").normal_()
    out = orth(g)
    x = out.float() if rows < cols else out.float().t().contiguous()
    u = g if rows < cols else g.t().contiguous()
    want = u.double() / u.double().norm()
    r = want @ want.t().contiguous()
    one = torch.eye(r.shape[0], dtype=torch.float64, device="cuda")
    m = one
    for _ in range(5):
        q = 3.4445 * one - 4.7750 * r + 2.0315 * (r @ r)
        m = q @ m
        r = q @ r @ q
    ref = m @ want
    torch.cuda.synchronize()
    err = (x.double() - ref).norm() / ref.norm()
    say(f"rel {float(err):.2e}")
    assert err <= 2 * b16


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8])
def test_orthogonalize_steps(steps):
    g = dev(gradient(np.random.default_rng(5), 150, 260, 200), torch.float32)
    check_update(orth(g, steps=steps, scale=0.2 * 260 ** 0.5), U.orthogonalize(to_f64(g), steps, scale=0.2 * 260 ** 0.5))


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_orthogonalize_with_momentum(nesterov, dtype):
    rng = np.random.default_rng(8)
    m = dev(rng.normal(size=(3, 200, 90)) * 1e-2, torch.float32)
    m64 = to_f64(m)
    for step in range(3):                               # the state carries over
        g = dev(np.stack([gradient(rng, 200, 90, 50) for _ in range(3)]), DT[dtype])
        u, m64 = U.update_of(to_f64(g), m64, 0.95, nesterov)
        out = orth(g, m, 0.95, nesterov)
        # one fused multiply-add a step, each off by u of its result; the state decays
        assert (np.abs(to_f64(m) - m64) <= 3 * u32 * np.abs(m64).max()).all()
        for i in range(3):
            check_update(out[i], U.orthogonalize(u[i]), f"step {step}")


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e4, 1e30])
def test_orthogonalize_does_not_depend_on_the_gradients_scale(scale):
    # squares of these leave fp32's range; eps below the norm's rounding
    g = (torch.randn(2, 96, 140, device="cuda") * scale).bfloat16()
    out = orth(g, eps=0.0)
    for i in range(2):
        check_update(out[i], U.orthogonalize(to_f64(g[i]), eps=0.0))


def test_orthogonalize_zero_and_nonfinite_matrices_keep_to_themselves():
    g = torch.randn(6, 140, 200, device="cuda")
    clean = orth(g)
    g[1] = 0.0
    g[3, 7, 9] = float("nan")
    g[4, 139, 199] = float("-inf")
    for eps in (1e-7, 0.0):
        out = orth(g, eps=eps)
        assert (out[1] == 0).all()
        assert torch.isnan(out[3]).all() and torch.isnan(out[4]).all()
    out = orth(g)
    for i in (0, 2, 5):
        assert torch.equal(out[i], clean[i])


def test_orthogonalize_tiny_against_eps():
    # a gradient as small as eps is not blown up
    g = dev(np.full((1, 40, 50), 1e-9), torch.float32)
    check_update(orth(g, eps=1e-7)[0], U.orthogonalize(to_f64(g[0]), eps=1e-7))


def test_orthogonalize_low_rank():
    rng = np.random.default_rng(9)
    for rank in (1, 4, 60):
        g = dev(rng.normal(size=(1, 256, rank)) @ rng.normal(size=(1, rank, 640)), torch.bfloat16)
        check_update(orth(g)[0], U.orthogonalize(to_f64(g[0])), f"rank {rank}")


def test_orthogonalize_axis_aligned():
    # diagonal matrices and a single large row: the diagonal parts carry everything
    g = torch.zeros(3, 200, 300, device="cuda")
    g[0, range(200), range(200)] = 1.0
    g[1, range(200), range(200)] = torch.logspace(0, -3, 200, device="cuda")
    g[2] = 1e-4 * torch.randn(200, 300, device="cuda")
    g[2, 3] = 1.0
    out = orth(g)
    for i in range(3):
        check_update(out[i], U.orthogonalize(to_f64(g[i])), f"{i}")


def test_orthogonalize_in_place_rows_and_transpose():
    g = torch.randn(4, 300, 170, device="cuda").bfloat16()
    out = orth(g)
    h = g.clone()
    assert torch.equal(orth(h, out=h), out)
    # the transpose goes through the same blocks: the same bits
    t = orth(g.mT.contiguous())
    assert torch.equal(t.mT, out)


def test_update_bits_streams_and_graph():
    """The same bits on every call, on another stream, and from a graph's replays
    between eager calls."""
    s = torch.cuda.Stream()
    g = torch.randn(3, 260, 400, device="cuda").bfloat16()
    x, dy = torch.randn(900, 1000, device="cuda").bfloat16(), torch.randn(900, 1000, device="cuda").bfloat16()
    gamma = torch.randn(1000, device="cuda")
    n = M.moe_orthogonalize_workspace_bytes(3, 260, 400)

    def state():
        return dict(g=g.clone(), m=torch.zeros(3, 260, 400, device="cuda"), out=torch.empty_like(g), x=x.clone(),
                    dy=dy.clone(), y=torch.empty_like(x), mean=f32(900), rstd=f32(900), dx=torch.empty_like(x),
                    dg=f32(1000), db=f32(1000), ws=torch.empty(n, dtype=torch.uint8, device="cuda"),
                    nws=torch.empty(M.moe_norm_workspace_bytes(900, 1000), dtype=torch.uint8, device="cuda"))

    def go(q, stream=None):
        M.moe_norm_forward(M.MOE_NORM_LAYER, q["x"], None, gamma, None, 1e-6, None, q["y"], q["mean"], q["rstd"], stream)
        M.moe_norm_backward(M.MOE_NORM_LAYER, q["dy"], q["x"], gamma, q["mean"], q["rstd"], None, q["dx"], q["dg"],
                            q["db"], q["nws"], stream)
        M.moe_orthogonalize(q["g"], q["m"], 0.9, True, 5, 1e-7, 1.0, q["out"], q["ws"], stream)

    names = ("out", "m", "y", "dx", "dg", "db")
    want, eager = [], state()
    for _ in range(4):
        go(eager)
        torch.cuda.synchronize()
        want.append({k: eager[k].clone() for k in names})
    side = state()
    torch.cuda.synchronize()
    for i in range(2):
        go(side, s)
        s.synchronize()
        assert all(torch.equal(side[k], want[i][k]) for k in names)
    rec = state()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        go(rec)
    rec["m"].zero_()
    for i in range(4):
        graph.replay()
        if i % 2:
            torch.cuda.synchronize()
        go(eager)                                       # eager work between the replays
        assert all(torch.equal(rec[k], want[i][k]) for k in names), i
        torch.cuda.synchronize()


def test_training_step_from_norm_to_update():
    """Pre-norm, the layer's training pass, the pre-norm's backward and the
    orthogonalised updates of the gradients, as a training step runs them."""
    s = configs.variant(configs.XS2_T4096, name="update_step_t300", T=300, D=256, E=16, k=4, F=256, Fs=256,
                        pad_frac=0.1, seq_len=64, aux_coef=0.1)
    inp = StackedInputs(LayerInputs(s))
    w = M.upload_train_weights(s, inp.w_router, inp.bias, inp.wgu, inp.wd, inp.shared())
    rng = np.random.default_rng(11)
    x, r = dev(rng.normal(size=(s.T, s.D)), torch.bfloat16), dev(rng.normal(size=(s.T, s.D)), torch.bfloat16)
    gamma = dev(1 + 0.1 * rng.normal(size=s.D), torch.float32)
    stream, y, rstd = torch.empty_like(x), torch.empty_like(x), f32(s.T)
    M.moe_norm_forward(M.MOE_NORM_RMS, x, r, gamma, None, 1e-6, stream, y, None, rstd)
    b = M.alloc_train_buffers(s, torch.from_numpy(token_mask(s)).cuda())
    M.train_forward(s, y, w, b, s.aux_coef)
    dout = M.to_device(dout_encoded(s), s, "cuda")
    M.train_backward(s, y, dout, w, b)
    ws = torch.empty(M.moe_norm_workspace_bytes(s.T, s.D), dtype=torch.uint8, device="cuda")
    dx, dgamma = torch.empty_like(x), f32(s.D)
    # the block's output is stream + layer(y): dout reaches the residual stream too
    M.moe_norm_backward(M.MOE_NORM_RMS, b.dx, stream, gamma, None, rstd, dout, dx, dgamma, None, ws)
    grads = {"dw_gate_up": b.dw_gate_up, "dw_down": b.dw_down, "dws_gate_up": b.dws_gate_up, "dws_down": b.dws_down,
             "dw_router": b.dw_router}
    outs = {k: orth(g, scale=0.2 * max(g.shape[-2:]) ** 0.5) for k, g in grads.items()}
    torch.cuda.synchronize()
    check_forward("rms", "bf16", x, r, gamma, None, 1e-6, stream, y, None, rstd)
    rx, rg, _ = U.norm_backward("rms", to_f64(b.dx), to_f64(stream), to_f64(gamma), np.zeros(s.T), to_f64(rstd),
                                to_f64(dout))
    np.testing.assert_allclose(to_f64(dx), rx, rtol=b16, atol=256 * u32 * np.abs(rx).max())
    np.testing.assert_allclose(to_f64(dgamma), rg, rtol=0, atol=256 * u32 * (np.abs(to_f64(b.dx)) * 5).sum(0).max())
    for k, g in grads.items():
        for i in range(g.shape[0] if g.dim() == 3 else 1):
            gi, oi = (g[i], outs[k][i]) if g.dim() == 3 else (g, outs[k])
            if not (gi != 0).any():
                assert (oi == 0).all()
                continue
            check_update(oi, U.orthogonalize(to_f64(gi), scale=0.2 * max(gi.shape) ** 0.5), f"{k} {i}")
