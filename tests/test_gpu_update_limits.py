"""The largest and smallest sizes that the pre-norm and the orthogonalised update
take, and calls that run beside each other."""
import numpy as np
import pytest
import torch

from mixture_experts_transformer_moe_amd import binding as M
from oracle import update_oracle as U
from tests.gpu_common import say, to_f64
from tests.test_gpu_update import b16, check_update, f32, orth, u32

pytestmark = pytest.mark.gpu


def in_64_bits(g):
    """The formula on the device, for a matrix with its short side first (Q commutes with R, so R' = Q R Q)."""
    want = g.double()
    want /= want.norm() + 1e-7
    r = want @ want.t().contiguous()
    one = torch.eye(r.shape[0], dtype=torch.float64, device="cuda")
    m = one
    for _ in range(5):
        q = U.A * one + U.B * r + U.C * (r @ r)
        m = q @ m
        r = q @ r @ q
    return m @ want


@pytest.mark.parametrize("tall", [False, True], ids=["wide", "tall"])
def test_largest_matrix(tall):
    # (11 GB of workspace; a side of 65535, 2^30 - 1 elements less one row)
    say(f"orthogonalize 16383 x 65535 bf16 {'tall' if tall else 'wide'}")
    g = torch.empty(16383, 65535, dtype=torch.bfloat16, device="cuda").normal_()
    out = orth(g.t().contiguous()).t() if tall else orth(g)
    ref = in_64_bits(g)
    err = float((out.double() - ref).norm() / ref.norm())
    say(f"rel {err:.2e}")
    # full rank, the roundings average over many terms: 1.66e-3 is the output's own
    assert err <= 2.3e-3
    rows = ((out.double() - ref).norm(dim=1) / ref.norm(dim=1)).max()
    assert float(rows) <= 2 * b16


@pytest.mark.parametrize("rows,cols", [(1, 65536), (65536, 1), (3, 65536), (65536, 2), (2, 2049), (33, 1025)])
def test_longest_sides(rows, cols):
    say(f"orthogonalize {rows} x {cols}")
    g = torch.randn(rows, cols, device="cuda")
    check_update(orth(g), U.orthogonalize(to_f64(g)), f"{rows}x{cols}")


@pytest.mark.parametrize("count,rows,cols", [(65535, 2, 3), (65535, 33, 31), (3000, 1, 2100), (2000, 150, 500)])
def test_many_matrices(count, rows, cols):
    say(f"orthogonalize {count} x {rows} x {cols}")
    g = torch.randn(count, rows, cols, device="cuda")
    out = orth(g)
    for i in (0, 1, count // 2, count - 2, count - 1):
        check_update(out[i], U.orthogonalize(to_f64(g[i])), f"{i}")
    # (the buffer held 9: every matrix is written)
    assert (out != 9.0).all() and torch.isfinite(out).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_of_more_than_two_to_the_31_rows(kind):
    # one column: rms y = x / sqrt(x^2 + eps); layer norm y = 0, and its gradient is 0
    rows = (1 << 31) + 7
    say(f"norm {rows} x 1 bf16 {kind}")
    x = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda").normal_()
    y = torch.full_like(x, 9.0)
    mean = torch.empty(rows, dtype=torch.float32, device="cuda")
    rstd = torch.empty(rows, dtype=torch.float32, device="cuda")
    k = M.MOE_NORM_LAYER if kind == "layer" else M.MOE_NORM_RMS
    M.moe_norm_forward(k, x, None, None, None, 1e-2, None, y, mean, rstd)
    dx, dg, db = torch.full_like(x, 9.0), f32(1), f32(1)
    ws = torch.empty(M.moe_norm_workspace_bytes(rows, 1), dtype=torch.uint8, device="cuda")
    M.moe_norm_backward(k, y, x, None, mean, rstd, None, dx, dg, db, ws)
    torch.cuda.synchronize()
    for part in (slice(0, 5000), slice(rows - 5000, rows)):
        xs, ys, rs = x[part, 0].double(), y[part, 0].double(), rstd[part].double()
        v = xs if kind == "rms" else 0 * xs
        want = v / (v * v + 1e-2).sqrt()
        assert ((ys - want).abs() <= b16 * want.abs() + 8 * u32).all()
        assert ((rs * (v * v + 1e-2).sqrt() - 1).abs() <= 8 * u32).all()
        # t = y: rstd (y - h (y h)), h = x rstd
        h = v * rs
        grad = rs * (ys - h * (ys * h)) if kind == "rms" else 0 * ys
        assert ((dx[part, 0].double() - grad).abs() <= b16 * grad.abs() + 16 * u32 * rs * ys.abs()).all()
    if kind == "layer":
        assert (y == 0).all() and (dx == 0).all() and float(dg) == 0.0 and float(db) == 0.0


def test_two_calls_beside_each_other():
    """Calls on two streams, a workspace each, queued in turn: the bits of the calls alone."""
    say("norm and update on two streams")
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    shapes = [(4, 300, 500), (6, 130, 700)]

    def state(i):
        g, x, dy = rand(*shapes[i]), rand(3000, 1030), rand(3000, 1030)
        return dict(g=g, x=x, dy=dy, out=torch.empty_like(g), y=torch.empty_like(x), dx=torch.empty_like(x), mean=f32(3000),
                    rstd=f32(3000), dg=f32(1030), db=f32(1030),
                    ws=torch.empty(M.moe_orthogonalize_workspace_bytes(*shapes[i]), dtype=torch.uint8, device="cuda"),
                    nws=torch.empty(M.moe_norm_workspace_bytes(3000, 1030), dtype=torch.uint8, device="cuda"))

    def go(q, stream):
        M.moe_norm_forward(M.MOE_NORM_LAYER, q["x"], None, None, None, 1e-6, None, q["y"], q["mean"], q["rstd"], stream)
        M.moe_norm_backward(M.MOE_NORM_LAYER, q["dy"], q["x"], None, q["mean"], q["rstd"], None, q["dx"], q["dg"], q["db"],
                            q["nws"], stream)
        M.moe_orthogonalize(q["g"], None, 0.0, False, 5, 1e-7, 1.0, q["out"], q["ws"], stream)

    states, names = [state(0), state(1)], ("out", "y", "dx", "dg", "db")
    want = []
    for q in states:
        go(q, None)
        torch.cuda.synchronize()
        want.append({k: q[k].clone() for k in names})
        for k in names:
            q[k].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for q, s in zip(states, streams):
            go(q, s)
    torch.cuda.synchronize()
    for q, w in zip(states, want):
        assert all(torch.equal(q[k], w[k]) for k in names)
