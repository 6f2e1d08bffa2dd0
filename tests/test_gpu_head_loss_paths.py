"""Each path of the head's loss (tests/head_loss_paths.py) against float64 on the GPU, every
output.

The tolerances are those that tests/test_gpu_head_loss.py derives, with two terms that
grow here: the join adds vocab / 8192 tiles a lane at most, and dx's sum over parts and
pieces as many terms as there are.
"""
import pytest
import torch

from mixture_experts_transformer_moe_amd import binding as M
from tests.gpu_common import say
from tests.head_loss_paths import PATHS

pytestmark = pytest.mark.gpu

u32, b16 = 2.0 ** -24, 2.0 ** -8


def banded(n, dtype):
    """(buffer, its middle n elements); 7 outside"""
    t = torch.full((n + 256,), 7.0, dtype=dtype, device="cuda")
    return t, t[128:128 + n]


def within(name, got, want, tol):
    bad = ~((got - want).abs() <= tol)                     # (NaN counts)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()}, worst {float(((got - want).abs() / tol).max()):.2f}"


@pytest.mark.parametrize("name", PATHS)
def test_path(name):
    (rows, cols, vocab), _, _, _, _, pieces, parts = PATHS[name]
    say(f"head loss {rows} x {cols} over {vocab}: {name}")
    g = torch.Generator(device="cuda").manual_seed(rows + vocab)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = (randn(vocab, cols) / cols ** 0.5).to(torch.bfloat16)
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    x = (2 * randn(rows, cols) + 6 * torch.rand(rows, 1, generator=g, device="cuda") * w[y.long()].float()).to(torch.bfloat16)
    y[torch.rand(rows, generator=g, device="cuda") < 0.1] = -100
    y[torch.rand(rows, generator=g, device="cuda") < 0.05] = vocab
    dloss = randn(rows) / rows
    (bl, loss), (bs, lse) = banded(rows, torch.float32), banded(rows, torch.float32)
    (bx, dx), (bw, dw) = banded(rows * cols, torch.bfloat16), banded(vocab * cols, torch.bfloat16)
    n = M.moe_head_loss_workspace_bytes(rows, cols, vocab)
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")       # (NaN as any type)
    work = ws[256:256 + n]
    M.moe_head_loss_forward(x, w, y, loss, lse, work)
    work.fill_(255)
    M.moe_head_loss_backward(x, w, y, lse, dloss, dx.view(rows, cols), dw.view(vocab, cols), work)
    torch.cuda.synchronize()
    for t in (bl, bs, bx, bw):
        assert (t[:128] == 7.0).all() and (t[-128:] == 7.0).all()
    assert (ws[:256] == 255).all() and (ws[-256:] == 255).all()

    say("in float64")
    dx, dw = dx.view(rows, cols).double(), dw.view(vocab, cols).double()
    w64 = w.double()
    zero = lambda: torch.zeros(vocab, cols, dtype=torch.float64, device="cuda")  # noqa: E731
    want_w, err_w, sq_w, ab_w = zero(), zero(), zero(), zero()
    dots = (cols / 16 + 6) * u32
    off = ref = 0.0
    step = max(1, int(1.5e8) // vocab)
    for i in range(0, rows, step):
        s = slice(i, min(i + step, rows))
        on = (y[s] >= 0) & (y[s] < vocab)
        t = torch.where(on, y[s], 0).long()[:, None]
        xs, gs = x[s].double() * on[:, None], (dloss[s] * on).double()
        z = xs @ w64.T
        top = torch.logsumexp(z, 1)
        zt = z.gather(1, t)[:, 0]
        e = dots * (xs.abs() @ w64.abs().T).max(1).values
        tol = e + 5e-6 + (100 + vocab / 8192) * u32 + 4 * u32 * top.abs()
        assert (loss[s][~on] == 0).all() and (lse[s][~on] == 0).all()
        within("lse", lse[s][on].double(), top[on], tol[on])
        tol = tol + e + 4 * u32 * (top.abs() + zt.abs())
        within("loss", loss[s][on].double(), (top - zt)[on], tol[on])
        # P from the lse the kernel left
        p = z.sub_(lse[s].double()[:, None]).exp_() * gs[:, None]
        q = p.abs()
        ep = q * (e[:, None] + 5e-6) + 4 * u32 * gs.abs()[:, None] * (q > 0)
        p.scatter_add_(1, t, -gs[:, None])
        q = p.abs()
        want = p @ w64
        squares = (p * p) @ (w64 * w64)
        tol = ep @ w64.abs() + 8 * b16 / 1.7 * squares.sqrt() + b16 * want.abs()
        tol += (vocab / 16 + 38 + max(parts) + pieces) * u32 * (q @ w64.abs()) + 1e-37
        within("dx", dx[s], want, tol)
        assert (dx[s][~on] == 0).all()
        off += float((dx[s] - want).square().sum())
        ref += float(want.square().sum() + squares.sum())
        want_w += p.T @ xs
        err_w += ep.T @ xs.abs()
        sq_w += (p * p).T @ (xs * xs)
        ab_w += q.T @ xs.abs()
    assert off ** 0.5 <= 1.5 * b16 * ref ** 0.5
    tol = err_w + 8 * b16 / 1.7 * sq_w.sqrt() + b16 * want_w.abs() + (rows / 16 + 38) * u32 * ab_w + 1e-37
    within("dw", dw, want_w, tol)
    assert float((dw - want_w).norm()) <= 1.5 * b16 * float(want_w.square().sum() + sq_w.sum()) ** 0.5
