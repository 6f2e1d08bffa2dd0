"""More of the head's loss on the GPU: empty batches."""
import pytest
import torch

from mixture_experts_transformer_moe_amd import binding as M

pytestmark = pytest.mark.gpu


def test_empty_batch_with_a_frozen_head():
    # dx alone, as a step takes it that does not train the head, on a rank with no rows
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(9, 64, dtype=torch.bfloat16, device="cuda")
    y, e = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    M.moe_head_loss_backward(x, w, y, e, e, torch.empty_like(x), None, None)
    torch.cuda.synchronize()
    assert (w == 1).all()


@pytest.mark.parametrize("rows,cols,vocab", [(512, 512, 4000), (40, 256, 3000), (2000, 1024, 9000)])
@pytest.mark.parametrize("kind", ["rival", "both"])
def test_rows_with_a_rival(kind, rows, cols, vocab):
    """hidden states that point at an entry that is not their target, or at both: beside the
    outputs' own rounding, 2^-8 / sqrt 3 of a value at most on average, there is P's, as much
    of each entry but the target's, common to the entry's whole row of w (of x)"""
    g = torch.Generator(device="cuda").manual_seed(rows)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = randn(vocab, cols).mul_(0.02).to(torch.bfloat16)
    y, rival = (torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32) for _ in range(2))
    at = lambda i: w[i.long()].float() / w[i.long()].float().square().sum(1, keepdim=True)  # noqa: E731
    x = (randn(rows, cols) + 14 * at(rival) + (14 * at(y) if kind == "both" else 0)).to(torch.bfloat16)
    dloss = (0.5 + torch.rand(rows, generator=g, device="cuda")) / rows
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(M.moe_head_loss_workspace_bytes(rows, cols, vocab), dtype=torch.uint8, device="cuda")
    M.moe_head_loss_forward(x, w, y, loss, lse, ws)
    M.moe_head_loss_backward(x, w, y, lse, dloss, dx, dw, ws)
    p = torch.exp(x.double() @ w.double().T - lse.double()[:, None])
    t = torch.arange(rows, device="cuda"), y.long()
    p[t] -= 1.0
    p *= dloss.double()[:, None]
    rounded = p.clone()
    rounded[t] = 0.0                                       # (the target's entry is held finer)
    for name, got, want, entries, m in (("dx", dx, p @ w.double(), rounded, w), ("dw", dw, p.T @ x.double(), rounded.T, x)):
        common = (entries.square().sum(0) * m.double().square().sum(1)).sum()
        off = (got.double() - want).norm()
        # (a tenth for what the sums over a few hundred large entries vary by)
        assert off <= 1.1 * 2.0 ** -8 / 3 ** 0.5 * (want.square().sum() + common).sqrt(), name
