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
