"""More of the head's loss on the CPU: empty batches."""
import os

import pytest

from mixture_experts_transformer_moe_amd import binding as M


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        from mixture_experts_transformer_moe_amd.build import build
        build(verbose=False)
    return M.lib()


def test_an_empty_batch_needs_no_outputs(L):
    # an empty tensor's address is NULL: dx [0, cols] alone is a call like any other
    none = [None] * 8
    assert L.moe_head_loss_backward(0, 64, 1000, M.MOE_BF16, *none, 0, None) == M.MOE_OK
    # its sizes are checked all the same
    assert L.moe_head_loss_backward(0, 60, 1000, M.MOE_BF16, *none, 0, None) == M.MOE_ERR_UNSUPPORTED
    assert L.moe_head_loss_backward(0, 64, 0, M.MOE_BF16, *none, 0, None) == M.MOE_ERR_INVALID_ARG
