"""Workspaces of the pre-norm's backward pass and of the orthogonalised update
over ranges of sizes, and the kernels that sizes choose, without a GPU."""
import os
import re

import pytest

from mixture_experts_transformer_moe_amd import binding


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        from mixture_experts_transformer_moe_amd.build import build
        build(verbose=False)
    return binding.lib()


@pytest.mark.parametrize("cols", [1, 64, 100, 256, 300, 513, 1000, 1024, 2048, 4100, 6000, 8192, 16384])
def test_norm_workspace_of_a_larger_batch_serves_a_smaller_one(L, cols):
    # a program whose batches vary keeps the workspace of its largest
    rows = list(range(1, 5000)) + [8191, 8192, 8193, 32768, 140000, 1 << 20, (1 << 40) - 1]
    sizes = [L.moe_norm_workspace_bytes(r, cols) for r in rows]
    down = [(a, b) for (a, x), (b, y) in zip(zip(rows, sizes), zip(rows[1:], sizes[1:])) if y < x]
    assert not down, f"{len(down)}, the first {down[0]}"
    # one row of sums of dgamma and one of dbeta, at most four workgroups a CU
    assert 2 * 4 * cols <= sizes[0] and sizes[-1] <= 256 * 4 * 2 * 4 * cols + 255


@pytest.mark.parametrize("rows,cols", [(1, 3000), (64, 200), (130, 600), (256, 256), (300, 2000), (1024, 2048), (2048, 512)])
def test_update_workspace_grows_with_the_count(L, rows, cols):
    sizes = [L.moe_orthogonalize_workspace_bytes(n, rows, cols) for n in range(1, 300)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[0] > 0


def test_norm_kernels_built_are_those_some_size_reaches(L):
    # batches of few rows take one vector a thread, or 1024 threads a row; only
    # they sum the columns by workgroups of their own (the last argument, 2)
    few = {(1, 16), (1, 32), (1, 64), (1, 256), (1, 1024), (2, 1024)}
    many = few | {(2, 64), (2, 256), (3, 256)}
    names = open(binding.LIB_PATH, "rb").read()
    built = {(t, int(ch), int(tpr), int(sums)) for t, ch, tpr, sums in
             re.findall(rb"norm_backward_kernelI([tf])Li(\d+)ELi(\d+)ELi(\d)E", names)}
    want = set()
    for t in (b"t", b"f"):
        wide = {(4, 1024)} if t == b"f" else set()
        want |= {(t, *f, 2) for f in few | wide} | {(t, *f, s) for f in many | wide for s in (0, 1)}
    assert built == want
