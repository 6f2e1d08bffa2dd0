"""The head's loss on the CPU: the oracle against differences, and what the library
refuses before anything is launched."""
import ctypes
import os

import numpy as np
import pytest

from mixture_experts_transformer_moe_amd import binding as M
from oracle import loss_oracle as O

P = lambda k: ctypes.c_void_p(k << 42)  # noqa: E731  (far apart: nothing overlaps)
BIG = 1 << 41


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        from mixture_experts_transformer_moe_amd.build import build
        build(verbose=False)
    return M.lib()


def test_oracle_gradients_match_differences():
    rng = np.random.default_rng(0)
    x, w = rng.normal(size=(6, 5)), rng.normal(size=(9, 5))
    y, g = np.array([0, 8, -1, 3, 9, 3]), rng.normal(size=6)
    value = lambda x, w: (O.forward(x, w, y)[0] * g).sum()  # noqa: E731
    loss, lse = O.forward(x, w, y)
    assert loss[2] == lse[2] == loss[4] == 0 and (loss[[0, 1, 3, 5]] > 0).all()
    dx, dw = O.backward(x, w, y, lse, g)
    h = 1e-6
    for a, da, of in ((x, dx, 0), (w, dw, 1)):
        for i in np.ndindex(a.shape):
            hi, lo = a.copy(), a.copy()
            hi[i] += h
            lo[i] -= h
            d = (value(hi, w) - value(lo, w) if of == 0 else value(x, hi) - value(x, lo)) / (2 * h)
            assert abs(d - da[i]) < 1e-7
    assert (dx[[2, 4]] == 0).all()
    # a row that takes no part may hold anything
    x[2] = np.nan
    again = O.backward(x, w, y, lse, g)
    assert np.array_equal(again[0], dx) and np.allclose(again[1], dw, rtol=1e-14, atol=0)


def test_workspace_sizes(L):
    size = L.moe_head_loss_workspace_bytes
    assert size(0, 64, 1000) == 0 and size(-1, 64, 1000) == 0
    for bad in ((16, 12, 1000), (16, 0, 1000), (16, 64, 0), (16, 65544, 1000), (1 << 22, 64, 10), (1 << 21, 64, 1 << 22)):
        assert size(*bad) == 0, bad
    # at least the forward pass's 8 bytes a row and tile, and P's piece both ways
    for rows, cols, vocab in ((1, 8, 1), (999, 2048, 50021), (8192, 4096, 100352)):
        n = size(rows, cols, vocab)
        assert n % 256 == 0 and n >= rows * ((vocab + 255) // 256) * 8
    # pieces bound it: neither the logits nor a probability matrix of the whole batch
    assert size(8192, 4096, 100352) < 2 * 8192 * 100352
    assert size(65536, 4096, 100352) < 65536 * 100352


def forward(L, rows=16, cols=64, vocab=1000, dtype=M.MOE_BF16, args=None, nbytes=BIG):
    a = args or [P(k) for k in range(1, 7)]
    return L.moe_head_loss_forward(rows, cols, vocab, dtype, *a, nbytes, None)


def backward(L, rows=16, cols=64, vocab=1000, dtype=M.MOE_BF16, args=None, nbytes=BIG):
    a = args or [P(k) for k in range(1, 9)]
    return L.moe_head_loss_backward(rows, cols, vocab, dtype, *a, nbytes, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_bad_sizes(L, call):
    for kw, status in ((dict(rows=-1), 1), (dict(cols=0), 1), (dict(vocab=0), 1), (dict(dtype=7), 1),
                       (dict(dtype=M.MOE_F32), 2), (dict(cols=60), 2), (dict(cols=65544), 2), (dict(rows=1 << 22), 2),
                       (dict(vocab=1 << 23), 2), (dict(rows=1 << 21, vocab=1 << 22), 2)):
        assert call(L, **kw) == status, kw
        assert L.moe_last_error()


@pytest.mark.parametrize("call,n,optional", [(forward, 6, ()), (backward, 8, (5, 6))])
def test_bad_pointers(L, call, n, optional):
    ws = n - 1
    for k in range(n):
        args = [P(i) for i in range(1, n + 1)]
        args[k] = ctypes.c_void_p((k + 1 << 42) + 4)
        assert call(L, args=args) == (M.MOE_ERR_WORKSPACE if k == ws else M.MOE_ERR_INVALID_ARG), k
        assert b"aligned" in L.moe_last_error()
        if k not in optional:
            args[k] = None
            assert call(L, args=args) == (M.MOE_ERR_WORKSPACE if k == ws else M.MOE_ERR_INVALID_ARG), k
    need = L.moe_head_loss_workspace_bytes(16, 64, 1000)
    assert call(L, nbytes=need - 1) == M.MOE_ERR_WORKSPACE
    # an output, or the workspace, over any other argument
    for o in ((3, 4, 5) if call is forward else (5, 6, 7)):
        for k in range(n):
            if k == o:
                continue
            args = [P(i) for i in range(1, n + 1)]
            args[k] = ctypes.c_void_p(args[o].value + 32)
            assert call(L, args=args) == M.MOE_ERR_INVALID_ARG, (o, k)
            assert b"overlap" in L.moe_last_error()


def test_empty_calls(L):
    assert forward(L, rows=0, args=[None] * 6, nbytes=0) == M.MOE_OK
    # nothing to write without dw
    assert backward(L, rows=0, args=[None] * 5 + [P(1), None, None], nbytes=0) == M.MOE_OK
    assert backward(L, args=[P(1), P(2), P(3), P(4), P(5), None, None, P(6)]) == M.MOE_ERR_INVALID_ARG


def test_binding_checks_tensors():
    import torch
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(10, 16, dtype=torch.bfloat16)
    y, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError):
        M.moe_head_loss_forward(x, w, y, f, f.clone(), None)                          # host tensors
    with pytest.raises(ValueError):
        M.moe_head_loss_forward(x, w[:, :8].contiguous(), y, f, f.clone(), None)     # another width
    with pytest.raises(ValueError):
        M.moe_head_loss_forward(x, w, y.long(), f, f.clone(), None)                  # another type


def test_workspace_does_not_shrink(L):
    for cols, vocab in ((4096, 100352), (1000, 33001), (8, 9000), (65536, 3)):
        sizes = [L.moe_head_loss_workspace_bytes(rows, cols, vocab) for rows in range(1, 40000, 97)]
        assert sizes == sorted(sizes) and sizes[0] > 0
