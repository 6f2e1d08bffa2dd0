"""The pre-norm and the orthogonalised update without a GPU: the oracle against
differences and singular values, and the refusals of the C entry points."""
import ctypes
import os

import numpy as np
import pytest

from mixture_experts_transformer_moe_amd import binding
from oracle import update_oracle as U


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        from mixture_experts_transformer_moe_amd.build import build
        build(verbose=False)
    return binding.lib()


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_backward_against_differences(kind):
    rng = np.random.default_rng(1)
    s, dy = rng.normal(size=(5, 7)) + 0.3, rng.normal(size=(5, 7))
    gamma, beta = rng.normal(size=7), rng.normal(size=7)
    _, mean, rstd = U.norm_forward(kind, s, gamma, beta)
    ds, dg, db = U.norm_backward(kind, dy, s, gamma, mean, rstd)
    f = lambda s, g, b: float((U.norm_forward(kind, s, g, b)[0] * dy).sum())  # noqa: E731
    h = 1e-5
    for got, at in ((ds, 0), (dg, 1), (db, 2)):
        for i in np.ndindex(got.shape):
            hi, lo = [s.copy(), gamma.copy(), beta.copy()], [s.copy(), gamma.copy(), beta.copy()]
            hi[at][i] += h
            lo[at][i] -= h
            # central differences: error h^2 times a third derivative of order 10
            assert abs((f(*hi) - f(*lo)) / (2 * h) - got[i]) < 1e-7


def test_layer_norm_gradient_is_orthogonal_to_the_row():
    # dx has no component along ones and (up to eps) along the normalised row
    rng = np.random.default_rng(2)
    s, dy = rng.normal(size=(3, 50)), rng.normal(size=(3, 50))
    _, mean, rstd = U.norm_forward("layer", s, eps=1e-12)
    ds, _, _ = U.norm_backward("layer", dy, s, None, mean, rstd)
    assert np.abs(ds.sum(1)).max() < 1e-12
    assert np.abs((ds * (s - mean[:, None])).sum(1)).max() < 1e-9


@pytest.mark.parametrize("shape", [(6, 9), (9, 6), (1, 5), (5, 1), (1, 1)])
def test_orthogonalize_acts_on_the_singular_values(shape):
    rng = np.random.default_rng(3)
    g = rng.normal(size=shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.linalg.norm(g) + 1e-7)
    for _ in range(5):
        s = U.A * s + U.B * s ** 3 + U.C * s ** 5
    # (1e-7 enters as the fp32 number: 1e-9 relative at most)
    np.testing.assert_allclose(U.orthogonalize(g), (u * s) @ vt, rtol=0, atol=1e-6)


def test_momentum_forms():
    g, m = np.array([[1.0, 2.0]]), np.array([[4.0, 8.0]])
    u, after = U.update_of(g, m, 0.5, True)
    assert after.tolist() == [[3.0, 6.0]] and u.tolist() == [[2.5, 5.0]]
    u, after = U.update_of(g, m, 0.5, False)
    assert u.tolist() == after.tolist() == [[3.0, 6.0]]
    assert U.update_of(g)[1] is None


# ------------------------------------------------------------------- refusals

P = lambda i: ctypes.c_void_p(i << 32)  # noqa: E731  (distinct, 16-byte aligned, far apart; never dereferenced)


def _fwd(L, kind=1, rows=4, cols=64, dtype=1, x=P(1), res=None, gamma=P(2), beta=None, eps=1e-6, sum=None, y=P(3),
         mean=None, rstd=P(4)):
    return L.moe_norm_forward(kind, rows, cols, dtype, x, res, gamma, beta, eps, sum, y, mean, rstd, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(kind=2), binding.MOE_ERR_INVALID_ARG, b"kind"),
    (dict(dtype=2), binding.MOE_ERR_INVALID_ARG, b"dtype"),
    (dict(rows=-1), binding.MOE_ERR_INVALID_ARG, b"rows"),
    (dict(cols=0), binding.MOE_ERR_INVALID_ARG, b"cols"),
    (dict(cols=16385), binding.MOE_ERR_UNSUPPORTED, b"16384"),
    (dict(eps=0.0), binding.MOE_ERR_INVALID_ARG, b"eps"),
    (dict(eps=float("nan")), binding.MOE_ERR_INVALID_ARG, b"eps"),
    (dict(eps=float("inf")), binding.MOE_ERR_INVALID_ARG, b"eps"),
    (dict(x=None), binding.MOE_ERR_INVALID_ARG, b"x is NULL"),
    (dict(y=None), binding.MOE_ERR_INVALID_ARG, b"y is NULL"),
    (dict(x=ctypes.c_void_p((1 << 32) + 2)), binding.MOE_ERR_INVALID_ARG, b"aligned"),
    (dict(gamma=ctypes.c_void_p((2 << 32) + 4)), binding.MOE_ERR_INVALID_ARG, b"aligned"),
    (dict(res=P(5)), binding.MOE_ERR_INVALID_ARG, b"sum"),
    (dict(sum=P(5)), binding.MOE_ERR_INVALID_ARG, b"sum"),
    (dict(res=P(5), sum=P(3)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(y=ctypes.c_void_p((1 << 32) + 16)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(rstd=P(1)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(kind=0, mean=P(9), rstd=P(9)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(gamma=P(7), y=P(7)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
])
def test_norm_forward_refusals(L, kw, status, word):
    assert _fwd(L, **kw) == status
    assert word in L.moe_last_error()


def test_norm_forward_of_no_rows_is_a_no_op(L):
    assert _fwd(L, rows=0, x=None, y=None, gamma=None, rstd=None) == binding.MOE_OK


def _bwd(L, kind=0, rows=4, cols=64, dtype=1, dy=P(1), x=P(2), gamma=P(3), mean=P(4), rstd=P(5), dsum=None, dx=P(6),
         dgamma=P(7), dbeta=P(8), ws=P(9), nbytes=None):
    if nbytes is None:
        nbytes = L.moe_norm_workspace_bytes(max(rows, 0), max(cols, 1))
    return L.moe_norm_backward(kind, rows, cols, dtype, dy, x, gamma, mean, rstd, dsum, dx, dgamma, dbeta, ws, nbytes,
                               None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(kind=-1), binding.MOE_ERR_INVALID_ARG, b"kind"),
    (dict(rows=-3), binding.MOE_ERR_INVALID_ARG, b"rows"),
    (dict(cols=20000), binding.MOE_ERR_UNSUPPORTED, b"cols"),
    (dict(dy=None), binding.MOE_ERR_INVALID_ARG, b"dy is NULL"),
    (dict(mean=None), binding.MOE_ERR_INVALID_ARG, b"mean is NULL"),
    (dict(rstd=None), binding.MOE_ERR_INVALID_ARG, b"rstd is NULL"),
    (dict(dx=None), binding.MOE_ERR_INVALID_ARG, b"dx is NULL"),
    (dict(ws=None), binding.MOE_ERR_WORKSPACE, b"workspace"),
    (dict(nbytes=8), binding.MOE_ERR_WORKSPACE, b"workspace"),
    (dict(dx=ctypes.c_void_p((2 << 32) + 64)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(dx=P(5)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(dbeta=P(7)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(dgamma=P(3)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(ws=P(1)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(ws=P(8)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
])
def test_norm_backward_refusals(L, kw, status, word):
    assert _bwd(L, **kw) == status
    assert word in L.moe_last_error()


def test_norm_workspace_sizes(L):
    assert L.moe_norm_workspace_bytes(0, 64) == 0
    assert L.moe_norm_workspace_bytes(-1, 64) == 0
    assert L.moe_norm_workspace_bytes(4, 0) == 0
    assert L.moe_norm_workspace_bytes(4, 16385) == 0
    n = L.moe_norm_workspace_bytes(1 << 20, 4096)
    assert n % 256 == 0 and 2 * 4096 * 4 <= n <= 64 << 20


def _orth(L, count=2, rows=64, cols=96, dtype=1, g=P(1), mom=None, mu=0.95, nesterov=1, steps=5, eps=1e-7, scale=1.0,
          out=P(2), ws=P(3), nbytes=None):
    if nbytes is None:
        nbytes = L.moe_orthogonalize_workspace_bytes(max(count, 0), max(rows, 0), max(cols, 0))
    return L.moe_orthogonalize(count, rows, cols, dtype, g, mom, mu, nesterov, steps, eps, scale, out, ws, nbytes, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(count=-1), binding.MOE_ERR_INVALID_ARG, b"negative"),
    (dict(rows=-1), binding.MOE_ERR_INVALID_ARG, b"negative"),
    (dict(count=65536), binding.MOE_ERR_UNSUPPORTED, b"count"),
    (dict(rows=65537, cols=8), binding.MOE_ERR_UNSUPPORTED, b"65536"),
    (dict(rows=8, cols=65537), binding.MOE_ERR_UNSUPPORTED, b"65536"),
    (dict(rows=1 << 15, cols=1 << 15), binding.MOE_ERR_UNSUPPORTED, b"2^30"),
    (dict(count=65535, rows=1024, cols=1025), binding.MOE_ERR_UNSUPPORTED, b"2^36"),
    (dict(dtype=3), binding.MOE_ERR_INVALID_ARG, b"dtype"),
    (dict(steps=0), binding.MOE_ERR_INVALID_ARG, b"steps"),
    (dict(steps=17), binding.MOE_ERR_INVALID_ARG, b"steps"),
    (dict(eps=-1e-9), binding.MOE_ERR_INVALID_ARG, b"eps"),
    (dict(eps=float("nan")), binding.MOE_ERR_INVALID_ARG, b"eps"),
    (dict(scale=float("inf")), binding.MOE_ERR_INVALID_ARG, b"scale"),
    (dict(mom=P(4), mu=1.0), binding.MOE_ERR_INVALID_ARG, b"mu"),
    (dict(mom=P(4), mu=-0.1), binding.MOE_ERR_INVALID_ARG, b"mu"),
    (dict(mom=P(4), mu=float("nan")), binding.MOE_ERR_INVALID_ARG, b"mu"),
    (dict(g=None), binding.MOE_ERR_INVALID_ARG, b"g is NULL"),
    (dict(out=None), binding.MOE_ERR_INVALID_ARG, b"out is NULL"),
    (dict(g=ctypes.c_void_p((1 << 32) + 8)), binding.MOE_ERR_INVALID_ARG, b"aligned"),
    (dict(ws=None), binding.MOE_ERR_WORKSPACE, b"workspace"),
    (dict(nbytes=128), binding.MOE_ERR_WORKSPACE, b"workspace"),
    (dict(rows=256, cols=1024, nbytes=1 << 20), binding.MOE_ERR_WORKSPACE, b"workspace"),
    (dict(dtype=0, out=P(1)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(out=ctypes.c_void_p((1 << 32) + 16)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(mom=P(2)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
    (dict(ws=P(1)), binding.MOE_ERR_INVALID_ARG, b"overlap"),
])
def test_orthogonalize_refusals(L, kw, status, word):
    assert _orth(L, **kw) == status
    assert word in L.moe_last_error()


def test_orthogonalize_of_nothing_is_a_no_op(L):
    for kw in (dict(count=0), dict(rows=0), dict(cols=0)):
        assert _orth(L, g=None, out=None, ws=None, nbytes=0, **kw) == binding.MOE_OK
    assert L.moe_orthogonalize_workspace_bytes(0, 64, 64) == 0
    assert L.moe_orthogonalize_workspace_bytes(3, 0, 64) == 0
    assert L.moe_orthogonalize_workspace_bytes(-1, 64, 64) == 0


def test_orthogonalize_workspace_does_not_depend_on_orientation(L):
    a = L.moe_orthogonalize_workspace_bytes(3, 100, 700)
    assert a == L.moe_orthogonalize_workspace_bytes(3, 700, 100) and a > 0 and a % 256 == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    x, rms = torch.zeros(4, 8), binding.MOE_NORM_RMS
    with pytest.raises(ValueError, match="device tensors"):
        binding.moe_norm_forward(rms, x, None, None, None, 1e-6, None, None, None, None)
    with pytest.raises(ValueError, match="device tensors"):
        binding.moe_orthogonalize(x, None, 0.0, True, 5, 1e-7, 1.0, None, None)
    with pytest.raises(ValueError, match="gamma is"):
        binding.moe_norm_forward(rms, x, None, torch.zeros(7), None, 1e-6, None, None, None, None)
    with pytest.raises(ValueError, match="mean is"):
        binding.moe_norm_forward(rms, x, None, None, None, 1e-6, None, None, torch.zeros(8), None)
    with pytest.raises(ValueError, match="y is"):
        binding.moe_norm_forward(rms, x, None, None, None, 1e-6, None, torch.zeros(4, 9), None, None)
    with pytest.raises(ValueError, match="rstd is"):
        binding.moe_norm_forward(rms, x, None, None, None, 1e-6, None, None, None, torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        binding.moe_norm_forward(rms, x.half(), None, None, None, 1e-6, None, None, None, None)
    with pytest.raises(ValueError, match="dy is"):
        binding.moe_norm_backward(rms, torch.zeros(4, 7), x, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="out is"):
        binding.moe_orthogonalize(x, None, 0.0, True, 5, 1e-7, 1.0, x.clone(), None)
    with pytest.raises(ValueError, match="momentum is"):
        binding.moe_orthogonalize(x, torch.zeros(8, 4), 0.0, True, 5, 1e-7, 1.0, None, None)
    with pytest.raises(ValueError, match="rows, cols"):
        binding.moe_orthogonalize(torch.zeros(4), None, 0.0, True, 5, 1e-7, 1.0, None, None)
    with pytest.raises(ValueError, match="rows, cols"):
        binding.moe_norm_backward(rms, x, torch.zeros(8), None, None, None, None, None, None, None, None)
