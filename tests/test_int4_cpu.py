"""4-bit expert weights on the CPU: the oracle's reading against its definition,
and what the library refuses before anything is launched."""
import ctypes
import os

import numpy as np
import pytest

from mixture_experts_transformer_moe_amd import binding as M, configs
from oracle import int4_oracle as I

P = lambda k: ctypes.c_void_p(k << 40)  # noqa: E731  (addresses far apart: nothing overlaps)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        from mixture_experts_transformer_moe_amd.build import build
        build(verbose=False)
    return M.lib()


def bits(a):
    return (np.asarray(a, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def test_bf16_rounding_of_the_oracle():
    v = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -9, 0.0, 1e-40], np.float32)
    want = np.array([1.0, 1.0, 1 + 2.0 ** -6, 1.0, 0.0], np.float32)
    assert np.array_equal(I.bf16_round(v)[:5], want)
    assert abs(I.bf16_round(v)[5] - 1e-40) <= 2.0 ** -134


def test_quantize_reading():
    w = np.zeros((2, 64), np.float32)
    w[0, :8] = [7, -7, 0.5, 1.5, 2.5, -0.5, 3.49, -6.9]
    w[1, 32:] = 1.75                                     # scale 0.25: code 7; its first group zero
    codes, scale = I.quantize(bits(w), 32)
    assert scale[0].tolist() == [1.0, 1.0] and scale[1].tolist() == [1.0, 0.25]
    # ties to the even code; 3.49 and -6.9 as bf16 truncates them
    assert codes[0, :8].tolist() == [7, -7, 0, 2, 2, 0, 3, -7]
    assert (codes[1, :32] == 0).all() and (codes[1, 32:] == 7).all()
    rng = np.random.default_rng(0)
    w = bits(rng.normal(size=(5, 256)))
    for g in (32, 64, 128):
        c, s = I.quantize(w, g)
        # half a step of the code, and what the scale's rounding takes from the largest weight
        assert np.abs(I.dequantize(c, s) - I.bf16_to_f32(w)).max() <= (0.5 + 7 * 2.0 ** -8) * s.max()


def test_layout_holds_every_code_once():
    rng = np.random.default_rng(1)
    for rows, cols in ((16, 128), (48, 256), (32, 384)):
        where = np.zeros(rows * cols, np.int64)
        for n in range(8):                               # (one bit pattern at a time would be the same)
            flat = rng.integers(0, 256, rows * cols // 2).astype(np.uint8)
            got = I.unpack(flat, 1, rows, cols)
            hist = np.bincount((got.reshape(-1) + 8).astype(int), minlength=16)
            want = np.bincount(np.concatenate([flat & 15, flat >> 4]), minlength=16)
            assert np.array_equal(hist, want)
        # a single code set shows up at one place
        for i in rng.integers(0, rows * cols // 2, 50):
            flat = np.full(rows * cols // 2, 0x88, np.uint8)
            flat[i] = 0x8F
            assert np.count_nonzero(I.unpack(flat, 1, rows, cols)) == 1
            where[np.flatnonzero(I.unpack(flat, 1, rows, cols))[0]] += 1
        assert where.sum() == 50


def test_sizes(L):
    assert L.moe_int4_packed_bytes(256, 2048, 4096) == 256 * 2048 * 2048
    assert L.moe_int4_packed_bytes(1, 16, 128) == 1024
    for bad in ((1, 24, 128), (1, 16, 64), (-1, 16, 128), (1, -16, 128)):
        assert L.moe_int4_packed_bytes(*bad) == 0


def test_load_time_calls_check_arguments(L):
    quant = lambda *a: L.moe_quantize_weights_int4(*a, None)  # noqa: E731
    assert quant(P(1), P(2), P(3), 1, 16, 128, 48) == M.MOE_ERR_INVALID_ARG
    assert b"group" in L.moe_last_error()
    for rows, cols in ((24, 128), (16, 192)):
        assert quant(P(1), P(2), P(3), 1, rows, cols, 32) == M.MOE_ERR_INVALID_ARG
        assert L.moe_pack_weights_int4(P(1), P(2), 1, rows, cols, None) == M.MOE_ERR_INVALID_ARG
    assert quant(P(1), P(2), P(3), -1, 16, 128, 32) == M.MOE_ERR_INVALID_ARG
    assert quant(P(1), P(2), P(3), 1 << 40, 1 << 20, 1 << 20, 32) == M.MOE_ERR_UNSUPPORTED
    for k in range(3):
        args = [P(1), P(2), P(3)]
        args[k] = None
        assert quant(*args, 1, 16, 128, 32) == M.MOE_ERR_INVALID_ARG
        args[k] = ctypes.c_void_p((1 << 42) + 8)
        assert quant(*args, 1, 16, 128, 32) == M.MOE_ERR_INVALID_ARG
        assert b"aligned" in L.moe_last_error()
    for out in ((P(1), P(3)), (P(2), P(1)), (P(2), ctypes.c_void_p((2 << 40) + 512))):
        assert quant(P(1), *out, 1, 16, 128, 32) == M.MOE_ERR_INVALID_ARG
        assert b"overlap" in L.moe_last_error()
    assert quant(None, None, None, 0, 16, 128, 32) == M.MOE_OK
    assert L.moe_pack_weights_int4(P(1), ctypes.c_void_p((1 << 40) + 512), 1, 16, 128, None) == M.MOE_ERR_INVALID_ARG
    assert L.moe_pack_weights_int4(None, P(2), 1, 16, 128, None) == M.MOE_ERR_INVALID_ARG
    assert L.moe_pack_weights_int4(None, None, 1, 0, 128, None) == M.MOE_OK


def _shape(**kw):
    return M.make_shape(configs.variant(configs.XS2_T4096, **{**dict(T=64, E=16, k=4), **kw}))


def _calls(L, s, group):
    sp = ctypes.byref(s)
    up = lambda a: L.moe_grouped_gate_up_int4(sp, group, *a, None)  # noqa: E731
    down = lambda a: L.moe_grouped_down_int4(sp, group, *a, None)  # noqa: E731
    return (up, [None] + [P(k) for k in range(1, 9)]), (down, [P(k) for k in range(1, 9)])


def test_products_check_arguments(L):
    for group in (0, 16, 48, 256, -32):
        for call, args in _calls(L, _shape(), group):
            assert call(args) == M.MOE_ERR_INVALID_ARG
            assert b"group" in L.moe_last_error()
    for call, args in _calls(L, _shape(dtype="f32"), 32):
        assert call(args) == M.MOE_ERR_UNSUPPORTED
    for call, args in _calls(L, _shape(D=384), 32):
        assert call(args) == M.MOE_ERR_UNSUPPORTED
    for call, args in _calls(L, _shape(T=0), 32):
        assert call([None] * len(args)) == M.MOE_OK
    for call, args in _calls(L, _shape(), 64):
        for k in range(len(args)):
            bad = list(args)
            bad[k] = ctypes.c_void_p((1 << 44) + 4)
            assert call(bad) == M.MOE_ERR_INVALID_ARG
            assert b"aligned" in L.moe_last_error()
            if args[k] is not None:
                bad[k] = None
                assert call(bad) == M.MOE_ERR_INVALID_ARG
                assert b"NULL" in L.moe_last_error()
    # each output over each input, by its last bytes
    for (call, args), outs in zip(_calls(L, _shape(), 64), ((8,), (6, 7))):
        for o in outs:
            for k in range(len(args)):
                if k == o or args[k] is None:
                    continue
                bad = list(args)
                bad[k] = ctypes.c_void_p(args[o].value + 64)
                assert call(bad) == M.MOE_ERR_INVALID_ARG, (o, k)
                assert b"overlap" in L.moe_last_error()


def test_binding_checks_tensors():
    import torch
    z = lambda n, dt=torch.bfloat16: torch.zeros(n, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError):
        M.moe_quantize_weights_int4(z(16 * 128), z(16 * 64, torch.uint8), z(64), 1, 16, 128, 32)   # host tensors
    with pytest.raises(M.MoEError):
        M.quantize_int4(torch.zeros(24, 128, dtype=torch.bfloat16), 32)
    with pytest.raises(M.MoEError):
        M.quantize_int4(torch.zeros(16, 128, dtype=torch.bfloat16), 48)
    with pytest.raises(ValueError):
        M.upload_weights(configs.XS2_T4096, None, None, None, None, None, fp8=True, int4=32)
