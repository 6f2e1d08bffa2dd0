"""CPU oracle of 4-bit expert weights (test infrastructure only).

Only the tests and the smoke check may import this module; the product path
never does.  It shares no code with the HIP path.

The pages list INT4 among the quantised releases of the MoE layers ("Laguna
M.1/XS.2 Technical Report", Key claims) without encoding details; the reading,
as include/moe.h states it: integers -8..7, one bf16 scale a row and group of
consecutive columns, scale = bf16(max |w| / 7) in fp32 (1 where that is zero),
code = w / scale (fp32 quotient) to the nearest integer, ties to even.
"""
from __future__ import annotations

from typing import Tuple

import numpy as np


def bf16_round(v: np.ndarray) -> np.ndarray:
    """float32 -> the nearest bf16 value (ties to even), as float32; finite input."""
    u = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)).view(np.float32)


def bf16_to_f32(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32)


def quantize(w_bits: np.ndarray, group: int) -> Tuple[np.ndarray, np.ndarray]:
    """(codes int8 [..., rows, cols], scales float32 [..., rows, cols / group]) of bf16 bit patterns."""
    w = bf16_to_f32(w_bits)
    g = w.reshape(*w.shape[:-1], w.shape[-1] // group, group)
    scale = bf16_round(np.abs(g).max(-1) / np.float32(7.0))
    scale = np.where(scale == 0, np.float32(1.0), scale).astype(np.float32)
    q = (g / scale[..., None]).astype(np.float32)
    codes = np.clip(np.rint(q.astype(np.float64)), -8, 7).astype(np.int8)
    return codes.reshape(w.shape), scale


def dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 weights code * scale."""
    s = np.asarray(scales, np.float64)
    return np.asarray(codes, np.float64) * np.repeat(s, codes.shape[-1] // s.shape[-1], axis=-1)


def two_a_byte(codes: np.ndarray) -> np.ndarray:
    """Row-major bytes of moe_pack_weights_int4: column 2j in the low half, 2j + 1 in the high half, each + 8."""
    c = (np.asarray(codes, np.int16) + 8).astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def unpack(flat: np.ndarray, count: int, rows: int, cols: int) -> np.ndarray:
    """Codes [count, rows, cols] from the packed layout include/moe.h documents."""
    r = np.arange(rows)[:, None]
    c = np.arange(cols)[None, :]
    word = ((r // 16) * (cols // 128) + c // 128) * 256 + ((r % 16) + 16 * ((c % 32) // 8)) * 4 + (c % 128) // 32
    shift = 4 * ((c % 8) // 2 + 4 * (c % 2))
    words = np.ascontiguousarray(flat).view("<u4").reshape(count, -1)
    return np.stack([((m[word] >> shift.astype(np.uint32)) & 15).astype(np.int16) - 8 for m in words]).astype(np.int8)


class Int4Weights:
    """A layer's inputs with every expert weight matrix replaced by its 4-bit reading (see Fp8Weights)."""

    def __init__(self, inputs, group: int):
        self._inputs, self._group = inputs, group
        self.x = inputs.x
        self.w_router = inputs.w_router
        self.bias = inputs.bias

    def _read(self, w):
        return dequantize(*quantize(w, self._group))

    def expert(self, e: int):
        a, b = self._inputs.expert(e)
        return self._read(a), self._read(b)

    def shared(self):
        sh = self._inputs.shared()
        return None if sh is None else (self._read(sh[0]), self._read(sh[1]))
