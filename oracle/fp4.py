"""Rows of 4-bit grouped-head pools (oracle; test only).

A row of n values is n/2 bytes of E2M1 codes (value 2i in the low half of byte i), then n/16
E4M3 block scales, then padding up to a multiple of 16 bytes. With the pool's scale c, a block's
scale is E4M3(max |x| / (6 c)), a code the E2M1 value nearest to x / (c block), ties to an even
code, magnitudes above 6 saturating; products and quotients in IEEE float32, the arithmetic the
library documents. A block with an infinity or NaN has the scale NaN and codes 0. Encoding compares
against every code, which is slow and plainly correct.
"""

from __future__ import annotations

import numpy as np

from . import fp8 as _fp8
from . import kv_write as _kw

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def row_bytes(n: int) -> int:
    return -(-(n // 2 + n // 16) // 16) * 16


def encode_e2m1(x) -> np.ndarray:
    """Codes of float64 values: nearest, ties to even, saturating; the sign of a zero is kept."""
    x = np.asarray(x, dtype=np.float64)
    dist = np.abs(np.minimum(np.abs(x), 6.0)[..., None] - MAGNITUDES)
    cand = dist == dist.min(-1, keepdims=True)
    even = cand & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1), even.argmax(-1), cand.argmax(-1)).astype(np.uint8)
    return pick | (np.signbit(x).astype(np.uint8) << 3)


def quantize_rows(bits, scale: float) -> np.ndarray:
    """BF16 bit patterns (uint16) ``[..., n]`` -> rows ``[..., row_bytes(n)]``."""
    x = _fp8.decode_bf16(bits).astype(np.float32)
    n = x.shape[-1]
    x = x.reshape(*x.shape[:-1], n // 16, 16)
    odd = ~np.isfinite(x).all(-1)
    x = np.where(odd[..., None], np.float32(0), x)
    with np.errstate(over="ignore"):  # infinity saturates
        most = np.abs(x).max(-1) / (np.float32(6.0) * np.float32(scale))
    block = _kw.encode_e4m3(most.astype(np.float64))
    step = np.float32(scale) * _fp8.decode_e4m3(block).astype(np.float32)
    y = np.divide(x, step[..., None], out=np.zeros_like(x), where=step[..., None] > 0)
    code = np.where(step[..., None] > 0, encode_e2m1(y.astype(np.float64)), 0).astype(np.uint8)
    code = code.reshape(*code.shape[:-2], n)
    out = np.zeros((*code.shape[:-1], row_bytes(n)), dtype=np.uint8)
    out[..., : n // 2] = code[..., 0::2] | (code[..., 1::2] << 4)
    out[..., n // 2: n // 2 + n // 16] = np.where(odd, 0x7F, block)
    return out


def decode_rows(rows, n: int) -> np.ndarray:
    """float64 block scale * code of rows ``[..., row_bytes]`` (without the pool's scale)."""
    rows = np.asarray(rows, dtype=np.uint8)
    code = np.empty((*rows.shape[:-1], n), dtype=np.int64)
    code[..., 0::2] = rows[..., : n // 2] & 15
    code[..., 1::2] = rows[..., : n // 2] >> 4
    value = MAGNITUDES[code & 7] * np.where(code & 8, -1.0, 1.0)
    return value * np.repeat(_fp8.decode_e4m3(rows[..., n // 2: n // 2 + n // 16]), 16, axis=-1)
