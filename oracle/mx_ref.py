"""Float64 oracle of microscaled 4-bit floating point (numpy, from the
formulas).

A code is a sign bit over three bits m: 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Blocks of
32 share a power of two (byte e: 2^(e - 127), 255 NaN), blocks of 16 a byte of 4
exponent bits (bias 7) and 3 mantissa bits (0x7f NaN) under a float32 scale of
the tensor, whose float32 reciprocal the values are multiplied by first.  Rows
[R, K]: codes [R, K/2], column 2i low; scales [R, 4 ceil(K/block/4)].
"""
from __future__ import annotations

import numpy as np

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
MIDDLES = (VALUES[1:] + VALUES[:-1]) / 2


def scale_row(K, block):
    return -(-(K // block) // 4) * 4


def small_float(byte):
    """The value of a 4-exponent, 3-mantissa byte (without a sign)."""
    e, m = byte >> 3, byte & 7
    if byte & 127 == 127:
        return np.nan
    return m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)


SMALL = np.array([small_float(b) for b in range(127)])


def nearest_small(v):
    """The byte of the value nearest to v >= 0, ties to the even byte."""
    hi = int(np.clip(np.searchsorted(SMALL, v), 1, 126))
    lo = hi - 1
    a, b = v - SMALL[lo], SMALL[hi] - v
    return lo if a < b or (a == b and lo % 2 == 0) else hi


def block_scales(v, block):
    """(bytes, values) of the blocks v [..., block] of float64 numbers."""
    with np.errstate(invalid="ignore"):
        most = np.abs(v).max(-1)
    byte = np.empty(most.shape, dtype=np.uint8)
    for i in np.ndindex(most.shape):
        m = most[i]
        if not np.isfinite(m):
            byte[i] = 255 if block == 32 else 127
        elif block == 32:
            e = int(np.frexp(m)[1]) - 1 if m > 0 else -200
            byte[i] = max(e - 2, -127) + 127
        else:
            byte[i] = nearest_small(m / 6)
    return byte, scale_values(byte, block)


def scale_values(byte, block):
    b = byte.astype(np.int64)
    if block == 32:
        return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    return np.append(SMALL, np.nan)[b & 127]


def prescaled(x, block, scale):
    if block == 32:
        return np.asarray(x, dtype=np.float64)
    r = np.float32(1) / np.float32(scale)
    with np.errstate(over="ignore", invalid="ignore"):
        return (np.asarray(x, np.float32) * r).astype(np.float64)


def quantize_rows(x, block, scale=1.0):
    """Codes and scales of x [R, K] (values of float32 or bf16)."""
    R, K = x.shape
    v = prescaled(x, block, scale).reshape(R, -1, block)
    byte, s = block_scales(v, block)
    mag = np.zeros(v.shape, dtype=np.int64)
    with np.errstate(invalid="ignore"):
        for i, m in enumerate(MIDDLES):
            edge = m * s[..., None]
            # the middle itself goes to the even code
            over = np.abs(v) > edge if i % 2 == 0 else np.abs(v) >= edge
            mag += over & (s[..., None] > 0)
    code = (mag + 8 * np.signbit(v)).reshape(R, K)
    scales = np.zeros((R, scale_row(K, block)), dtype=np.uint8)
    scales[:, :K // block] = byte
    return (code[:, 0::2] + 16 * code[:, 1::2]).astype(np.uint8), scales


def code_values(codes):
    """float64 [R, K] of codes [R, K/2]."""
    q = np.stack([codes % 16, codes // 16], -1).reshape(codes.shape[0], -1)
    q = q.astype(np.int64)
    return VALUES[q % 8] * np.where(q >= 8, -1.0, 1.0)


def dequantize_rows(codes, scales, block, scale=1.0):
    v = code_values(codes)
    s = scale_values(scales[:, :v.shape[1] // block], block)
    return v * np.repeat(s, block, 1) * np.float64(np.float32(scale))


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))
