"""Float64 oracle of the 4-bit expert weights (numpy, from the formulas).

    w[k, n] = (code[k, n] - zero[k // group, n]) * scale[k // group, n]

codes [n, K/2, N] uint8 hold row 2i in the low and row 2i+1 in the high four
bits; scales are given as float64 (bf16 values), zeros as uint8 or None (8).
"""
from __future__ import annotations

import numpy as np


def unpack(codes):
    """uint8 [n, K/2, N] -> int64 codes [n, K, N]."""
    n, half, N = codes.shape
    out = np.empty((n, 2 * half, N), dtype=np.int64)
    out[:, 0::2], out[:, 1::2] = codes % 16, codes // 16
    return out


def dequantize(codes, scales, zeros, group):
    q = unpack(codes).astype(np.float64)
    for g in range(scales.shape[1]):
        rows = q[:, g * group:(g + 1) * group]
        rows -= 8.0 if zeros is None else zeros[:, g:g + 1]
        rows *= scales[:, g:g + 1]
    return q


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def swiglu(x, offsets, experts, wg, wu, wd):
    """(h, y) of the sorted rows; group i
    holds rows offsets[i]..offsets[i+1] and uses expert experts[i]."""
    R = offsets[-1]
    h = np.zeros((R, wg.shape[2]))
    y = np.zeros((R, wd.shape[2]))
    for i, e in enumerate(experts):
        a, z = offsets[i], offsets[i + 1]
        if z > a:
            h[a:z] = silu(x[a:z] @ wg[e]) * (x[a:z] @ wu[e])
            y[a:z] = h[a:z] @ wd[e]
    return h, y
