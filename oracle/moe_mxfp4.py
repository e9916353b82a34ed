"""The statement of 4-bit microscaled floats (OCP MX: MXFP4) and of their
product by expert, on the CPU in numpy, from the format's definition: a value is
(-1)^sign * magnitude * 2^(scale byte - 127), blocks of 32 values share the
scale byte, 255 stands for NaN.
"""
from __future__ import annotations

import numpy as np

from . import moe_grouped

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def pack(nibbles):
    """[rows, cols] 4-bit codes, two to a byte, the even column in the low half."""
    n = np.asarray(nibbles, np.uint8)
    return (n[:, 0::2] | (n[:, 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    c = np.asarray(codes, np.uint8)
    out = np.empty((c.shape[0], 2 * c.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = c & 15, c >> 4
    return out


def slices(scales):
    """[rows, cols / 32] scale bytes -> [ceil(cols / 256), rows, 8], 127 past the row."""
    rows, blocks = scales.shape
    s = np.full((rows, -(-blocks // 8) * 8), 127, np.uint8)
    s[:, :blocks] = scales
    return np.ascontiguousarray(s.reshape(rows, -1, 8).transpose(1, 0, 2))


def rows_of(scales, blocks):
    """The other way: [S, rows, 8] -> [rows, blocks]."""
    s = np.asarray(scales, np.uint8).transpose(1, 0, 2)
    return s.reshape(s.shape[0], -1)[:, :blocks]


def quantize_rows(x):
    """(codes [rows, cols / 2], scales [S, rows, 8]) of float32 x, bit for bit.
    Nearest magnitude by comparing distances; ties to the even index."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    b = x.reshape(rows, cols // BLOCK, BLOCK)
    fine = np.all(np.isfinite(b), axis=2)
    safe = np.where(fine[:, :, None], b, np.float32(0)).astype(np.float64)
    amax = np.max(np.abs(safe), axis=2)
    # frexp: amax = m 2^e with 0.5 <= m < 1, so floor(log2 amax) = e - 1
    exponent = np.maximum(np.frexp(amax)[1] - 1 - 2, -127)
    exponent = np.where(amax == 0, 0, exponent)
    q = np.abs(safe) * np.exp2(-exponent.astype(np.float64))[:, :, None]
    q = np.minimum(q, MAGNITUDES[-1])
    index = np.zeros(q.shape, np.int64)
    best = np.full(q.shape, np.inf)
    for i in (0, 2, 4, 6, 1, 3, 5, 7):     # (even ones first: they keep a tie)
        d = np.abs(q - MAGNITUDES[i])
        index = np.where(d < best, i, index)
        best = np.minimum(best, d)
    nib = index + 8 * np.signbit(np.where(fine[:, :, None], b, np.float32(0)))
    scales = np.where(fine, exponent + 127, 255).astype(np.uint8)
    return pack(nib.reshape(rows, cols)), slices(scales)


def dequantize_rows(codes, scales):
    """float64 values [rows, cols]."""
    nib = unpack(codes)
    v = MAGNITUDES[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    blocks = nib.shape[1] // BLOCK
    byte = rows_of(scales, blocks).astype(np.int64)
    scale = np.where(byte == 255, np.nan, np.exp2((byte - 127).astype(np.float64)))
    return v * np.repeat(scale, BLOCK, axis=1)


def matmul(a, a_scales, w, w_scales, offsets):
    """(c, sum of |terms|) of moe_grouped.matmul over the dequantised operands;
    w [E, N, K / 2], w_scales [S, E, N, 8]."""
    av = dequantize_rows(a, a_scales)
    wv = np.stack([dequantize_rows(w[e], w_scales[:, e]) for e in range(w.shape[0])])
    return moe_grouped.matmul(av, wv, offsets)
