"""The float64 statement of the grouped matrix products and of the 8-bit
integer product, on the CPU in numpy, from their definitions:

* forward   c[r] = W_e a[r] for the rows r of expert e's queue
* backward  da[r] = W_e^T dc[r], dW_e = sum over the queue of dc[r] a[r]^T
* quantise  s = max(amax / 127, 2^-126) (1 for a zero row), q = rint(x / s)
* int8      c[r, n] = (sum_k qa qw) sa[r] sw[e, n]

Beside each result stands the sum of the absolute values of its terms, from
which the tests derive how far a float32 accumulation may be off.
"""
from __future__ import annotations

import numpy as np


def queues(offsets):
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]


def matmul(a, w, offsets):
    """(c, sum of |terms|), both [R, N]; rows outside every queue are NaN."""
    a, w = np.asarray(a, np.float64), np.asarray(w, np.float64)
    c = np.full((a.shape[0], w.shape[1]), np.nan)
    t = np.zeros_like(c)
    for e, lo, hi in queues(offsets):
        c[lo:hi] = a[lo:hi] @ w[e].T
        t[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w[e]).T
    return c, t


def matmul_backward(a, w, offsets, dc):
    """((da, its terms), (dw, its terms)); da rows outside every queue are NaN."""
    a, w, dc = (np.asarray(v, np.float64) for v in (a, w, dc))
    da = np.full(a.shape, np.nan)
    dat = np.zeros_like(da)
    dw = np.zeros_like(w)
    dwt = np.zeros_like(w)
    for e, lo, hi in queues(offsets):
        da[lo:hi] = dc[lo:hi] @ w[e]
        dat[lo:hi] = np.abs(dc[lo:hi]) @ np.abs(w[e])
        dw[e] = dc[lo:hi].T @ a[lo:hi]
        dwt[e] = np.abs(dc[lo:hi]).T @ np.abs(a[lo:hi])
    return (da, dat), (dw, dwt)


def quantize_rows_int8(x):
    """(codes int8, scales float32), bit for bit: both quotients are rounded
    to float32 once (a float64 quotient of float32 numbers, rounded to
    float32, is the correctly rounded float32 quotient)."""
    x = np.asarray(x, np.float32)
    fine = np.all(np.isfinite(x), axis=1)
    safe = np.where(fine[:, None], x, np.float32(0))
    amax = np.max(np.abs(safe), axis=1).astype(np.float64)
    s = np.maximum((amax / 127.0).astype(np.float32), np.float32(2.0 ** -126))
    s = np.where(amax == 0, np.float32(1), s)
    q = np.rint((safe.astype(np.float64) / s.astype(np.float64)[:, None]).astype(np.float32)).astype(np.int8)
    return q, np.where(fine, s, np.float32(np.nan))


def matmul_int8(qa, sa, qw, sw, offsets):
    """c [R, N] in float64 from the exact integer sums; rows outside every
    queue are NaN."""
    qa, qw = np.asarray(qa, np.float64), np.asarray(qw, np.float64)
    sa, sw = np.asarray(sa, np.float64), np.asarray(sw, np.float64)
    c = np.full((qa.shape[0], qw.shape[1]), np.nan)
    for e, lo, hi in queues(offsets):
        c[lo:hi] = (qa[lo:hi] @ qw[e].T) * sa[lo:hi, None] * sw[e]
    return c
