"""The operators around the update in fp64 NumPy, written from their formulas.

Layer norm and RMS norm with their gradients.  Inputs are taken as the values
they hold (16-bit inputs converted exactly); nothing is rounded.
"""
from __future__ import annotations

import numpy as np


def layer_norm(x, weight=None, bias=None, eps=1e-5, rms=False):
    """(y, mean, rstd) of the rows of x; mean is zeros for the RMS norm."""
    x = np.asarray(x, dtype=np.float64)
    mean = np.zeros(x.shape[0]) if rms else x.sum(1) / x.shape[1]
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(1) / x.shape[1] + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, rms=False):
    """(dx, dweight, dbias) from the formulas, with the statistics as given."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    rstd = np.asarray(rstd, dtype=np.float64)[:, None]
    xh = (x if rms else x - np.asarray(mean, dtype=np.float64)[:, None]) * rstd
    g = dy if weight is None else dy * np.asarray(weight, dtype=np.float64)
    n = x.shape[1]
    dx = g - xh * ((g * xh).sum(1, keepdims=True) / n)
    if not rms:
        dx = dx - g.sum(1, keepdims=True) / n
    return rstd * dx, (dy * xh).sum(0), dy.sum(0)


QUINTIC = (3.4445, -4.7750, 2.0315)


def orthogonalize(x, steps=5, coeffs=QUINTIC, eps=1e-7):
    """The Newton-Schulz output of each matrix of the stack x [batch, rows, cols]."""
    a, b, c = coeffs
    x = np.asarray(x, dtype=np.float64)
    tall = x.shape[1] > x.shape[2]
    y = x.transpose(0, 2, 1) if tall else x
    y = y / (np.sqrt((y * y).sum((1, 2), keepdims=True)) + eps)
    for _ in range(steps):
        gram = y @ y.transpose(0, 2, 1)
        y = a * y + (b * gram + c * (gram @ gram)) @ y
    return y.transpose(0, 2, 1) if tall else y


def e4m3(x):
    """x rounded to e4m3 (ties to even), as fp64: three bits behind the leading one, steps of 2^-9 below 2^-6."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(np.maximum(np.abs(x), 2.0 ** -6))      # |x| in [2^(e-1), 2^e)
    step = np.ldexp(1.0, e - 4)
    return np.rint(x / step) * step


def block_exponents(x, block_rows):
    """The exponent of each block_rows x 128 block of x: the smallest k >= -127 with max|x| <= 448 2^k, 0 for zeros."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    rows, cols = -(-x.shape[0] // block_rows), -(-x.shape[1] // 128)
    k = np.zeros((rows, cols), dtype=np.int64)
    for i in range(rows):
        for j in range(cols):
            m = x[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128].max()
            if m > 0:
                f, e = np.frexp(m)                         # m = f 2^e, 448 = 0.875 2^9
                k[i, j] = max(-127, e - 9 if f <= 0.875 else e - 8)
    return k


def spread(k, block_rows, rows, cols):
    """Each block's entry at every element of it."""
    return np.repeat(np.repeat(k, block_rows, 0)[:rows], 128, 1)[:, :cols]


def block_quantize(x, block_rows):
    """(values of the e4m3 matrix, scale bytes) of x."""
    x = np.asarray(x, dtype=np.float64)
    k = block_exponents(x, block_rows)
    return e4m3(np.ldexp(x, -spread(k, block_rows, *x.shape))), (k + 127).astype(np.uint8)


def block_values(q, scale):
    """What a quantised matrix stands for, fp64; its scales are for each row or each 128 rows."""
    q = np.asarray(q, dtype=np.float64)
    rows = 1 if scale.shape[0] == q.shape[0] else 128
    return np.ldexp(q, spread(scale.astype(np.int64) - 127, rows, *q.shape))
