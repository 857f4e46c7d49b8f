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
