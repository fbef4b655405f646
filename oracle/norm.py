"""Oracle: layer norm and its RMS form, forward and gradients, in fp64.

The pages name no norm; the layer whose shapes the workloads take has an RMS
norm in front of its router and experts.  Readings: biased variance, eps inside
the square root, statistics of each row by itself.
"""

import numpy as np


def forward(x, w, b, eps, rms):
    """(y, mean, rstd) of the rows of x [T, D]; w, b [D] or None."""
    x = np.asarray(x, np.float64)
    mean = np.zeros(x.shape[0]) if rms else x.mean(1)
    v = x - mean[:, None]
    rstd = 1.0 / np.sqrt((v * v).mean(1) + eps)
    y = v * rstd[:, None]
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, mean, rstd


def backward(dy, x, w, mean, rstd, rms):
    """(dx, dw, db) from the statistics as given."""
    dy, x, r = (np.asarray(a, np.float64) for a in (dy, x, rstd))
    r = r[:, None]
    h = (x if rms else x - np.asarray(mean, np.float64)[:, None]) * r
    g = dy if w is None else dy * np.asarray(w, np.float64)
    dx = g - h * (g * h).mean(1, keepdims=True)
    if not rms:
        dx = dx - g.mean(1, keepdims=True)
    return dx * r, (dy * h).sum(0), dy.sum(0)
