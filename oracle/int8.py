"""Oracle: 8-bit integers with one fp32 scale per row (W8A8), and their grouped
products.

Readings (the pages name no such format): per row with amax a, in IEEE fp32,
s = a / 127 and q = x / s rounded to nearest even, clamped to [-127, 127]; 0
where s is 0.  A row with an infinity or a NaN gets that as its scale, and zeros.
The product's sum is exact; it is rounded to fp32, multiplied by the row's scale,
then by the channel's, each in fp32.
"""

import numpy as np


def quantize(x):
    """(q int8 [rows, K], s fp32 [rows]) of fp32 values."""
    x = np.ascontiguousarray(x, np.float32)
    rows, K = x.shape
    with np.errstate(all="ignore"):
        a = np.abs(x).max(1) if K else np.zeros(rows, np.float32)  # (a NaN stays one)
        s = (a / np.float32(127)).astype(np.float32)
        live = np.isfinite(a) & (s > 0)
        r = np.rint(x / np.where(live, s, np.float32(1))[:, None])
        q = np.where(live[:, None], np.clip(r, -127, 127), 0)
    return q.astype(np.int8), s


def grouped_gemm(aq, a_s, bq, b_s, offsets):
    """C [M, N] in fp32 as defined; rows at and past offsets[E] are zeros."""
    M, N = aq.shape[0], bq.shape[1]
    c = np.zeros((M, N), np.float32)
    with np.errstate(all="ignore"):
        for e in range(bq.shape[0]):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            if hi > lo:
                # whole numbers below 2^31: exact in fp64
                n = aq[lo:hi].astype(np.float64) @ bq[e].astype(np.float64).T
                c[lo:hi] = n.astype(np.float32) * a_s[lo:hi, None] * b_s[e][None, :]
    return c
