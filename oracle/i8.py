"""Rows of 8-bit integers with one scale each, and their product (fp64 numpy
oracle).  Symmetric absmax quantization to [-127, 127], nearest integer with
ties to even."""

import numpy as np


def i8_quantize(x):
    """x [rows, cols] fp64 holding bf16 values -> (codes int8, scale fp32).
    127 |x| / amax of bf16 numbers is exact to 2^-53 in fp64 and never nearer
    to a half-way point than 2^-17 without being one, so rint is the exact
    quotient's."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(axis=1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(x), x, 0.0)).max(axis=1))
    safe = np.where(amax > 0, amax, 1.0)
    q = np.where((amax > 0)[:, None], np.rint(127.0 * np.where(bad[:, None], 0.0, x) / safe[:, None]), 0.0)
    scale = (amax / 127.0).astype(np.float32)
    scale[bad] = np.nan
    return q.astype(np.int8), scale


def i8_matmul(xq, sx, wq, sw):
    """sx sw^T o (xq wq^T)."""
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T   # integers below 2^53: exact
    return acc * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
