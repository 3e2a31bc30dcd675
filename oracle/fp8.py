"""Oracle of the block-scaled 8-bit product and its quantiser (numpy).  TEST INFRASTRUCTURE ONLY.

Quantiser: a block of largest magnitude m (at least 2^-100) has scale fl(m / top) and codes
T(fl(x fl(top / m))), fl rounding to fp32 and T to the 8-bit format, to nearest even.  Every
step is one correctly rounded operation, so codes and scales are compared bit by bit.
Product: sum over K of a sa b sb, in fp64 from the codes' values.
"""

from __future__ import annotations

import numpy as np

TOP = {"e4m3": 448.0, "e5m2": 57344.0}
_SHAPE = {"e4m3": (-6, 3), "e5m2": (-14, 2)}  # least exponent, mantissa bits


def to_grid(v, fmt):
    """The nearest value of the format, ties to even, saturating at its largest; NaN stays."""
    low, bits = _SHAPE[fmt]
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        e = np.maximum(np.frexp(v)[1] - 1, low)
        step = np.ldexp(1.0, e - bits)
        return np.clip(np.rint(v / step) * step, -TOP[fmt], TOP[fmt])


def quantise(x, fmt="e4m3", square=False):
    """(values of the codes [R, C] as fp64, scale fp32) of x [R, C] in blocks of 128 columns of a
    row, or of 128 x 128."""
    x = np.asarray(x, dtype=np.float32)
    R, C = x.shape
    br = 128 if square else 1
    nr, nc = -(-R // br), -(-C // 128)
    codes, scale = np.empty((R, C)), np.empty((nr, nc), np.float32)
    top = np.float32(TOP[fmt])
    with np.errstate(all="ignore"):
        for i in range(nr):
            for j in range(nc):
                at = np.s_[i * br:(i + 1) * br, j * 128:(j + 1) * 128]
                m = np.maximum(np.abs(x[at]).max(), np.float32(2.0 ** -100))  # NaN stays NaN
                scale[i, j] = m / top
                codes[at] = to_grid(x[at] * (top / m), fmt)
    return codes, scale


def spread(scale, rows, cols):
    """A scale for every element."""
    br = 1 if scale.shape[0] == rows else 128
    return np.repeat(np.repeat(np.asarray(scale, np.float64), br, 0)[:rows], 128, 1)[:, :cols]


def product(a, sa, b, sb, bias=None):
    """(a sa) (b sb)^T + bias and the sums of its terms' magnitudes; a, b: the codes' values."""
    a = np.asarray(a, np.float64) * spread(sa, *a.shape)
    b = np.asarray(b, np.float64) * spread(sb, *b.shape)
    out, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if bias is not None:
        bias = np.asarray(bias, np.float64)
        out, mag = out + bias, mag + np.abs(bias)
    return out, mag
