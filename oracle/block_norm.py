"""Oracle of a block's norms, gate and residual in fp64 (numpy).  TEST INFRASTRUCTURE ONLY.

    stream = beta x + alpha g (N_post(y) w_post + b_post),  normed = N_pre(stream) w_pre + b_pre

over rows [R, C]; N is "rms" (x / sqrt(mean x^2 + eps)), "layer" (the same of x - mean x) or
None.  g is [C] or has a row for every `R / len(g)` rows.  The gradients are written row by row
from the Jacobian of N: for n = (x - m) r, r = (mean (x - m)^2 + eps)^(-1/2),
dx = r (dn - mean(dn) [layer] - n mean(dn n)).
"""

from __future__ import annotations

import numpy as np


def stats(x, kind, eps):
    """(mean, 1 / sqrt(..)) of each row, [R, 1] each."""
    m = x.mean(1, keepdims=True) if kind == "layer" else np.zeros((len(x), 1))
    return m, 1.0 / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + eps)


def _full(v, shape, default):
    """A parameter [C], or a gate of one row for several, over all rows."""
    if v is None:
        return np.full(shape, default)
    v = np.atleast_2d(np.asarray(v, dtype=np.float64))
    return np.repeat(v, shape[0] // len(v), 0) if len(v) else np.zeros(shape)


def forward(x, y, post, post_w, post_b, gate, alpha, beta, pre, pre_w, pre_b, eps):
    """(stream, normed, stats [R, 4]); normed is None without a pre norm."""
    s = np.zeros((len(x), 4))
    stream = x
    if y is not None:
        n = y
        if post is not None:
            m, r = stats(y, post, eps)
            s[:, 0:1], s[:, 1:2] = m, r
            n = (y - m) * r
        z = n * _full(post_w, y.shape, 1.0) + _full(post_b, y.shape, 0.0)
        stream = beta * x + alpha * _full(gate, y.shape, 1.0) * z
    normed = None
    if pre is not None:
        m, r = stats(stream, pre, eps)
        s[:, 2:3], s[:, 3:4] = m, r
        normed = (stream - m) * r * _full(pre_w, x.shape, 1.0) + _full(pre_b, x.shape, 0.0)
    return stream, normed, s


def _back(n, r, dn, kind):
    d = dn - n * (dn * n).mean(1, keepdims=True)
    return r * (d - dn.mean(1, keepdims=True) if kind == "layer" else d)


def backward(dstream, dnormed, stream, y, s, post, post_w, post_b, gate, alpha, beta, pre, pre_w, pre_b):
    """Gradients by x, y, post_weight, post_bias, gate, pre_weight, pre_bias, and for those summed
    over rows the sums of their terms' magnitudes (the scale of their rounding error)."""
    shape = stream.shape
    D = np.zeros(shape) if dstream is None else dstream.copy()
    g, mag = {}, {}
    if pre is not None:
        dh = np.zeros(shape) if dnormed is None else dnormed
        n = (stream - s[:, 2:3]) * s[:, 3:4]
        g["pre_weight"], mag["pre_weight"] = (dh * n).sum(0), np.abs(dh * n).sum(0)
        g["pre_bias"], mag["pre_bias"] = dh.sum(0), np.abs(dh).sum(0)
        D = D + _back(n, s[:, 3:4], dh * _full(pre_w, shape, 1.0), pre)
    g["x"] = (beta if y is not None else 1.0) * D
    if y is None:
        return g, mag
    n = (y - s[:, 0:1]) * s[:, 1:2] if post is not None else y
    full = _full(gate, shape, 1.0)
    z = n * _full(post_w, shape, 1.0) + _full(post_b, shape, 0.0)
    if gate is not None:
        rows = len(np.atleast_2d(gate))
        t = (alpha * D * z).reshape(rows, -1, shape[1])
        g["gate"], mag["gate"] = t.sum(1).reshape(np.shape(gate)), np.abs(t).sum(1).reshape(np.shape(gate))
    dz = alpha * full * D
    g["post_weight"], mag["post_weight"] = (dz * n).sum(0), np.abs(dz * n).sum(0)
    g["post_bias"], mag["post_bias"] = dz.sum(0), np.abs(dz).sum(0)
    g["y"] = _back(n, s[:, 1:2], dz * _full(post_w, shape, 1.0), post) if post is not None else dz
    return g, mag
