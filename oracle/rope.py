"""Oracle of rotary positions with several axes in fp64 (numpy).  TEST INFRASTRUCTURE ONLY.

Definition: pair j of a head turns by the angle p[axis_j] * freq_j of its token,
(u, v) -> (u cos t - v sin t, u sin t + v cos t); its columns are j and n + j of n pairs, or
2 j and 2 j + 1; columns past 2 n stay.  Its gradient is the turn by -t.
"""

from __future__ import annotations

import numpy as np


def tables(sections, base=10000.0, per_axis=False, interleave=False):
    """(axis, freq) of each pair, pair by pair from the rule's words."""
    left = list(sections)
    n = sum(left)
    axis, freq, turn = [], [], 0
    for j in range(n):
        if interleave:
            while left[turn % len(left)] == 0:
                turn += 1
            a = turn % len(left)
            turn += 1
        else:
            a = next(i for i, s in enumerate(left) if s > 0)
        i = sections[a] - left[a]
        left[a] -= 1
        axis.append(a)
        freq.append(base ** (-i / sections[a]) if per_axis else base ** (-j / n))
    return np.array(axis), np.array(freq)


def apply(x, positions, axis, freq, adjacent=False, inverse=False):
    """x [B, H, L, d] turned; positions [axes, B, L] or [axes, L]."""
    x = np.array(x, dtype=np.float64)
    p = np.asarray(positions, dtype=np.float64)
    if p.ndim == 2:
        p = np.repeat(p[:, None], x.shape[0], 1)
    n = len(axis)
    out = x.copy()
    for j in range(n):
        t = p[axis[j]] * freq[j]
        if inverse:
            t = -t
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        a, b = (2 * j, 2 * j + 1) if adjacent else (j, n + j)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
    return out


def magnitude(x, n, adjacent=False):
    """|u| + |v| of each element's pair (|x| past them): the scale of its rounding error."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    out = x.copy()
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
    out[..., a] = out[..., b] = x[..., a] + x[..., b]
    return out
