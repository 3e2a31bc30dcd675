"""Pins of oracle.rope, oracle.block_norm and oracle.fp8 (CPU).

Rotary: against complex multiplication, lengths kept, the inverse undoes it, scores depend on
position differences only.  Norms: the forward against scalar loops, the backward against
central differences in every argument.  8-bit: the grid against torch's own conversion of
every fp16 value, the quantiser's error bound, the product against scalar loops.
"""

import numpy as np
import pytest
import torch

from oracle import block_norm as ON
from oracle import fp8 as O8
from oracle import rope as OR


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_is_complex_multiplication(adjacent):
    rng = np.random.default_rng(1)
    axis, freq = OR.tables([3, 2, 4], per_axis=True)
    x, p = rng.standard_normal((2, 3, 5, 22)), rng.integers(-50, 50, (3, 2, 5))
    got = OR.apply(x, p, axis, freq, adjacent)
    u, v = (x[..., 0:18:2], x[..., 1:18:2]) if adjacent else (x[..., :9], x[..., 9:18])
    z = (u + 1j * v) * np.exp(1j * p[axis].transpose(1, 2, 0) * freq)[:, None]
    gu, gv = (got[..., 0:18:2], got[..., 1:18:2]) if adjacent else (got[..., :9], got[..., 9:18])
    assert np.allclose(gu, z.real, atol=1e-13) and np.allclose(gv, z.imag, atol=1e-13)
    assert np.array_equal(got[..., 18:], x[..., 18:])
    assert np.allclose(OR.apply(got, p, axis, freq, adjacent, inverse=True), x, atol=1e-13)


def test_rope_scores_depend_on_differences():
    rng = np.random.default_rng(2)
    axis, freq = OR.tables([4, 4])
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    score = lambda a, b: (OR.apply(q, a, axis, freq) * OR.apply(k, b, axis, freq)).sum()  # noqa: E731
    a, b, shift = np.array([[3], [9]]), np.array([[1], [4]]), np.array([[100], [-7]])
    assert abs(score(a, b) - score(a + shift, b + shift)) < 1e-12


def test_rope_tables():
    axis, freq = OR.tables([2, 1, 1], base=16.0)
    assert axis.tolist() == [0, 0, 1, 2] and np.allclose(freq, [1, 0.5, 0.25, 0.125])
    axis, freq = OR.tables([3, 1], base=16.0, per_axis=True, interleave=True)
    assert axis.tolist() == [0, 1, 0, 0] and np.allclose(freq, [1, 1, 16 ** (-1 / 3), 16 ** (-2 / 3)])


def _case(post, pre, gate_rows, seed, R=6, C=5):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s)  # noqa: E731
    gate = None if gate_rows == 0 else r(C) if gate_rows == 1 else r(gate_rows, C)
    return dict(x=r(R, C), y=r(R, C), post=post, post_w=r(C) if post else None, post_b=r(C) if post else None,
                gate=gate, alpha=0.7, beta=0.9, pre=pre, pre_w=r(C) if pre else None, pre_b=r(C) if pre else None,
                eps=1e-3), r(R, C), r(R, C)


def test_norm_forward_against_scalar_loops():
    a, _, _ = _case("layer", "rms", 3, 4)
    stream, normed, _ = ON.forward(**a)
    for i in range(6):
        y = a["y"][i]
        m = sum(y) / 5
        r = (sum((v - m) ** 2 for v in y) / 5 + 1e-3) ** -0.5
        row = [0.9 * a["x"][i][c] + 0.7 * a["gate"][i // 2][c] * ((y[c] - m) * r * a["post_w"][c] + a["post_b"][c])
               for c in range(5)]
        q = (sum(v * v for v in row) / 5 + 1e-3) ** -0.5
        for c in range(5):
            assert abs(stream[i, c] - row[c]) < 1e-12
            assert abs(normed[i, c] - (row[c] * q * a["pre_w"][c] + a["pre_b"][c])) < 1e-12


@pytest.mark.parametrize("post,pre,gate_rows", [("rms", "rms", 1), ("layer", "layer", 3), (None, "rms", 6),
                                                ("layer", None, 1), ("rms", "layer", 0), (None, None, 2)])
def test_norm_backward_against_differences(post, pre, gate_rows):
    a, ds, dn = _case(post, pre, gate_rows, 7)
    if pre is None:
        dn = None

    def loss(**change):
        stream, normed, _ = ON.forward(**{**a, **change})
        return (ds * stream).sum() + (0 if dn is None else (dn * normed).sum())

    stream, _, s = ON.forward(**a)
    g, mag = ON.backward(ds, dn, stream, a["y"], s, *(a[k] for k in ("post", "post_w", "post_b", "gate", "alpha", "beta",
                                                                     "pre", "pre_w", "pre_b")))
    names = {"x": "x", "y": "y", "post_w": "post_weight", "post_b": "post_bias", "gate": "gate", "pre_w": "pre_weight",
             "pre_b": "pre_bias"}
    h = 1e-5
    for arg, name in names.items():
        if a[arg] is None:
            continue
        for at in np.ndindex(a[arg].shape):
            up, down = a[arg].copy(), a[arg].copy()
            up[at] += h
            down[at] -= h
            diff = (loss(**{arg: up}) - loss(**{arg: down})) / (2 * h)
            assert abs(diff - g[name][at]) < 1e-7 * max(1.0, abs(diff)), (arg, at)  # h^2 and 1e-16 / h
        if name in mag:
            assert (mag[name] >= np.abs(g[name]) - 1e-12).all()


@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_grid_is_torchs(fmt, dtype):
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.float16).float()
    v = v[v.isfinite() & (v.abs() <= O8.TOP[fmt])]
    assert np.array_equal(O8.to_grid(v.numpy(), fmt), v.to(dtype).double().numpy())
    assert O8.to_grid(1e9, fmt) == O8.TOP[fmt] and np.isnan(O8.to_grid(np.nan, fmt))


def test_quantiser_error_and_blocks():
    x = np.random.default_rng(3).standard_normal((130, 257)).astype(np.float32)
    for square in (False, True):
        codes, scale = O8.quantise(x, square=square)
        assert scale.shape == ((2, 3) if square else (130, 3))
        s = O8.spread(scale, 130, 257)
        # half a step of the value, or of the least normal 2^-6
        assert (np.abs(codes * s - x) <= np.maximum(np.abs(x) * (2.0 ** -4 + 1e-6), 2.0 ** -10 * s * 1.01)).all()
    codes, scale = O8.quantise(np.zeros((1, 3), np.float32))
    assert (codes == 0).all() and np.isfinite(scale).all()


def test_product_against_scalar_loops():
    rng = np.random.default_rng(5)
    a, b = rng.standard_normal((3, 150)), rng.standard_normal((2, 150))
    sa, sb, bias = rng.random((3, 2)), rng.random((1, 2)), rng.standard_normal(2)
    out, mag = O8.product(a, sa, b, sb, bias)
    for m in range(3):
        for n in range(2):
            t = [a[m, k] * sa[m, k // 128] * b[n, k] * sb[0, k // 128] for k in range(150)] + [bias[n]]
            assert abs(out[m, n] - sum(t)) < 1e-12 and abs(mag[m, n] - sum(map(abs, t))) < 1e-12
