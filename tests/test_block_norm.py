"""The norms before and after a block with its gate and residual (bsa_block_norm and backward).

CPU: refusals of the C ABI before any device work, the workspace's size.
GPU: both directions against the fp64 oracle over norms, gates, types, parameter types, one row
to many, odd columns, rows without alignment; in place; zero rows; two captured graphs; the
autograd form, whole and in parts.

Tolerance (from the arithmetic), with u the half step of the type (2^-8 bf16, 2^-11 fp16, 2^-24
fp32) and v = 2^-24 that of fp32.  A row's sum of C terms is added by threads of at most 24
terms and then over at most 5 + 4 steps of pairs, so it errs by less than 40 v of the sum of
magnitudes; hence 1/sqrt(..) by 25 v relative and the mean by 40 v mean|x|, and a normalised
value n by 64 v (|n| + mean|x| r).  Each further product or sum adds v of its operands.  So an
output errs by u |ref| plus 2^-17 = 128 v of the magnitudes of what it is a sum of.  Sums over R
rows add at most (R + 64) v of the sum of their terms' magnitudes (a thread adds its rows one
after the other), and the terms' own 2^-17.
"""

import ctypes

import numpy as np
import pytest
import torch

from block_sparse_attention_bigbird_b200 import bsa
from oracle import block_norm as ON

gpu = pytest.mark.gpu
needs_cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
EPS = 1e-5


# ---------------------------------------------------------------- CPU
def _args(**kw):
    a = dict(B=2, rows_per_batch=3, C=64, type=bsa.BF16, param_type=bsa.FP32, post=1, pre=1, post_weight=1 << 20,
             post_bias=None, gate=1 << 20, pre_weight=1 << 20, pre_bias=None, gate_rows=1, branch_scale=1.0,
             stream_scale=1.0, eps=1e-5)
    a.update(kw)
    return bsa.BlockNormArgs(*[a[n] for n, _ in bsa.BlockNormArgs._fields_])


def test_forward_refuses_before_device_work():
    f, p = bsa.lib.bsa_block_norm, 1 << 20
    call = lambda x=p, y=p, out=p, normed=2 * p, stats=None, **kw: f(  # noqa: E731
        ctypes.byref(_args(**kw)), x, y, out, normed, stats, None)
    assert f(None, p, p, p, p, None, None) == bsa.BSA_ERR_INVALID_ARG
    for kw in (dict(B=-1), dict(rows_per_batch=-1), dict(C=0), dict(post=3), dict(pre=-1), dict(gate_rows=3),
               dict(eps=-1.0), dict(eps=float("nan")), dict(branch_scale=float("nan")), dict(post=0), dict(pre=0),
               dict(x=None), dict(out=None), dict(normed=None), dict(y=None), dict(x=p + 1), dict(stats=p + 4),
               dict(gate=p + 2), dict(normed=p), dict(y=None, post=0, post_weight=None, gate=None, pre=0, pre_weight=None)):
        assert call(**kw) == bsa.BSA_ERR_INVALID_ARG, kw
    for kw in (dict(C=8193), dict(type=bsa.E4M3), dict(type=bsa.BF16, param_type=bsa.FP16)):
        assert call(**kw) == bsa.BSA_ERR_UNSUPPORTED, kw
    assert call(B=0) == bsa.BSA_OK  # no rows


def test_backward_refuses_before_device_work():
    f, p = bsa.lib.bsa_block_norm_backward, 1 << 20
    order = ("dstream", "dnormed", "x", "y", "stats", "dx", "dy", "dpw", "dpb", "dg", "dw", "db", "ws")

    def call(**kw):
        a = {n: p for n in order} | {"dy": 2 * p, "dpb": None, "db": None}
        a.update({k: v for k, v in kw.items() if k in order})
        return f(ctypes.byref(_args(**{k: v for k, v in kw.items() if k not in order})), *[a[n] for n in order], 1 << 30, None)
    for kw in (dict(x=None), dict(dx=None), dict(stats=None), dict(dy=None), dict(y=None), dict(dpb=p), dict(db=p),
               dict(gate=None), dict(pre=0, pre_weight=None), dict(x=p + 1), dict(dg=p + 1), dict(dy=p)):
        assert call(**kw) == bsa.BSA_ERR_INVALID_ARG, kw


# ---------------------------------------------------------------- GPU
def _make(B, L, C, post, pre, gate, bias, ty, pt, seed, y=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, t=ty, scale=1.0, shift=0.0: (torch.randn(*s, generator=g, device="cuda") * scale + shift).to(t)  # noqa: E731
    a = dict(post=post, pre=pre, branch_scale=0.75, stream_scale=0.875) if y else dict(post=None, pre=pre)
    for n, k in (("post", post), ("pre", pre)):
        a[n + "_weight"] = r(C, t=pt, scale=0.3, shift=1.0) if k else None
        a[n + "_bias"] = r(C, t=pt, scale=0.3) if k and bias else None
    a["gate"] = {0: None, 1: lambda: r(C, t=pt, scale=0.5, shift=0.5), 2: lambda: r(B, C, t=pt, scale=0.5, shift=0.5)}[gate]
    a["gate"] = a["gate"]() if a["gate"] else None
    x, yy = r(B, L, C, scale=2.0, shift=0.3), r(B, L, C, scale=0.7, shift=-0.2) if y else None
    return a, x, yy, r(B, L, C), r(B, L, C) if pre else None


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy().reshape(-1, t.shape[-1])


def _oracle(a):
    one = lambda t: None if t is None else t.detach().double().cpu().numpy()  # noqa: E731
    return (a["post"], one(a["post_weight"]), one(a["post_bias"]), one(a["gate"]), a.get("branch_scale", 1.0),
            a.get("stream_scale", 1.0), a["pre"], one(a["pre_weight"]), one(a["pre_bias"]))


def _near(got, ref, mag, u, name):
    got = got.detach().double().cpu().numpy().reshape(ref.shape)
    bad = np.abs(got - ref) > u * (np.abs(ref) + mag) + mag + 2.0 ** -24 * (u == 2.0 ** -11)
    assert not bad.any(), (name, int(bad.sum()), np.abs(got - ref).max())


def _mag(x, kind, w, b):
    """Magnitude of a normalised row's outputs: (|n| + mean|x| r) |w| + |b|."""
    m, r = ON.stats(x, kind, EPS)
    n = np.abs((x - m) * r) + np.abs(x).mean(1, keepdims=True) * r
    return n * (1.0 if w is None else np.abs(w)) + (0.0 if b is None else np.abs(b))


def _check(a, x, y, ds, dn):
    ty = x.dtype
    X, Y = _np(x), _np(y)
    o = _oracle(a)
    post, pw, pb, gate, alpha, beta, pre, w, b = o
    stream, normed, stats = bsa.bsa_block_norm(x, y, eps=EPS, save_stats=True, **a)
    ref_s, ref_n, ref_st = ON.forward(X, Y, *o, EPS)
    full = ON._full(None if gate is None else np.abs(gate), X.shape, 1.0)
    smag = np.abs(X) * abs(beta)
    if y is not None:
        smag = smag + abs(alpha) * full * (_mag(Y, post, pw, pb) if post else np.abs(Y))
        _near(stream, ref_s, 2.0 ** -17 * smag, U[ty], "stream")
    else:
        assert stream is x
    if pre:
        _, r = ON.stats(ref_s, pre, EPS)
        mag = _mag(ref_s, pre, w, b) + smag * r * (1.0 if w is None else np.abs(w))
        mag = mag + np.abs(smag).mean(1, keepdims=True) * r * (1.0 if w is None else np.abs(w))
        _near(normed, ref_n, 2.0 ** -17 * mag, U[ty], "normed")
    else:
        assert normed is None
    # the backward starts from what the forward left: its stream and statistics
    S, st = _np(stream), stats.double().cpu().numpy()
    g = bsa.bsa_block_norm_backward(ds, dn, stream, y, stats, **a)
    ref, mags = ON.backward(_np(ds), _np(dn), S, Y, st, *o)
    R = len(S)
    # magnitudes of D: each of its terms' absolute values, row means among them
    dmag = np.zeros(S.shape) if ds is None else np.abs(_np(ds))
    if pre:
        n = np.abs(S - st[:, 2:3]) * st[:, 3:4]
        if dn is not None:
            t = np.abs(_np(dn)) * (1.0 if w is None else np.abs(w))
            dmag = dmag + st[:, 3:4] * (t + t.mean(1, keepdims=True) + n * (t * n).mean(1, keepdims=True))
    _near(g["x"], ref["x"], 2.0 ** -17 * dmag * abs(beta), U[ty], "dx")
    if y is not None:
        ym = (np.abs(Y - st[:, 0:1]) * st[:, 1:2]) if post else np.abs(Y)
        t = abs(alpha) * full * dmag * (1.0 if pw is None else np.abs(pw))
        mag = st[:, 1:2] * (t + t.mean(1, keepdims=True) + ym * (t * ym).mean(1, keepdims=True)) if post else t
        _near(g["y"], ref["y"], 2.0 ** -17 * mag, U[ty], "dy")
        z = ym * (1.0 if pw is None else np.abs(pw)) + (0.0 if pb is None else np.abs(pb))
        terms = {"gate": abs(alpha) * dmag * z, "post_weight": abs(alpha) * full * dmag * ym,
                 "post_bias": abs(alpha) * full * dmag}
    else:
        terms = {}
    if pre and dn is not None:
        terms |= {"pre_weight": np.abs(_np(dn)) * n, "pre_bias": np.abs(_np(dn))}
    for name in ("post_weight", "post_bias", "gate", "pre_weight", "pre_bias"):
        t = a[name]
        assert (g[name] is None) == (t is None)
        if t is None:
            continue
        if name not in terms:
            assert (g[name] == 0).all()
            continue
        rows = len(t) if t.dim() == 2 else 1
        total = terms[name].reshape(rows, -1, S.shape[1]).sum(1).reshape(t.shape)
        _near(g[name], ref[name].reshape(t.shape), ((R + 64) * 2.0 ** -24 + 2.0 ** -17) * total, U[t.dtype], name)
    return stream, normed, stats, g


CASES = [  # B, L, C, post, pre, gate, bias, type, parameter type
    (1, 1, 64, "rms", "rms", 1, False, torch.bfloat16, torch.bfloat16),
    (8, 1, 768, "rms", "rms", 2, False, torch.bfloat16, torch.float32),
    (2, 77, 768, "layer", "layer", 1, True, torch.bfloat16, torch.float32),
    (3, 50, 512, "layer", "rms", 2, False, torch.float16, torch.float16),
    (2, 33, 768, "rms", "layer", 2, True, torch.float32, torch.float32),
    (1, 700, 256, "rms", "rms", 1, False, torch.bfloat16, torch.bfloat16),
    (2, 9, 1024, "layer", "layer", 2, True, torch.bfloat16, torch.bfloat16),
    (2, 21, 4096, "rms", "rms", 1, False, torch.bfloat16, torch.float32),
    (1, 12, 8192, "layer", "layer", 1, True, torch.float32, torch.float32),
    (5, 7, 8192, "rms", "rms", 2, False, torch.float16, torch.float32),
    (3, 31, 1030, "layer", "layer", 1, True, torch.float32, torch.float32),   # pairs of elements
    (2, 11, 54, "rms", "layer", 2, True, torch.bfloat16, torch.float32),
    (2, 13, 8190, "layer", "rms", 1, False, torch.bfloat16, torch.bfloat16),
    (2, 17, 333, "rms", "rms", 2, True, torch.bfloat16, torch.float32),       # single elements
    (1, 5, 8191, "layer", "layer", 1, True, torch.float16, torch.float16),
    (1, 9, 4097, "rms", "rms", 0, False, torch.float32, torch.float32),
    (4, 3, 1, "rms", "rms", 1, True, torch.float32, torch.float32),
    (40, 3, 96, "rms", "rms", 2, True, torch.bfloat16, torch.float32),        # more gate rows than 32
    (16, 40, 128, "layer", None, 2, False, torch.bfloat16, torch.float32),
    (2, 19, 320, None, "rms", 1, False, torch.bfloat16, torch.float32),
    (2, 19, 320, None, None, 2, False, torch.bfloat16, torch.bfloat16),
    (3, 600, 768, "rms", "rms", 0, False, torch.bfloat16, torch.float32),
    (3, 2866, 59, "rms", "rms", 1, False, torch.bfloat16, torch.float32),     # every team of every block has rows
    (2, 4000, 42, "layer", "layer", 2, True, torch.float32, torch.float32),
    (1, 5000, 48, "rms", "layer", 1, True, torch.bfloat16, torch.bfloat16),
]


@gpu
@needs_cuda
@pytest.mark.parametrize("B,L,C,post,pre,gate,bias,ty,pt", CASES)
def test_matches_oracle(B, L, C, post, pre, gate, bias, ty, pt):
    a, x, y, ds, dn = _make(B, L, C, post, pre, gate, bias, ty, pt, B * L + C)
    first = _check(a, x, y, ds, dn)
    again = bsa.bsa_block_norm(x, y, eps=EPS, save_stats=True, **a)
    assert all(p is None or torch.equal(p, q) for p, q in zip(first[:3], again))
    g = bsa.bsa_block_norm_backward(ds, dn, first[0], y, first[2], **a)
    assert all(v is None or torch.equal(v, first[3][n]) for n, v in g.items())


@gpu
@needs_cuda
@pytest.mark.parametrize("pre,C", [("rms", 768), ("layer", 768), ("layer", 1001), ("rms", 2050)])
def test_norm_alone_and_missing_gradients(pre, C):
    a, x, _, ds, dn = _make(2, 23, C, None, pre, 0, pre == "layer", torch.bfloat16, torch.float32, C, y=False)
    _check(a, x, None, ds, dn)
    _check(a, x, None, None, dn)
    b, x, y, ds, dn = _make(2, 23, C, "rms", pre, 1, True, torch.bfloat16, torch.float32, C + 1)
    _check(b, x, y, None, dn)
    _check(b, x, y, ds, None)
    stream, _, stats = bsa.bsa_block_norm(x, y, eps=EPS, save_stats=True, **b)
    with_, without = (bsa.bsa_block_norm_backward(ds, dn, stream, y, stats, params=p, **b) for p in (True, False))
    assert torch.equal(with_["x"], without["x"]) and torch.equal(with_["y"], without["y"])
    assert all(without[n] is None for n in ("gate", "post_weight", "pre_weight"))


@gpu
@needs_cuda
def test_shapes_alignment_and_in_place():
    a, x, y, ds, dn = _make(3, 10, 256, "rms", "layer", 1, True, torch.bfloat16, torch.float32, 3)
    want = bsa.bsa_block_norm(x, y, **a)
    flat = bsa.bsa_block_norm(x.view(30, 256), y.view(30, 256), **a)
    assert torch.equal(flat[0].view_as(x), want[0]) and torch.equal(flat[1].view_as(x), want[1])
    one = bsa.bsa_block_norm(x[0, 0], y[0, 0], **a)
    assert torch.equal(one[0], want[0][0, 0]) and torch.equal(one[1], want[1][0, 0])
    # rows that do not start at 16 bytes: another kernel, the same numbers up to the order of sums
    store = torch.empty(2, 3 * 10 * 256 + 1, dtype=torch.bfloat16, device="cuda")
    u, v = (store[i, 1:].view(3, 10, 256) for i in range(2))
    u.copy_(x), v.copy_(y)
    got = bsa.bsa_block_norm(u, v, **a)
    for p, q in zip(got[:2], want[:2]):
        assert (p.float() - q.float()).abs().max() <= 2 * 2.0 ** -8 * q.float().abs().max()
    _check(a, u, v, ds, dn)
    xi, yi = x.clone(), y.clone()
    s, n, _ = bsa.bsa_block_norm(xi, yi, out=xi, normed=yi, **a)
    assert s is xi and n is yi and torch.equal(xi, want[0]) and torch.equal(yi, want[1])


@gpu
@needs_cuda
def test_zero_rows():
    a, x, y, ds, dn = _make(2, 0, 64, "layer", "rms", 1, True, torch.bfloat16, torch.float32, 1)
    s, n, st = bsa.bsa_block_norm(x, y, eps=EPS, save_stats=True, **a)
    assert s.shape == n.shape == x.shape and st.shape == (0, 4)
    g = bsa.bsa_block_norm_backward(ds, dn, s, y, st, **a)
    assert all((g[k] == 0).all() for k in ("gate", "post_weight", "post_bias", "pre_weight", "pre_bias"))


@gpu
@needs_cuda
def test_nan_rows_stay_in_their_rows():
    a, x, y, ds, dn = _make(1, 8, 768, "rms", "rms", 1, False, torch.bfloat16, torch.float32, 9)
    want = bsa.bsa_block_norm(x, y, **a)
    x[0, 3, 5], y[0, 6, 700] = float("nan"), float("inf")
    got = bsa.bsa_block_norm(x, y, **a)
    for p, q in zip(got[:2], want[:2]):
        for row in range(8):
            if row in (3, 6):
                assert p[0, row].isnan().any()
            else:
                assert torch.equal(p[0, row], q[0, row])


@gpu
@needs_cuda
def test_binding_refuses():
    a, x, y, ds, dn = _make(2, 5, 64, "rms", "rms", 1, False, torch.bfloat16, torch.float32, 2)
    call = lambda x=x, y=y, **kw: bsa.bsa_block_norm(x, y, **{**a, **kw})  # noqa: E731
    call()
    w = a["pre_weight"]
    for kw in (dict(x=x.double()), dict(x=x.transpose(0, 1)), dict(y=y[:1]), dict(y=y.float()), dict(x=x.cpu()),
               dict(post="batch"), dict(pre_weight=w[:63]), dict(pre_weight=w.half()), dict(pre_weight=w.bfloat16()),
               dict(gate=w.expand(3, 64).contiguous()), dict(gate=w.view(1, 1, 64)), dict(pre=None), dict(post=None),
               dict(pre_weight=w.cpu()), dict(y=None), dict(out=x[:1]), dict(normed=x.float()),
               dict(gate=torch.zeros(2, 128, device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            call(**kw)
    s, n, st = bsa.bsa_block_norm(x, y, save_stats=True, **a)
    for kw in (dict(dstream=ds[:1]), dict(dnormed=dn.float()), dict(stats=st[:4]), dict(stats=st.double())):
        with pytest.raises(ValueError):
            bsa.bsa_block_norm_backward(**{**dict(dstream=ds, dnormed=dn, x=s, y=y, stats=st), **kw}, **a)


@gpu
@needs_cuda
def test_two_graphs_and_streams():
    cases = [_make(2, 40, 768, "rms", "rms", 2, False, torch.bfloat16, torch.float32, i) for i in (1, 2)]
    graphs, got = [], []
    for a, x, y, ds, dn in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s, n, st = bsa.bsa_block_norm(x, y, eps=EPS, save_stats=True, **a)
            got.append((s, n, bsa.bsa_block_norm_backward(ds, dn, s, y, st, **a)))
        graphs.append(graph)
    for _, x, y, _, _ in cases:
        x.mul_(0.5)
        y.add_(1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs[0].replay()
    with torch.cuda.stream(side):
        graphs[1].replay()
    torch.cuda.synchronize()
    for (a, x, y, ds, dn), (s, n, g) in zip(cases, got):
        ws, wn, st = bsa.bsa_block_norm(x, y, eps=EPS, save_stats=True, stream=side, **a)
        wg = bsa.bsa_block_norm_backward(ds, dn, ws, y, st, stream=side, **a)
        side.synchronize()
        assert torch.equal(s, ws) and torch.equal(n, wn)
        assert all(v is None or torch.equal(v, wg[k]) for k, v in g.items())


@gpu
@needs_cuda
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", None), (None, "layer")])
def test_autograd(post, pre):
    from block_sparse_attention_bigbird_b200 import block_norm
    a, x, y, ds, dn = _make(2, 9, 128, post, pre, 2, True, torch.float32, torch.float32, 4)
    leaves = {k: v.clone().requires_grad_() for k, v in {"x": x, "y": y, **a}.items() if torch.is_tensor(v)}
    s, n = block_norm(leaves["x"], leaves["y"], eps=EPS, **{**a, **{k: v for k, v in leaves.items() if k not in "xy"}})
    loss = (s * ds).sum() + ((n * dn).sum() if pre else 0)
    got = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    st = bsa.bsa_block_norm(x, y, eps=EPS, save_stats=True, **a)
    want = bsa.bsa_block_norm_backward(ds, dn, st[0], y, st[2], **a)
    assert all(torch.equal(got[k], want[k]) for k in leaves)
    # against central differences in fp32: h = 2^-5, error h^2 of the third derivative and
    # 2^-24 / h of the loss's terms
    for name in leaves:
        v = leaves[name].detach()
        e = torch.zeros_like(v)
        e.view(-1)[v.numel() // 2] = 2.0 ** -5
        def f(t):  # noqa: E306
            args = {**a, "x": x, "y": y, name: t}
            p, q, _ = bsa.bsa_block_norm(args.pop("x"), args.pop("y"), eps=EPS, **args)
            return (p.double() * ds).sum() + ((q.double() * dn).sum() if pre else 0)
        diff = ((f(v + e) - f(v - e)) * 2.0 ** 4).item()
        assert abs(diff - got[name].view(-1)[v.numel() // 2].item()) < 0.02 * max(1.0, abs(diff)), name
    # the norm alone: the stream's own path is torch's
    if pre:
        w = leaves["pre_weight"]
        s, n = block_norm(leaves["x"], pre=pre, pre_weight=w, eps=EPS)
        assert s is leaves["x"]
        gx, = torch.autograd.grad((s * ds).sum() + (n * dn).sum(), leaves["x"])
        st = bsa.bsa_block_norm(x, pre=pre, pre_weight=a["pre_weight"], eps=EPS, save_stats=True)[2]
        want = bsa.bsa_block_norm_backward(None, dn, x, None, st, pre=pre, pre_weight=a["pre_weight"])["x"] + ds
        assert torch.equal(gx, want)


@gpu
@needs_cuda
def test_the_norm_alone_has_no_scales():
    # without y the stream is x itself, whatever the C structure's scales hold (a zeroed one, too)
    a, x, _, _, dn = _make(2, 7, 768, None, "rms", 0, False, torch.bfloat16, torch.float32, 8, y=False)
    _, n, st = bsa.bsa_block_norm(x, eps=EPS, save_stats=True, **a)
    want = bsa.bsa_block_norm_backward(None, dn, x, None, st, **a)
    for alpha, beta in ((0.0, 0.0), (3.0, -0.5)):
        args = _args(rows_per_batch=7, C=768, post=0, post_weight=None, gate=None, pre_weight=a["pre_weight"].data_ptr(),
                     branch_scale=alpha, stream_scale=beta)
        got, dx = torch.empty_like(x), torch.empty_like(x)
        stream = torch.cuda.current_stream().cuda_stream
        assert bsa.lib.bsa_block_norm(ctypes.byref(args), x.data_ptr(), None, None, got.data_ptr(), None, stream) == bsa.BSA_OK
        assert bsa.lib.bsa_block_norm_backward(ctypes.byref(args), None, dn.data_ptr(), x.data_ptr(), None, st.data_ptr(),
                                               dx.data_ptr(), None, None, None, None, None, None, None, 0,
                                               stream) == bsa.BSA_OK
        assert torch.equal(dx, want["x"]) and torch.equal(got, n)


@gpu
@needs_cuda
@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("C", [1, 4, 64, 512, 1024, 8192])
@pytest.mark.parametrize("offset", [0, 1])  # rows with and without 16-byte starts
def test_layer_norm_gradient_is_that_of_the_stored_stream(C, ty, offset):
    # Rows close to constant, whose rounding to 16 bits moves them by more than, or a good part of,
    # their deviation: x = 4 + k steps of the type, stream_scale 1 + a quarter step / 4, so that the
    # stream is stored as x itself.  The gradient of a layer norm at x has neither a component
    # along the ones nor one along x - mean x beyond eps's.  C is a power of two and k small, so
    # that the sums behind mean and variance are exact in fp32 and the tolerance is that of a
    # normalised value without the mean's term.
    R, step = 6, {torch.bfloat16: 2.0 ** -5, torch.float16: 2.0 ** -8, torch.float32: 2.0 ** -8}[ty]
    g = torch.Generator(device="cuda").manual_seed(C)
    make = lambda: torch.empty(R * C + offset, dtype=ty, device="cuda")[offset:].view(R, C)  # noqa: E731
    x, y, ds, dn = make(), make(), make(), make()
    k = torch.randint(-4, 5, (R, C), generator=g, device="cuda")
    k[:2] = 0  # constant rows
    x.copy_(4 + step * k), y.zero_(), ds.copy_(torch.randn(R, C, generator=g, device="cuda"))
    dn.copy_(torch.randn(R, C, generator=g, device="cuda") + 0.5)
    beta = 1 + step / 16 if ty != torch.float32 else 1.0
    w = torch.rand(C, generator=g, device="cuda") + 0.5
    b = torch.rand(C, generator=g, device="cuda")
    a = dict(post=None, pre="layer", pre_weight=w, pre_bias=b, stream_scale=beta)
    stream, _, st = bsa.bsa_block_norm(x, y, eps=EPS, save_stats=True, **a)
    assert torch.equal(stream, x)
    got = bsa.bsa_block_norm_backward(ds, dn, stream, y, st, **a)
    X, W = _np(x), w.double().cpu().numpy()
    m, r = ON.stats(X, "layer", EPS)
    ref, mags = ON.backward(_np(ds), _np(dn), X, _np(y), np.concatenate([0 * m, 0 * r, m, r], 1), None, None, None, None,
                            1.0, beta, "layer", W, b.double().cpu().numpy())
    n, t = np.abs(X - m) * r, np.abs(_np(dn)) * W
    dmag = np.abs(_np(ds)) + r * (t + t.mean(1, keepdims=True) + n * (t * n).mean(1, keepdims=True))
    _near(got["x"], ref["x"], 2.0 ** -17 * dmag * beta, U[ty], "dx")
    _near(got["pre_weight"], ref["pre_weight"], (70 * 2.0 ** -24 + 2.0 ** -17) * mags["pre_weight"], U[torch.float32], "weight")


@gpu
@needs_cuda
def test_statistics_are_kept_only_for_a_gradient(monkeypatch):
    from block_sparse_attention_bigbird_b200 import autograd
    asked, forward = [], bsa.bsa_block_norm
    monkeypatch.setattr(bsa, "bsa_block_norm", lambda *p, save_stats, **k: (asked.append(save_stats), forward(*p, save_stats=save_stats, **k))[1])
    a, x, y, _, _ = _make(2, 9, 128, "rms", "layer", 1, True, torch.bfloat16, torch.float32, 5)
    want = forward(x, y, **a)
    leaf = x.clone().requires_grad_()
    weight = a["post_weight"].clone().requires_grad_()
    with torch.no_grad():
        got = [autograd.block_norm(leaf, y, eps=1e-6, **a)]
    with torch.inference_mode():
        got.append(autograd.block_norm(leaf, y, eps=1e-6, **a))
    got.append(autograd.block_norm(x, y, eps=1e-6, **a))
    assert asked == [False] * 3
    got.append(autograd.block_norm(leaf, y, eps=1e-6, **a))
    got.append(autograd.block_norm(x, y, eps=1e-6, **{**a, "post_weight": weight}))
    assert asked[3:] == [True] * 2 and got[3][0].requires_grad and got[4][1].requires_grad
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)
