"""The block quantiser and the block-scaled 8-bit product (bsa_fp8_quantize, bsa_fp8_matmul).

CPU: refusals of the C ABI before any device work.
GPU: codes and scales bit by bit against the oracle (every step of the definition is one correctly
rounded operation), blocks with zeros, infinities and NaN; the product against the fp64
oracle over types, scale forms, one row to many, odd sizes, a K that ends inside a block, splits
of K; what lies behind a row's end is not used; captured, on other streams, with another call's
workspace; the linear layer's three products through autograd.

Tolerance of the product (from the arithmetic): the codes' products are exact in fp32; a block's
128 are added in fp32 by the tensor cores in some order with at most a unit of the last place
lost a step (2^-23), then kb blocks with their scale (the scales' product and the fma round, 2^-24
each) and at most 32 splits and a bias.  So the error is below (128 + kb + 40) 2^-23 of the sum of
magnitudes; rounding to the result's type adds half a step, 2^-8 (bf16) or 2^-24.
"""

import ctypes

import numpy as np
import pytest
import torch

from block_sparse_attention_bigbird_b200 import bsa
from oracle import fp8 as O8

gpu = pytest.mark.gpu
needs_cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
NAME = {E4: "e4m3", E5: "e5m2"}


# ---------------------------------------------------------------- CPU
def test_quantize_refuses_before_device_work():
    p = 1 << 20

    def call(x=p, ty=bsa.BF16, R=4, C=20, square=0, ct=bsa.E4M3, codes=p, ld=32, scale=p, codes_t=p, ld_t=16, scale_t=p):
        return bsa.lib.bsa_fp8_quantize(x, ty, R, C, square, ct, codes, ld, scale, codes_t, ld_t, scale_t, None)
    for kw in (dict(x=None), dict(R=-1), dict(C=-1), dict(codes=None, codes_t=None), dict(scale=None), dict(scale_t=None),
               dict(x=p + 1), dict(codes=p + 8), dict(codes_t=p + 8), dict(ld=20), dict(ld=16), dict(ld_t=8),
               dict(ld_t=0), dict(R=17)):
        assert call(**kw) == bsa.BSA_ERR_INVALID_ARG, kw
    for kw in (dict(ty=bsa.E4M3), dict(ct=bsa.BF16), dict(ty=77)):
        assert call(**kw) == bsa.BSA_ERR_UNSUPPORTED, kw
    assert call(R=0) == bsa.BSA_OK and call(C=0) == bsa.BSA_OK


def test_quantize_refuses_scales_between_elements():
    p = 1 << 20
    for scale, scale_t in ((p + 2, p), (p, p + 1)):
        code = bsa.lib.bsa_fp8_quantize(p, bsa.BF16, 4, 20, 0, bsa.E4M3, p, 32, scale, p, 16, scale_t, None)
        assert code == bsa.BSA_ERR_INVALID_ARG, (scale, scale_t)


def test_matmul_refuses_before_device_work():
    p = 1 << 20

    def call(a=p, at=bsa.E4M3, lda=64, sa=p, ar=1, b=p, bt=bsa.E5M2, ldb=64, sb=p, br=128, bias=None, biast=bsa.BF16, M=4,
             N=8, K=50, out=p, ot=bsa.BF16):
        return bsa.lib.bsa_fp8_matmul(a, at, lda, sa, ar, b, bt, ldb, sb, br, bias, biast, M, N, K, out, ot, None, 0, None)
    for kw in (dict(a=None), dict(b=None), dict(sa=None), dict(sb=None), dict(out=None), dict(M=-1), dict(N=-1),
               dict(K=0), dict(a=p + 8), dict(b=p + 4), dict(lda=60), dict(ldb=48), dict(out=p + 1), dict(sa=p + 2),
               dict(bias=p + 1)):
        assert call(**kw) == bsa.BSA_ERR_INVALID_ARG, kw
    for kw in (dict(at=bsa.BF16), dict(bt=bsa.FP32), dict(ot=bsa.FP16), dict(ar=64), dict(br=0),
               dict(bias=p, biast=bsa.FP16)):
        assert call(**kw) == bsa.BSA_ERR_UNSUPPORTED, kw
    assert call(M=0) == bsa.BSA_OK and call(N=0) == bsa.BSA_OK
    n = ctypes.c_size_t(7)
    assert bsa.lib.bsa_fp8_matmul_workspace_bytes(4, 8, 50, ctypes.byref(n)) == bsa.BSA_OK and n.value == 0
    assert bsa.lib.bsa_fp8_matmul_workspace_bytes(4, 8, 0, ctypes.byref(n)) == bsa.BSA_ERR_INVALID_ARG
    assert bsa.lib.bsa_fp8_matmul_workspace_bytes(4, 8, 50, None) == bsa.BSA_ERR_INVALID_ARG


def test_linear_refuses_a_gradient_type_at_once():
    from block_sparse_attention_bigbird_b200 import fp8_linear
    for bad in (torch.bfloat16, torch.float8_e8m0fnu):
        with pytest.raises(ValueError, match="grad_dtype"):
            fp8_linear(torch.zeros(2, 16), torch.zeros(4, 16), grad_dtype=bad)


# ---------------------------------------------------------------- GPU: quantiser
def _same_codes(codes, scale, x, fmt, square):
    ref, ref_scale = O8.quantise(x.float().cpu().numpy(), fmt, square)
    assert np.array_equal(scale.cpu().numpy(), ref_scale, equal_nan=True)
    assert np.array_equal(codes.float().cpu().numpy().astype(np.float64), ref, equal_nan=True)


@gpu
@needs_cuda
@pytest.mark.parametrize("R,C", [(1, 1), (1, 768), (3, 128), (128, 128), (129, 257), (77, 1000), (200, 24), (16, 4096),
                                 (300, 333), (1000, 8)])
@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float16, torch.float32])
def test_quantiser_bit_by_bit(R, C, ty):
    g = torch.Generator(device="cuda").manual_seed(R + C)
    x = (torch.randn(R, C, generator=g, device="cuda") * torch.logspace(-4, 3, C, device="cuda")).to(ty)
    for square in (False, True):
        for dt in (E4, E5):
            both = bsa.bsa_fp8_quantize(x, square=square, rows=True, cols=True, dtype=dt)
            rows = bsa.bsa_fp8_quantize(x, square=square, dtype=dt)
            cols = bsa.bsa_fp8_quantize(x, square=square, rows=False, cols=True, dtype=dt)
            _same_codes(*rows, x, NAME[dt], square)
            _same_codes(*cols, x.t(), NAME[dt], square)
            for a, b in zip(both, rows + cols):
                assert a.shape == b.shape and a.dtype == b.dtype
                assert torch.equal(a.float(), b.float())
            assert rows[0].shape == (R, C) and rows[0].stride(0) % 16 == 0 and cols[0].shape == (C, R)


@gpu
@needs_cuda
def test_quantiser_special_blocks():
    x = torch.zeros(256, 384, device="cuda")
    x[1, 5], x[2, 200], x[3, 300] = float("nan"), float("inf"), -float("inf")
    x[4, 10], x[4, 11] = 1e-38, -3e-39           # below the least maximum and subnormal
    x[5, 130:140], x[6, :] = 3.4e38, 1e-30
    x[130, :] = torch.linspace(-1, 1, 384, device="cuda")
    for dt in (E4, E5):
        _same_codes(*bsa.bsa_fp8_quantize(x, dtype=dt), x, NAME[dt], False)
        _same_codes(*bsa.bsa_fp8_quantize(x, rows=False, cols=True, dtype=dt), x.t(), NAME[dt], False)
        _same_codes(*bsa.bsa_fp8_quantize(x, square=True, dtype=dt), x, NAME[dt], True)
    codes, scale = bsa.bsa_fp8_quantize(torch.zeros(3, 0 + 5, device="cuda"))
    assert (codes.float() == 0).all() and scale.isfinite().all()
    # neighbours of a block that is not finite are untouched
    codes, scale = bsa.bsa_fp8_quantize(x)
    assert scale[1, 0].isnan() and scale[1, 1:].isfinite().all() and scale[2, 1].isinf() and scale[130].isfinite().all()


@gpu
@needs_cuda
def test_quantiser_shapes_and_refusals():
    x = torch.randn(2, 5, 40, device="cuda")
    codes, scale = bsa.bsa_fp8_quantize(x)
    assert codes.shape == (10, 40) and scale.shape == (10, 1)
    e = bsa.bsa_fp8_quantize(torch.zeros(0, 64, device="cuda"), rows=True, cols=True)
    assert e[0].shape == (0, 64) and e[2].shape == (64, 0) and e[3].shape == (64, 0)
    # an address that is not 16-byte aligned: the same codes
    y = torch.randn(64 * 40 + 1, device="cuda").bfloat16()[1:].view(64, 40)
    assert all(torch.equal(a.float(), b.float()) for a, b in
               zip(bsa.bsa_fp8_quantize(y, cols=True), bsa.bsa_fp8_quantize(y.clone(), cols=True)))
    for kw in (dict(x=x.cpu()), dict(x=x.double()), dict(x=x.transpose(0, 1)), dict(x=x, dtype=torch.int8),
               dict(x=x, rows=False), dict(x=torch.tensor(1.0, device="cuda"))):
        with pytest.raises(ValueError):
            bsa.bsa_fp8_quantize(**kw)


# ---------------------------------------------------------------- GPU: product
def _codes(rows, K, dt, g, garbage=True):
    """Random finite codes in padded rows; what lies behind a row's end is NaN."""
    ld = -(-K // 16) * 16
    raw = torch.full((rows, ld), 0x7F, dtype=torch.uint8, device="cuda").view(dt)
    v = (torch.randn(rows, K, generator=g, device="cuda") * (60 if dt is E4 else 3000))
    raw[:, :K] = v.clamp(-O8.TOP[NAME[dt]], O8.TOP[NAME[dt]]).to(dt)
    return raw[:, :K]


def _operands(M, N, K, ta, tb, ar, br, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kb = -(-K // 128)
    s = lambda n, r: torch.rand(-(-n // r), kb, generator=g, device="cuda") * 0.02 + 1e-3  # noqa: E731
    return _codes(M, K, ta, g), s(M, ar), _codes(N, K, tb, g), s(N, br), g


def _check(got, a, sa, b, sb, bias=None):
    ref, mag = O8.product(*(t.float().cpu().numpy() for t in (a, sa, b, sb)), None if bias is None else
                          bias.float().cpu().numpy())
    err = (128 + sa.shape[1] + 40) * 2.0 ** -23 * mag
    u = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    bad = np.abs(got.double().cpu().numpy() - ref) > u * (np.abs(ref) + err) + err
    assert not bad.any(), int(bad.sum())


SIZES = [(1, 64, 64), (1, 1, 1), (3, 17, 129), (8, 300, 1000), (8, 2304, 768), (5, 100, 2048 + 16), (7, 33, 8320),
         (9, 256, 512), (33, 64, 50), (128, 128, 128), (129, 257, 130), (100, 2050, 1104), (300, 70, 4096), (64, 1000, 23),
         (777, 514, 272), (1300, 768, 640), (40, 16, 8192), (2000, 1, 384)]


@gpu
@needs_cuda
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("ar,br", [(1, 128), (1, 1), (128, 128)])
def test_product_matches_oracle(M, N, K, ar, br):
    ta, tb = ((E4, E4), (E5, E4), (E4, E5))[(M + N + K) % 3]
    a, sa, b, sb, g = _operands(M, N, K, ta, tb, ar, br, M + 7 * N + K)
    bias = torch.randn(N, generator=g, device="cuda")
    for dt, bs in ((torch.bfloat16, None), (torch.float32, bias), (torch.bfloat16, bias.bfloat16()), (torch.float32, None)):
        got = bsa.bsa_fp8_matmul(a, sa, b, sb, bias=bs, out_dtype=dt)
        assert got.shape == (M, N) and got.dtype == dt
        _check(got, a, sa, b, sb, bs)
        assert torch.equal(got, bsa.bsa_fp8_matmul(a, sa, b, sb, bias=bs, out_dtype=dt))
    assert bsa.bsa_sync_status() == 0


@gpu
@needs_cuda
def test_product_sampled_rows_at_the_layers_size():
    M, N, K = 4 * 16384, 2304, 768
    a, sa, b, sb, g = _operands(M, N, K, E4, E4, 1, 128, 3)
    got = bsa.bsa_fp8_matmul(a, sa, b, sb)
    rows = torch.randint(0, M, (96,), generator=g, device="cuda")
    rows[:3] = torch.tensor([0, M - 1, 127])
    _check(got[rows], a[rows], sa[rows], b, sb)
    a, sa, b, sb, g = _operands(512, 768, 65536, E5, E4, 1, 1, 4)  # K split over SMs
    assert bsa.bsa_fp8_matmul_workspace_bytes(512, 768, 65536) > 0
    got = bsa.bsa_fp8_matmul(a, sa, b, sb, out_dtype=torch.float32)
    _check(got[::37], a[::37], sa[::37], b, sb)


@gpu
@needs_cuda
def test_product_of_codes_that_are_not_finite():
    a, sa, b, sb, _ = _operands(200, 300, 256, E4, E4, 1, 128, 5)
    want = bsa.bsa_fp8_matmul(a, sa, b, sb, out_dtype=torch.float32)
    a[7, 3] = float("nan")
    sa[9, 1] = float("inf")
    got = bsa.bsa_fp8_matmul(a, sa, b, sb, out_dtype=torch.float32)
    keep = [i for i in range(200) if i not in (7, 9)]
    assert got[7].isnan().all() and not got[9].isfinite().any() and torch.equal(got[keep], want[keep])


@gpu
@needs_cuda
def test_product_out_workspace_streams_and_graphs():
    a, sa, b, sb, _ = _operands(256, 128, 8192, E4, E4, 1, 128, 6)
    n = bsa.bsa_fp8_matmul_workspace_bytes(256, 128, 8192)
    assert n > 0
    want = bsa.bsa_fp8_matmul(a, sa, b, sb)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty(256, 128, dtype=torch.bfloat16, device="cuda")
    assert bsa.bsa_fp8_matmul(a, sa, b, sb, out=out, workspace=ws) is out and torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = bsa.bsa_fp8_matmul(a, sa, b, sb, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graphs = []
    for i in range(2):  # two graphs, each with its own allocation
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q = bsa.bsa_fp8_quantize(want, square=False, rows=True, cols=True)
            graphs.append((graph, bsa.bsa_fp8_matmul(a, sa, b, sb), bsa.bsa_fp8_matmul(q[0], q[1], q[0], q[1])))
    for graph, *_ in graphs:
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.current_stream())
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want) and torch.equal(graphs[1][1], want) and torch.equal(graphs[0][2], graphs[1][2])
    assert bsa.bsa_sync_status() == 0


@gpu
@needs_cuda
def test_a_product_that_gives_up_is_reported():
    ops = _operands(64, 64, 256, E4, E4, 1, 128, 8)[:4]
    want = bsa.bsa_fp8_matmul(*ops)
    assert bsa.bsa_sync_status() == 0
    bsa.bsa_debug_product_wait_timeout(2_000_000)  # 2 ms at a barrier that nothing completes
    assert bsa.bsa_sync_status() == bsa.BSA_ERR_DEVICE_TIMEOUT
    assert bsa.bsa_sync_status() == 0  # the status is cleared
    bsa.bsa_debug_wait_timeout(2_000_000)
    bsa.bsa_debug_product_wait_timeout(2_000_000)
    assert bsa.bsa_sync_status() == bsa.BSA_ERR_DEVICE_TIMEOUT
    assert bsa.bsa_sync_status() == 0  # both are
    assert torch.equal(bsa.bsa_fp8_matmul(*ops), want)


@gpu
@needs_cuda
def test_product_empty_and_refused():
    a, sa, b, sb, _ = _operands(20, 40, 100, E4, E5, 1, 1, 7)
    z = bsa.bsa_fp8_matmul(a[:0], sa[:0], b, sb)
    assert z.shape == (0, 40)
    assert bsa.bsa_fp8_matmul(a, sa, b[:0], sb[:0]).shape == (20, 0)
    tight = a.contiguous()  # rows of 100 bytes
    for kw in (dict(a=tight), dict(a=a.float()), dict(a=a.t()), dict(b=b[:, :64]), dict(a_scale=sa[:, :0]),
               dict(a_scale=sa[:19]), dict(b_scale=sb.double()), dict(a_scale=sa.cpu()), dict(a=a[:, 1:], b=b[:, 1:]),
               dict(bias=torch.zeros(39, device="cuda")), dict(bias=torch.zeros(40, device="cuda").half()),
               dict(out_dtype=torch.float16), dict(out=torch.zeros(20, 41, device="cuda")),
               dict(out=torch.zeros(20, 40, device="cuda"), out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            bsa.bsa_fp8_matmul(**{**dict(a=a, a_scale=sa, b=b, b_scale=sb), **kw})
    big = _operands(256, 128, 8192, E4, E4, 1, 128, 6)[:4]
    with pytest.raises(bsa.BsaError) as e:
        bsa.bsa_fp8_matmul(*big, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == bsa.BSA_ERR_WORKSPACE


# ---------------------------------------------------------------- GPU: the linear layer
@gpu
@needs_cuda
@pytest.mark.parametrize("shape,N,xt,wt,gt", [((3, 50, 192), 130, torch.bfloat16, torch.float32, E4),
                                              ((700, 256), 384, torch.float32, torch.bfloat16, E5),
                                              ((1, 1, 64), 40, torch.bfloat16, torch.bfloat16, E4)])
def test_linear_gradients_are_the_products(shape, N, xt, wt, gt):
    from block_sparse_attention_bigbird_b200 import fp8_linear
    g = torch.Generator(device="cuda").manual_seed(N)
    K = shape[-1]
    x = torch.randn(*shape, generator=g, device="cuda").to(xt).requires_grad_()
    w = (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).to(wt).requires_grad_()
    bias = torch.randn(N, generator=g, device="cuda").requires_grad_()
    y = fp8_linear(x, w, bias, grad_dtype=gt)
    dy = torch.randn(*shape[:-1], N, generator=g, device="cuda").to(xt)
    dx, dw, db = torch.autograd.grad(y, (x, w, bias), dy)
    assert y.shape == (*shape[:-1], N) and y.dtype == xt and dx.dtype == xt and dw.dtype == wt

    def q(t, square=False, fmt="e4m3"):
        return O8.quantise(t.detach().float().reshape(-1, t.shape[-1]).cpu().numpy(), fmt, square)

    def near(got, a, b, bs=None):
        ref, mag = O8.product(*a, *b, bs)
        err = (128 + a[1].shape[1] + 40) * 2.0 ** -23 * mag
        u = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[got.dtype]
        got = got.detach().double().cpu().numpy().reshape(ref.shape)
        assert (np.abs(got - ref) <= u * (np.abs(ref) + err) + err).all()
    x2, d2 = x.detach().reshape(-1, K), dy.reshape(-1, N)
    f = NAME[gt]
    near(y, q(x2), q(w, True), bias.detach().cpu().numpy())
    near(dx, q(d2, fmt=f), q(w.t(), True))
    near(dw, q(d2.t(), fmt=f), q(x2.t()))
    assert torch.allclose(db, d2.float().sum(0), atol=1e-4 * len(d2), rtol=1e-5)
    # the exact layer is near: each operand is off by at most 2^-4 of its value, or by half its
    # format's least step of its block's maximum, so the product by 2^-2.9 of its magnitudes
    exact = x2.double() @ w.detach().double().t() + bias.detach().double()
    mags = x2.double().abs() @ w.detach().double().abs().t()
    assert ((y.detach().double().reshape(-1, N) - exact).abs() <= 0.14 * mags + 2.0 ** -8 * exact.abs() + 0.02).all()


@gpu
@needs_cuda
def test_linear_parts_and_no_rows():
    from block_sparse_attention_bigbird_b200 import fp8_linear
    w = torch.randn(32, 64, device="cuda", requires_grad=True)
    x = torch.zeros(0, 64, device="cuda", requires_grad=True)
    y = fp8_linear(x, w)
    dx, dw = torch.autograd.grad(y.sum(), (x, w))
    assert y.shape == (0, 32) and dx.shape == (0, 64) and (dw == 0).all()
    x = torch.randn(5, 64, device="cuda")
    dw, = torch.autograd.grad(fp8_linear(x, w).sum(), w)
    xg = x.clone().requires_grad_()
    dx, = torch.autograd.grad(fp8_linear(xg, w.detach()).sum(), xg)
    both = torch.autograd.grad(fp8_linear(xg, w).sum(), (xg, w))
    assert torch.equal(both[0], dx) and torch.equal(both[1], dw)
    with torch.no_grad():
        assert torch.equal(fp8_linear(xg, w), fp8_linear(xg.detach(), w.detach()))
    for bad in ((x.half(), w), (x[:, :60], w), (x, w[:0]), (x[:, :0], w[:, :0])):
        with pytest.raises(ValueError):
            fp8_linear(*bad)
