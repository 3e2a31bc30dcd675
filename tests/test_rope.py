"""Rotary positions with several axes (bsa_rope_build, bsa_rope_from_table, bsa_rope_apply).

CPU: the tables of both builders against the oracle; refusals of the C ABI and of the binding,
all before any device work.
GPU: against the fp64 oracle over types, pair orders, strides, one token to many, odd sizes;
in place; far positions; captured and replayed; gradients through autograd.

Tolerance (from the arithmetic): the angle is formed in fp64 and reduced to a fraction of a turn
in [-1/2, 1/2] that is rounded to fp32 (2^-26 turns, 2^-23.3 radians); for |p freq| < 2^24
radians the fp64 product errs by less than 2^-28.  sincospi errs by at most 2 units of the
last place (2^-23).  So each of sin and cos errs by less than 2^-21.5, and an element of a pair
(u, v), two products and a sum in fp32 (3 x 2^-24), by less than 2^-21 (|u| + |v|); rounding to
the result's type adds half a step, relative 2^-8 (bf16), 2^-11 (fp16) or 2^-24 (fp32).
"""

import copy
import ctypes
import pickle

import numpy as np
import pytest
import torch

from block_sparse_attention_bigbird_b200 import bsa
from oracle import rope as OR

gpu = pytest.mark.gpu
needs_cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")


# ---------------------------------------------------------------- CPU
@pytest.mark.parametrize("sections,kw", [((32,), {}), ((8, 12, 12), {}), ((16, 24, 24), dict(base=1e6)),
                                         ((5, 0, 3), dict(per_axis=True)), ((6, 5, 5), dict(interleave=True)),
                                         ((1, 7), dict(interleave=True, per_axis=True)), ((128,), {})])
def test_tables_match_oracle(sections, kw):
    r = bsa.bsa_rope_build(sections, adjacent=True, **kw)
    axis, freq = bsa.bsa_rope_table(r)
    ref_axis, ref_freq = OR.tables(sections, **kw)
    assert np.array_equal(axis, ref_axis) and np.allclose(freq, ref_freq, rtol=1e-14)
    assert r.n_pairs == sum(sections) and r.adjacent and r.n_axes == ref_axis.max() + 1
    r2 = bsa.bsa_rope_from_table(axis, freq)
    assert all(np.array_equal(a, b) for a, b in zip(bsa.bsa_rope_table(r2), (axis, freq))) and not r2.adjacent


@pytest.mark.parametrize("args", [((), 1e4), ((0, 0), 1e4), ((-1, 4), 1e4), ((129,), 1e4), ((1,) * 9, 1e4),
                                  ((4,), 0.0), ((4,), -2.0), ((4,), float("nan")), ((4,), float("inf")),
                                  ((64,), 5e-324)])  # 5e-324 ** (-63 / 64) overflows
def test_build_refuses(args):
    with pytest.raises(bsa.BsaError) as e:
        bsa.bsa_rope_build(*args)
    assert e.value.code == bsa.BSA_ERR_INVALID_ARG


@pytest.mark.parametrize("axis,freq", [([0, 8], [1, 1]), ([-1], [1]), ([0], [np.inf]), ([0], [np.nan]), ([], []),
                                       ([0, 1], [1.0])])
def test_from_table_refuses(axis, freq):
    with pytest.raises(bsa.BsaError):
        bsa.bsa_rope_from_table(axis, freq)


def test_apply_refuses_before_device_work():
    rope = bsa.bsa_rope_build([4, 4])
    a, b = 1 << 20, 1 << 21
    strides, ps = (ctypes.c_int64 * 12)(*[16] * 12), (ctypes.c_int64 * 3)(1, 1, 1)

    def call(q=a, qo=a, H=2, k=b, ko=b, Hk=1, B=1, L=4, d=16, ty=bsa.BF16, st=strides, pos=a, pt=bsa.INT64, pst=ps,
             r=rope.handle):
        return bsa.lib.bsa_rope_apply(q, qo, H, k, ko, Hk, B, L, d, ty, st, pos, pt, pst, r, 0, None)
    for kw in (dict(q=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(r=None), dict(st=None), dict(pst=None),
               dict(B=-1), dict(L=-1), dict(H=-1), dict(Hk=-1), dict(d=0), dict(d=15), dict(q=a + 1), dict(ko=b + 1), dict(qo=b), dict(ko=a), dict(k=3 << 20, qo=b)):
        assert call(**kw) == bsa.BSA_ERR_INVALID_ARG, kw
    for kw in (dict(ty=bsa.E4M3), dict(ty=9), dict(pt=bsa.BF16), dict(d=258)):
        assert call(**kw) == bsa.BSA_ERR_UNSUPPORTED, kw
    for kw in (dict(B=0), dict(L=0), dict(H=0, k=None)):
        assert call(**kw) == bsa.BSA_OK, kw  # empty calls


def test_apply_refuses_positions_between_elements():
    rope = bsa.bsa_rope_build([4, 4])
    a, b = 1 << 20, 1 << 21
    strides, ps = (ctypes.c_int64 * 12)(*[16] * 12), (ctypes.c_int64 * 3)(1, 1, 1)
    for ty, off in ((bsa.INT64, 4), (bsa.INT64, 1), (bsa.INT32, 2), (bsa.FP32, 2)):
        code = bsa.lib.bsa_rope_apply(a, a, 2, b, b, 1, 1, 4, 16, bsa.BF16, strides, a + off, ty, ps, rope.handle, 0, None)
        assert code == bsa.BSA_ERR_INVALID_ARG, (ty, off)


def test_a_code_is_copied_and_stored_by_its_tables():
    for rope in (bsa.bsa_rope_build([8, 12, 12], 1e6, per_axis=True), bsa.bsa_rope_from_table([2, 0], [0.5, -3.0], True)):
        for again in (copy.deepcopy(rope), pickle.loads(pickle.dumps(rope))):
            assert (again.n_pairs, again.n_axes, again.adjacent) == (rope.n_pairs, rope.n_axes, rope.adjacent)
            assert again.handle.value != rope.handle.value
            assert all((s == t).all() for s, t in zip(bsa.bsa_rope_table(again), bsa.bsa_rope_table(rope)))


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 2, 4, 16)
    with pytest.raises(ValueError):
        bsa.bsa_rope_apply(q, None, torch.zeros(1, 4, dtype=torch.int64), bsa.bsa_rope_build([8]))


def test_positions_that_want_a_gradient_are_refused():
    from block_sparse_attention_bigbird_b200 import rotary
    pos = torch.zeros(1, 4, requires_grad=True)
    with pytest.raises(ValueError, match="positions"):
        rotary(torch.zeros(1, 2, 4, 16), None, pos, bsa.bsa_rope_build([8]))
    with torch.no_grad(), pytest.raises(ValueError, match="q must be"):  # none is wanted: q is what is wrong
        rotary(torch.zeros(1, 2, 4, 16), None, pos, bsa.bsa_rope_build([8]))


# ---------------------------------------------------------------- GPU
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def _check(got, x, positions, rope, inverse=False):
    axis, freq = bsa.bsa_rope_table(rope)
    xs = x.detach().double().cpu().numpy()
    ref = OR.apply(xs, positions.cpu().numpy(), axis, freq, rope.adjacent, inverse)
    err = 2.0 ** -21 * OR.magnitude(xs, len(axis), rope.adjacent)
    tol = U[x.dtype] * (np.abs(ref) + err) + err + 2.0 ** -25 * (x.dtype == torch.float16)
    bad = np.abs(got.detach().double().cpu().numpy() - ref) > tol
    assert not bad.any(), int(bad.sum())


CASES = [  # B, H, Hk, L, d, sections, type, adjacent
    (1, 1, 1, 1, 64, (32,), torch.bfloat16, False),
    (8, 16, 4, 1, 128, (16, 24, 24), torch.bfloat16, False),
    (2, 3, 5, 77, 64, (8, 12, 12), torch.bfloat16, True),
    (1, 13, 2, 33, 80, (20,), torch.float16, False),       # a tail of 40 columns
    (2, 2, 2, 19, 96, (16, 16), torch.float32, True),      # a tail of 32
    (1, 2, 1, 5, 6, (1, 1), torch.float32, False),         # no vectors: 2 of 3 pairs
    (3, 1, 2, 9, 15, (3, 4), torch.bfloat16, True),        # an odd head
    (1, 2, 2, 4, 2, (1,), torch.float16, False),
    (1, 4, 4, 300, 256, (128,), torch.bfloat16, False),
    (2, 12, 12, 1031, 64, (8, 12, 12), torch.bfloat16, False),
]


@gpu
@needs_cuda
@pytest.mark.parametrize("B,H,Hk,L,d,sections,ty,adjacent", CASES)
def test_matches_oracle(B, H, Hk, L, d, sections, ty, adjacent):
    g = torch.Generator(device="cuda").manual_seed(B * 100 + L)
    rope = bsa.bsa_rope_build(sections, adjacent=adjacent, per_axis=L % 2 == 0)
    q, k = (torch.randn(B, h, L, d, generator=g, device="cuda").to(ty) for h in (H, Hk))
    pos = torch.randint(-1000, 100_000, (len(sections), B, L), generator=g, device="cuda")
    for inverse in (False, True):
        for p in (pos, pos.to(torch.int32), pos.float(), pos[:, 0].contiguous()):
            got = bsa.bsa_rope_apply(q, k, p, rope, inverse=inverse)
            for x, y in zip((q, k), got):
                assert y.is_contiguous() and y.shape == x.shape
                _check(y, x, p, rope, inverse)
    again = bsa.bsa_rope_apply(q, k, pos, rope)
    assert all(torch.equal(a, b) for a, b in zip(again, bsa.bsa_rope_apply(q, k, pos, rope)))
    only, none = bsa.bsa_rope_apply(q, None, pos, rope)
    assert none is None and torch.equal(only, again[0])


@gpu
@needs_cuda
def test_strided_inputs_and_in_place():
    g = torch.Generator(device="cuda").manual_seed(5)
    rope = bsa.bsa_rope_build([8, 12, 12])
    B, L, H = 2, 65, 3
    pos = torch.randint(0, 5000, (3, B, L), generator=g, device="cuda")
    packed = torch.randn(B, L, 3, H, 64, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = (packed[:, :, i].transpose(1, 2) for i in range(3))
    want = bsa.bsa_rope_apply(q.contiguous(), k.contiguous(), pos, rope)
    got = bsa.bsa_rope_apply(q, k, pos, rope)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # rows that start at odd elements: no vector access
    odd = torch.randn(B, H, L, 65, generator=g, device="cuda").to(torch.bfloat16)[..., 1:]
    assert torch.equal(bsa.bsa_rope_apply(odd, None, pos, rope)[0], bsa.bsa_rope_apply(odd.contiguous(), None, pos, rope)[0])
    # a broadcast input (all heads the same memory) and positions shared by expand
    one = torch.randn(B, 1, L, 64, generator=g, device="cuda").to(torch.bfloat16)
    shared = pos[:, :1].expand(3, B, L)
    assert torch.equal(bsa.bsa_rope_apply(one.expand(B, H, L, 64), None, shared, rope)[0],
                       bsa.bsa_rope_apply(one.repeat(1, H, 1, 1), None, shared.contiguous(), rope)[0])
    # in place, in the packed tensor: v stays
    before = v.clone()
    a, b = bsa.bsa_rope_apply(q, k, pos, rope, q_out=q, k_out=k)
    assert a is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before)
    # in place with columns past the pairs: they stay too
    part = bsa.bsa_rope_build([8])
    x = torch.randn(B, H, L, 64, generator=g, device="cuda").to(torch.bfloat16)
    want = bsa.bsa_rope_apply(x, None, pos[:1], part)[0]
    bsa.bsa_rope_apply(x, None, pos[:1], part, q_out=x)
    assert torch.equal(x, want)


@gpu
@needs_cuda
def test_far_positions_keep_their_phase():
    # |p freq| up to 2^31 radians: the fp64 product errs by 2^-22 at most, twice the bound's 2^-23.3
    rope = bsa.bsa_rope_from_table([0, 0], [1.0, 0.001])
    pos = torch.tensor([[2 ** 31 - 1, 2 ** 31 - 7, 10 ** 6, -(2 ** 31)]], device="cuda")
    x = torch.ones(1, 1, 4, 4, device="cuda")
    got = bsa.bsa_rope_apply(x, None, pos, rope)[0].double().cpu().numpy()
    ref = OR.apply(np.ones((1, 1, 4, 4)), pos.cpu().numpy(), *bsa.bsa_rope_table(rope))
    assert np.abs(got - ref).max() < 2 * 2.0 ** -20


@gpu
@needs_cuda
def test_empty_and_refused_calls():
    rope = bsa.bsa_rope_build([8, 12, 12])
    pos = torch.zeros(3, 2, 0, dtype=torch.int64, device="cuda")
    assert bsa.bsa_rope_apply(torch.zeros(2, 3, 0, 64, device="cuda"), None, pos, rope)[0].shape == (2, 3, 0, 64)
    q = torch.zeros(2, 3, 4, 64, device="cuda")
    pos = torch.zeros(3, 2, 4, dtype=torch.int64, device="cuda")
    ok = lambda **kw: bsa.bsa_rope_apply(**{**dict(q=q, k=q, positions=pos, rope=rope), **kw})  # noqa: E731
    ok()
    for kw in (dict(q=q.to(torch.float64)), dict(q=q.transpose(2, 3)), dict(q=q[0]), dict(k=q[:, :, :3]),
               dict(k=q.half()), dict(positions=pos[:2]), dict(positions=pos[:, :1]), dict(positions=pos[..., :3]),
               dict(positions=pos.to(torch.int16)), dict(positions=pos.cpu()), dict(k=None, k_out=q),
               dict(q_out=q.half()), dict(q_out=q[:1].expand(2, 3, 4, 64)), dict(k=q.cpu())):
        with pytest.raises(ValueError):
            ok(**kw)
    with pytest.raises(bsa.BsaError):
        ok(q=q[..., :32].contiguous(), k=None)  # 32 pairs need 64 columns


@gpu
@needs_cuda
def test_streams_and_graphs():
    rope = bsa.bsa_rope_build([8, 12, 12])
    q, k = torch.randn(2, 2, 4, 50, 64, device="cuda").unbind(0)
    pos = torch.randint(0, 999, (3, 2, 50), device="cuda")
    want = bsa.bsa_rope_apply(q, k, pos, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for given in (s, s.cuda_stream):
        got = bsa.bsa_rope_apply(q, k, pos, rope, stream=given)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bsa.bsa_rope_apply(q, k, pos, rope)
    q.mul_(2)
    graph.replay()
    assert torch.equal(got[0], bsa.bsa_rope_apply(q, k, pos, rope)[0])


@gpu
@needs_cuda
def test_gradients():
    from block_sparse_attention_bigbird_b200 import rotary
    rope = bsa.bsa_rope_build([8, 12, 12])
    g = torch.Generator(device="cuda").manual_seed(8)
    pos = torch.randint(0, 5000, (3, 2, 21), generator=g, device="cuda")
    q = torch.randn(2, 4, 21, 64, generator=g, device="cuda", requires_grad=True)
    k = torch.randn(2, 1, 21, 64, generator=g, device="cuda", requires_grad=True)
    dq, dk = torch.randn(2, 4, 21, 64, generator=g, device="cuda"), torch.randn(2, 1, 21, 64, generator=g, device="cuda")
    a, b = rotary(q, k, pos, rope)
    gq, gk = torch.autograd.grad((a * dq).sum() + (b * dk).sum(), (q, k))
    _check(gq, dq, pos, rope, inverse=True)
    _check(gk, dk, pos, rope, inverse=True)
    # a key head shared by four query heads through expand: its gradient is their sum
    a, b = rotary(q, k.expand(2, 4, 21, 64), pos, rope)
    gs, = torch.autograd.grad((a.detach() * b).sum(), k)
    ref = bsa.bsa_rope_apply(a.detach(), None, pos, rope, inverse=True)[0].sum(1, keepdim=True)
    assert torch.equal(gs, ref)
    # only k used; a gradient that is one number everywhere (stride 0)
    a, b = rotary(q, k, pos, rope)
    gk, = torch.autograd.grad(b.sum(), k, retain_graph=True)
    _check(gk, torch.ones_like(k), pos, rope, inverse=True)
    assert torch.autograd.grad(b.sum(), q, allow_unused=True)[0] is None
    # against a central difference of the whole map, in fp64 on the oracle's side: the map is
    # linear, so the difference over h = 1 is the map itself
    e = torch.zeros_like(q)
    e[1, 2, 3, 5] = 1.0
    up, _ = bsa.bsa_rope_apply(q.detach() + e, None, pos, rope)
    down, _ = bsa.bsa_rope_apply(q.detach() - e, None, pos, rope)
    diff = ((up - down) / 2 * dq).sum().item()
    assert abs(diff - torch.autograd.grad((rotary(q, None, pos, rope)[0] * dq).sum(), q)[0][1, 2, 3, 5].item()) < 1e-5


@gpu
@needs_cuda
def test_more_heads_than_a_grid_has_rows():
    rope = bsa.bsa_rope_build([2, 2], adjacent=True)
    g = torch.Generator(device="cuda").manual_seed(13)
    for L in (1, 3):
        q, k = (torch.randn(1, h, L, 8, generator=g, device="cuda") for h in (66_000, 5_001))
        pos = torch.randint(0, 999, (2, 1, L), generator=g, device="cuda")
        for x, y in zip((q, k), bsa.bsa_rope_apply(q, k, pos, rope)):
            _check(y, x, pos, rope)


@gpu
@needs_cuda
def test_a_replayed_graph_reads_all_of_its_inputs_again():
    rope = bsa.bsa_rope_build([8, 12, 12])
    g = torch.Generator(device="cuda").manual_seed(12)
    q = torch.randn(2, 6, 50, 64, generator=g, device="cuda")
    k = torch.randn(2, 50, 3, 64, generator=g, device="cuda").transpose(1, 2)
    pos = torch.randint(0, 999, (3, 2, 50), generator=g, device="cuda")
    bsa.bsa_rope_apply(q, k, pos, rope)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bsa.bsa_rope_apply(q, k, pos, rope)
    for change in (lambda: q.mul_(2), lambda: k.add_(1), lambda: pos.add_(17), lambda: (q.neg_(), k.mul_(3), pos.mul_(2))):
        change()
        graph.replay()
        want = bsa.bsa_rope_apply(q, k, pos, rope)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        _check(got[1], k, pos, rope)
