"""The operators around the attention together: BigBirdSelfAttention with rotary positions and
8-bit projections, and BigBirdBlock.

CPU: refusals; the layer with rotary positions over fakes of the library on the fp64 oracle,
against the same steps spelled out (positions by default, the order of turning and copying).
GPU: a stack of two blocks, fused over their border, equal to the same calls made one by one;
its gradients against those of the same steps in torch fp32 with the kernels' roundings as
noise: a wrong path is off by the gradient's own size, the bound is a fraction of it.
"""

import copy
import pickle

import numpy as np
import pytest
import torch

from block_sparse_attention_bigbird_b200 import bsa
from block_sparse_attention_bigbird_b200 import layer as LY
from oracle import rope as OR

gpu = pytest.mark.gpu
needs_cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")


def test_refusals():
    with pytest.raises(ValueError):
        LY.BigBirdSelfAttention(128, 2, fused=True, fp8=True)
    with pytest.raises(ValueError):
        LY.BigBirdSelfAttention(128, 2, rope=(20, 20))  # 40 pairs of a head of 64
    with pytest.raises(ValueError):
        LY.BigBirdSelfAttention(128, 2)(torch.zeros(1, 64, 128), positions=torch.zeros(1, 64))
    with pytest.raises(ValueError):
        LY.BigBirdSelfAttention(128, 2, fp8=True)(torch.zeros(1, 64, 128))
    with pytest.raises(ValueError):
        LY.BigBirdBlock(128, 2, pre=None)
    one, other = LY.BigBirdBlock(128, 2), LY.BigBirdBlock(128, 2, eps=1e-5)
    with pytest.raises(ValueError, match="eps"):
        one(torch.zeros(1, 64, 128), following=other)


def test_the_block_refuses_types_that_do_not_go_together():
    x = torch.zeros(1, 64, 128, dtype=torch.bfloat16)
    block = LY.BigBirdBlock(128, 2, post="layer")  # all fp32, for a bf16 stream
    with pytest.raises(ValueError, match="projections"):
        block(x)
    with pytest.raises(ValueError, match="fused"):
        LY.BigBirdBlock(128, 2, fused=True)(x)
    block.attention.to(torch.bfloat16)
    for module, kw in ((block, dict(gate=torch.zeros(128, dtype=torch.bfloat16))),
                       (block, dict(following=LY.BigBirdBlock(128, 2).to(torch.bfloat16))),
                       (LY.BigBirdBlock(128, 2, fp8=True).half(), {})):
        with pytest.raises(ValueError, match="norm parameters and gate"):
            module(x, **kw)
    block.post_bias.data = block.post_bias.data.double()
    with pytest.raises(ValueError, match="norm parameters and gate"):
        block(x)


def test_the_block_takes_the_types_that_do(monkeypatch):
    # over a norm and an attention that do nothing: which calls get past the types
    monkeypatch.setattr(LY, "block_norm", lambda x, y=None, **_: (x, x))
    x = torch.zeros(1, 64, 128, dtype=torch.bfloat16)
    for kw, attention, rest in ((dict(fp8=True), torch.float32, torch.float32), (dict(fp8=True), torch.bfloat16, torch.float32),
                                (dict(fused=True), torch.bfloat16, torch.float32), ({}, torch.bfloat16, torch.bfloat16),
                                ({}, torch.bfloat16, torch.float32)):
        block = LY.BigBirdBlock(128, 2, **kw).to(rest)
        block.attention.to(attention)
        block.attention.forward = lambda t, **_: t
        assert block(x, following=block)[0] is x
    block = LY.BigBirdBlock(128, 2)  # autocast casts the projections' weights
    block.attention.forward = lambda t, **_: t
    with torch.autocast("cpu", torch.bfloat16):
        assert block(x) is x
    assert block(x.float()).dtype == torch.float32


def test_a_block_with_rotary_positions_is_copied():
    m = LY.BigBirdBlock(128, 2, rope=(8, 12, 12))
    again = copy.deepcopy(m)
    assert again.attention.rope is not m.attention.rope and again.attention.rope.n_pairs == 32
    assert all((s == t).all() for s, t in zip(m.state_dict().values(), again.state_dict().values()))


def test_a_block_that_has_run_is_copied_and_stored():
    m = LY.BigBirdBlock(128, 2, rope=(8, 12, 12))
    m.attention._layouts[(64, "cuda:0")] = bsa.bsa_layout_build(2, 64)  # what a call leaves behind
    for again in (copy.deepcopy(m), pickle.loads(pickle.dumps(m))):
        assert not again.attention._layouts and len(m.attention._layouts) == 1  # built again on first use
        assert all((s == t).all() for s, t in zip(m.state_dict().values(), again.state_dict().values()))
        assert again.attention.rope.n_pairs == 32


def test_rotary_in_the_layer_over_fakes(monkeypatch):
    seen = {}

    def fake_apply(q, k, positions, rope, inverse=False, **_):
        axis, freq = bsa.bsa_rope_table(rope)
        turn = lambda t: None if t is None else torch.from_numpy(  # noqa: E731
            OR.apply(t.detach().numpy(), positions.numpy(), axis, freq, inverse=inverse))
        seen["positions"] = positions
        return turn(q), turn(k)

    def fake_attention(q, k, v, layout, key_mask=None):
        assert all(t.is_contiguous() for t in (q, k, v))
        return torch.softmax(q @ k.transpose(-1, -2) / 8, -1) @ v
    monkeypatch.setattr(bsa, "bsa_rope_apply", fake_apply)
    monkeypatch.setattr(LY, "block_sparse_attention", fake_attention)
    monkeypatch.setattr(LY.BigBirdSelfAttention, "layout", lambda self, L, device: None)
    torch.manual_seed(0)
    B, H, L = 2, 2, 6
    m = LY.BigBirdSelfAttention(128, H, rope=(8, 12)).double()
    x = torch.randn(B, L, 128, dtype=torch.float64, requires_grad=True)
    q, k, v = m.qkv(x).view(B, L, 3, H, 64).permute(2, 0, 3, 1, 4).unbind(0)
    axis, freq = (torch.from_numpy(t) for t in bsa.bsa_rope_table(m.rope))
    for pos in (None, torch.randint(0, 50, (2, B, L))):
        p = torch.arange(L).expand(2, B, L) if pos is None else pos
        t = (p[axis.long()].permute(1, 2, 0) * freq)[:, None]
        turned = [torch.cat((u[..., :20] * t.cos() - u[..., 20:40] * t.sin(), u[..., :20] * t.sin() + u[..., 20:40] * t.cos(),
                             u[..., 40:]), -1) for u in (q, k)]
        want = m.proj((torch.softmax(turned[0] @ turned[1].transpose(-1, -2) / 8, -1) @ v).transpose(1, 2).reshape(B, L, 128))
        got = m(x, positions=pos)
        assert torch.allclose(got, want, atol=1e-12)
        g = torch.randn_like(got)
        a, b = (torch.autograd.grad(o, (x, m.qkv.weight), g, retain_graph=True) for o in (got, want))
        assert all(torch.allclose(u, w, atol=1e-11) for u, w in zip(a, b))
    assert seen["positions"].shape == (2, B, L)


def _blocks(**kw):
    torch.manual_seed(3)
    made = [LY.BigBirdBlock(256, 4, window=1, num_global=1, num_random=1, rope=(8, 12, 12), branch_scale=0.5, **kw)
            for _ in range(2)]
    for m in made:
        m.to("cuda")
        m.attention.to(torch.bfloat16)
        with torch.no_grad():
            for p in (m.pre_weight, m.post_weight, m.gate):
                p.add_(0.2 * torch.randn_like(p))
    return made


@gpu
@needs_cuda
@pytest.mark.parametrize("kw", [dict(fp8=True), dict(fused=True), dict(pre="layer", post="layer"),
                                dict(fp8=True, pre="layer")])
def test_stack_of_blocks(kw):
    from block_sparse_attention_bigbird_b200 import block_norm
    first, second = _blocks(**kw)
    B, L = 2, 192
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(B, L, 256, generator=g, device="cuda").bfloat16().requires_grad_()
    pos = torch.randint(0, 300, (3, B, L), generator=g, device="cuda")
    mask = torch.ones(B, L, dtype=torch.uint8, device="cuda")
    mask[1, 150:] = 0
    gate = torch.rand(B, 256, generator=g, device="cuda").requires_grad_()
    stream, normed = first(x, key_mask=mask, positions=pos, gate=gate, following=second)
    out = second(stream, key_mask=mask, positions=pos, normed=normed)
    assert bsa.bsa_sync_status() == 0
    dout = torch.randn(B, L, 256, generator=g, device="cuda").bfloat16()
    leaves = [x, gate] + [p for m in (first, second) for p in m.parameters() if p is not first.gate]
    grads = torch.autograd.grad(out, leaves, dout)
    assert bsa.bsa_sync_status() == 0
    # the same calls one by one: the border's norm from the rounded stream instead
    h = x
    for m, gt in ((first, gate), (second, None)):
        _, n = block_norm(h, pre=m.pre, pre_weight=m.pre_weight, pre_bias=m.pre_bias, eps=m.eps)
        y = m.attention(n, key_mask=mask, positions=pos)
        h, _ = block_norm(h, y, post=m.post, post_weight=m.post_weight, post_bias=m.post_bias,
                          gate=m.gate if gt is None else gt, branch_scale=m.branch_scale, pre=None, eps=m.eps)
    again = torch.autograd.grad(h, leaves, dout)
    scale = lambda t: t.float().norm() / t.numel() ** 0.5  # noqa: E731
    # the border's norm of the rounded stream moves its input by half a bf16 step (2^-9 rms), 8-bit
    # codes of it by up to a step of theirs (2^-3 each, independent): 5 % of the sums they enter
    for a, b in zip((out, *grads), (h, *again)):
        assert a.shape == b.shape and a.isfinite().all()
        assert (a.float() - b.float()).norm() <= 0.05 * max(b.float().norm(), 1e-6), a.shape
    assert (out.float() - h.float()).norm() <= 0.02 * scale(h) * h.numel() ** 0.5
    # a repeat is bit-identical
    stream2, normed2 = first(x, key_mask=mask, positions=pos, gate=gate, following=second)
    assert torch.equal(second(stream2, key_mask=mask, positions=pos, normed=normed2), out)


def _dense(m, x, lay, pos, mask, gate):
    """BigBirdBlock in plain torch, fp32 throughout."""
    def norm(t, kind, w, b):
        t = t - t.mean(-1, keepdim=True) if kind == "layer" else t
        t = t * (t.square().mean(-1, keepdim=True) + m.eps).rsqrt() * w
        return t if b is None else t + b
    B, L, C = x.shape
    H = C // 64
    a = m.attention
    f = lambda t: None if t is None else t.float()  # noqa: E731
    h = norm(x, m.pre, m.pre_weight, m.pre_bias)
    q, k, v = torch.nn.functional.linear(h, f(a.qkv.weight), f(a.qkv.bias)).view(B, L, 3, H, 64).permute(2, 0, 3, 1, 4)
    axis, freq = (torch.from_numpy(t).cuda() for t in bsa.bsa_rope_table(a.rope))
    t = (pos.double()[axis.long()].permute(1, 2, 0) * freq)[:, None].float()
    n = len(axis)
    q, k = (torch.cat((u[..., :n] * t.cos() - u[..., n:] * t.sin(), u[..., :n] * t.sin() + u[..., n:] * t.cos()), -1)
            for u in (q, k))
    rp, ci = bsa.bsa_layout_csr(lay)
    allowed = torch.zeros(H, L // 64, L // 64, dtype=torch.bool)
    for r in range(H * (L // 64)):
        allowed[r // (L // 64), r % (L // 64), ci[rp[r]:rp[r + 1]]] = True
    allowed = allowed.repeat_interleave(64, 1).repeat_interleave(64, 2).cuda() & (mask != 0)[:, None, None]
    o = torch.softmax((q @ k.transpose(-1, -2) / 8).masked_fill(~allowed, -np.inf), -1) @ v
    y = torch.nn.functional.linear(o.transpose(1, 2).reshape(B, L, C), f(a.proj.weight), f(a.proj.bias))
    return m.stream_scale * x + m.branch_scale * gate[:, None] * norm(y, m.post, m.post_weight, m.post_bias)


@gpu
@needs_cuda
@pytest.mark.parametrize("kw,bound", [(dict(fused=True), 0.03), (dict(pre="layer", post="layer"), 0.03),
                                      (dict(fp8=True), 0.12)])
def test_block_against_dense_fp32(kw, bound):
    # bf16 between the steps errs by 2^-9 a rounding, some ten of them in a row and each seen by
    # both operands of the products after it: 3 %.  8-bit operands err by 2^-4 / sqrt(3) of their
    # value (uniform over a step of relative size up to 2^-3), 3.6 % each and twice that from both,
    # in two projections and again in their gradients' products: 12 %.
    m, _ = _blocks(**kw)
    B, L = 2, 192
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(B, L, 256, generator=g, device="cuda").bfloat16().requires_grad_()
    pos = torch.randint(0, 300, (3, B, L), generator=g, device="cuda")
    mask = torch.ones(B, L, dtype=torch.uint8, device="cuda")
    mask[0, 100:] = 0
    gate = torch.rand(B, 256, generator=g, device="cuda").requires_grad_()
    dout = torch.randn(B, L, 256, generator=g, device="cuda").bfloat16()
    leaves = [x, gate, m.pre_weight, m.post_weight, m.attention.qkv.weight, m.attention.proj.weight]
    out = m(x, key_mask=mask, positions=pos, gate=gate)
    grads = torch.autograd.grad(out, leaves, dout)
    xf = x.detach().float().requires_grad_()
    ref = _dense(m, xf, m.attention.layout(L, x.device), pos, mask, gate)
    want = torch.autograd.grad(ref, [xf] + leaves[1:], dout.float())
    for a, b in zip((out, *grads), (ref, *want)):
        assert (a.float() - b.float()).norm() <= bound * b.float().norm(), a.shape


@gpu
@needs_cuda
def test_a_captured_step_replays_with_new_inputs():
    m, _ = _blocks(fp8=True)
    B, L = 2, 192
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(B, L, 256, generator=g, device="cuda").bfloat16().requires_grad_()
    pos = torch.randint(0, 300, (3, B, L), generator=g, device="cuda")
    dout = torch.randn(B, L, 256, generator=g, device="cuda").bfloat16()
    leaves = [x] + list(m.parameters())

    def step():
        out = m(x, positions=pos)
        return [t.detach() for t in (out, *torch.autograd.grad(out, leaves, dout))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # layouts are built and uploaded on first use
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (5, 6):
        with torch.no_grad():
            x.copy_(torch.randn(x.shape, generator=g.manual_seed(seed), device="cuda"))
        pos.random_(0, 1000, generator=g)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
    assert bsa.bsa_sync_status() == 0
