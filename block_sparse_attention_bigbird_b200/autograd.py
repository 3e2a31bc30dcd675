"""torch.autograd bindings of the block-sparse attention and of the operators around it.

``block_sparse_attention(q, k, v, layout)`` runs bsa_forward and records a node
whose backward runs bsa_backward, so the kernels take part in an ordinary
training step (the pages train BigBird-style models: "BERT 稀疏注意力机制入门指南",
生产环境部署建议; "BigBird 稀疏注意力机制解析", 避坑指南).  It is argument
marshalling only: both directions are the library's kernels.  ``rotary``, ``block_norm`` and
``fp8_linear`` do the same for rotary positions, a block's norms and residual, and linear
layers in 8-bit floating point.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import bsa


class _BlockSparseAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, layout, key_mask, scale):
        out, lse = bsa.bsa_forward(q, k, v, layout, key_mask=key_mask, scale=scale)
        ctx.save_for_backward(q, k, v, out, lse, key_mask)
        ctx.layout = layout
        ctx.scale = scale
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    def backward(ctx, dout, _dlse):
        q, k, v, out, lse, key_mask = ctx.saved_tensors
        dq, dk, dv = bsa.bsa_backward(q, k, v, out, dout.contiguous(), lse, ctx.layout, key_mask=key_mask,
                                      scale=ctx.scale)
        return dq, dk, dv, None, None, None


def block_sparse_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, layout: "bsa.Layout",
                           key_mask: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                           return_lse: bool = False):
    """O = softmax(q k^T * scale restricted to the layout) v, differentiable in q, k, v.

    q, k, v: contiguous bf16 CUDA tensors [B, H, L, 64]; layout: an uploaded
    bsa.Layout for this H and L; key_mask: optional uint8 [B, L] (1 = keep);
    scale: None for 1/sqrt(64).  Returns O (bf16), and lse (fp32 [B, H, L], not
    differentiable) when ``return_lse``.
    """
    out, lse = _BlockSparseAttention.apply(q, k, v, layout, key_mask, scale)
    return (out, lse) if return_lse else out


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, rope):
        ctx.save_for_backward(positions)
        ctx.rope = rope
        ctx.set_materialize_grads(False)
        q, k = bsa.bsa_rope_apply(q, k, positions, rope)
        return (q, k) if k is not None else q

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk=None):
        (positions,) = ctx.saved_tensors
        grads = [None if g is None else g if g.shape[3] == 1 or g.stride(3) == 1 else g.contiguous() for g in (dq, dk)]
        first, second = grads if grads[0] is not None else (grads[1], None)
        if first is None:
            return None, None, None, None
        a, b = bsa.bsa_rope_apply(first, second, positions, ctx.rope, inverse=True)
        return (a, b, None, None) if grads[0] is not None else (None, a, None, None)


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, rope: "bsa.Rope"):
    """(q, k) with rotary positions (see bsa.bsa_rope_apply), differentiable in q and k.  Positions
    have no gradient: those that want one are refused."""
    if positions.requires_grad and torch.is_grad_enabled():
        raise ValueError("positions have no gradient: detach them")
    got = _Rotary.apply(q, k, positions, rope)
    return got if k is not None else (got, None)


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, post_weight, post_bias, gate, pre_weight, pre_bias, post, pre, branch_scale, stream_scale,
                eps, grads):
        stream, normed, stats = bsa.bsa_block_norm(
            x, y, post=post, post_weight=post_weight, post_bias=post_bias, gate=gate, branch_scale=branch_scale,
            stream_scale=stream_scale, pre=pre, pre_weight=pre_weight, pre_bias=pre_bias, eps=eps,
            save_stats=grads and any(ctx.needs_input_grad))
        ctx.save_for_backward(stream, y, stats, post_weight, post_bias, gate, pre_weight, pre_bias)
        ctx.kinds = (post, pre, branch_scale, stream_scale)
        ctx.set_materialize_grads(False)
        if y is None:
            return normed
        return (stream, normed) if pre is not None else stream

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        stream, y, stats, post_weight, post_bias, gate, pre_weight, pre_bias = ctx.saved_tensors
        post, pre, branch_scale, stream_scale = ctx.kinds
        dstream, dnormed = (None, grads[0]) if y is None else grads if pre is not None else (grads[0], None)
        if dstream is None and dnormed is None:
            return (None,) * 13
        g = bsa.bsa_block_norm_backward(
            None if dstream is None else dstream.contiguous(), None if dnormed is None else dnormed.contiguous(),
            stream, y, stats, post=post, post_weight=post_weight, post_bias=post_bias, gate=gate,
            branch_scale=branch_scale, stream_scale=stream_scale, pre=pre, pre_weight=pre_weight, pre_bias=pre_bias,
            params=any(ctx.needs_input_grad[2:7]))
        return (g["x"], g["y"], g["post_weight"], g["post_bias"], g["gate"], g["pre_weight"], g["pre_bias"],
                None, None, None, None, None, None)


def block_norm(x: torch.Tensor, y: Optional[torch.Tensor] = None, post: Optional[str] = None, post_weight=None,
               post_bias=None, gate=None, branch_scale: float = 1.0, stream_scale: float = 1.0,
               pre: Optional[str] = "rms", pre_weight=None, pre_bias=None, eps: float = 1e-6):
    """(stream, normed) of the residual after a block and the norm before the next (see
    bsa.bsa_block_norm), differentiable in x, y, the gate and the parameters.  Without y the
    stream is x; with pre None normed is None.
    """
    # inside a Function gradients are always off, so whether any are wanted is asked here
    got = _BlockNorm.apply(x, y, post_weight, post_bias, gate, pre_weight, pre_bias, post, pre, branch_scale,
                           stream_scale, eps, torch.is_grad_enabled())
    if y is None:
        return x, got
    return got if pre is not None else (got, None)


class _Fp8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, grad_dtype, grads):
        rows = x.reshape(-1, x.shape[-1]).contiguous()
        need_x, need_w = (grads and need for need in ctx.needs_input_grad[:2])
        xs = bsa.bsa_fp8_quantize(rows, cols=need_w)
        ws = bsa.bsa_fp8_quantize(weight.contiguous(), square=True, cols=need_x)
        y = bsa.bsa_fp8_matmul(xs[0], xs[1], ws[0], ws[1], bias=bias, out_dtype=x.dtype)
        ctx.save_for_backward(*(xs[2:] if need_w else (None, None)), *(ws[2:] if need_x else (None, None)))
        ctx.about = (x.shape, x.dtype, weight.shape, weight.dtype, None if bias is None else bias.dtype, grad_dtype)
        return y.view(*x.shape[:-1], weight.shape[0])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        xt, xt_scale, wt, wt_scale = ctx.saved_tensors
        x_shape, x_dtype, w_shape, w_dtype, b_dtype, grad_dtype = ctx.about
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        dy = dy.reshape(-1, w_shape[0]).contiguous()
        dx = dw = db = None
        if need_x or need_w:
            q = bsa.bsa_fp8_quantize(dy, rows=need_x, cols=need_w, dtype=grad_dtype)
        if need_x:
            dx = bsa.bsa_fp8_matmul(q[0], q[1], wt, wt_scale, out_dtype=x_dtype).view(x_shape)
        if need_w:
            wide = w_dtype if w_dtype in (torch.bfloat16, torch.float32) else torch.float32
            if dy.shape[0] == 0:  # no rows: nothing to sum over
                dw = dy.new_zeros(w_shape, dtype=w_dtype)
            else:
                dw = bsa.bsa_fp8_matmul(q[-2], q[-1], xt, xt_scale, out_dtype=wide).to(w_dtype)
        if need_b:
            db = dy.sum(0, dtype=torch.float32).to(b_dtype)
        return dx, dw, db, None, None


def fp8_linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               grad_dtype: torch.dtype = torch.float8_e4m3fn):
    """x weight^T + bias with the three products of a linear layer in 8-bit floating point.

    x: bf16 or fp32 [.., K] (the result's type); weight: bf16, fp16 or fp32 [N, K]; bias: bf16
    or fp32 [N].  x is quantised with a scale for each row's 128 columns, the weight for each
    128 x 128, both to e4m3; the backward quantises the gradient to ``grad_dtype`` along its
    columns for x's gradient and along its rows for the weight's, whose other operand is x
    quantised along its rows (bsa.bsa_fp8_quantize, bsa.bsa_fp8_matmul).  Differentiable in x,
    weight and bias (the bias's gradient is torch's sum over rows).  The weight is quantised in
    every call: who multiplies many times by one weight keeps its codes and calls
    bsa.bsa_fp8_matmul (4 x 8192 x 8192: 17 us, 61 with the quantisers).
    """
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x must be bf16 or fp32")
    if weight.dim() != 2 or weight.numel() == 0 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x must be [.., K] and weight [N, K], N and K at least 1")
    if grad_dtype not in (torch.float8_e4m3fn, torch.float8_e5m2, None):  # None: e4m3, as in bsa_fp8_quantize
        raise ValueError("grad_dtype must be torch.float8_e4m3fn or torch.float8_e5m2")
    # inside a Function gradients are always off, so whether any are wanted is asked here
    return _Fp8Linear.apply(x, weight, bias, grad_dtype, torch.is_grad_enabled())
