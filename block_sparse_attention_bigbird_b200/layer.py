"""BigBird self-attention layer: QKV projection, block-sparse attention, output
projection; and the block around it, with its norms, gate and residual.

The layer the pages build around the attention: one linear map of the hidden
states to q, k, v ("BigBird 稀疏注意力机制解析", 代码实现: ``self.qkv =
nn.Linear(dim, dim * 3)``, split into heads), the attention over the BigBird
layout, and an output projection ("BERT 稀疏注意力机制入门指南", PyTorch 实现:
``self.proj = nn.Linear(dim, dim)``).  The two projections are plain dense GEMMs
(torch, i.e. cuBLAS) by default; the attention and its gradients are the
library's kernels through ``block_sparse_attention``.

With ``fused=True`` (bf16 on an sm_100 device) the forward runs the library's
own projection kernels instead, with the head split and merge inside them:
``bsa_qkv_projection`` writes q, k and v straight into the attention's
[B, H, L, 64] layout, and ``bsa_out_projection`` reads the attention output in
that layout through its tile loads.  So the layer's forward is three library
kernels (four with the split-row merge) and no transposes.  The projections'
gradients are plain GEMMs in torch.

With ``fp8=True`` both projections and their gradients run in 8-bit floating point
(``fp8_linear``).  With ``rope`` the heads of q and k are turned by rotary positions of one
or more axes (``rotary``), which reads them from the packed projection output and writes the
attention's layout.

``BigBirdBlock`` puts the layer between a norm before it and a norm, gate and residual after
it (``block_norm``); given the block that follows, it takes that block's first norm in the
same pass.
"""

from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import bsa
from .autograd import block_norm, block_sparse_attention, fp8_linear, rotary


class _QKVProjection(torch.autograd.Function):
    """q, k, v = heads of x W^T + b by the library kernel; gradients by torch GEMMs."""

    @staticmethod
    def forward(ctx, x, weight, bias, num_heads):
        x, weight = x.contiguous(), weight.contiguous()
        q, k, v = bsa.bsa_qkv_projection(x, weight, bias.contiguous() if bias is not None else None, num_heads)
        ctx.save_for_backward(x, weight)
        ctx.has_bias = bias is not None
        return q, k, v

    @staticmethod
    def backward(ctx, dq, dk, dv):
        x, weight = ctx.saved_tensors
        B, L, C = x.shape
        H = C // 64
        grads = [torch.zeros((B, H, L, 64), dtype=x.dtype, device=x.device) if g is None else g
                 for g in (dq, dk, dv)]
        # the projection's output gradient [B, L, 3C]: the heads merged back in q, k, v order
        dy = torch.stack(grads, 0).permute(1, 3, 0, 2, 4).reshape(B, L, 3 * C)
        dx = dy @ weight
        dw = dy.reshape(-1, 3 * C).t() @ x.reshape(-1, C)
        db = dy.sum((0, 1)) if ctx.has_bias else None
        return dx, dw, db, None


class _OutProjection(torch.autograd.Function):
    """y = merge_heads(o) W^T + b by the library kernel; gradients by torch GEMMs."""

    @staticmethod
    def forward(ctx, o, weight, bias):
        o, weight = o.contiguous(), weight.contiguous()
        y = bsa.bsa_out_projection(o, weight, bias.contiguous() if bias is not None else None)
        ctx.save_for_backward(o, weight)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        o, weight = ctx.saved_tensors
        B, H, L, d = o.shape
        N = weight.shape[0]
        dy = dy.contiguous()
        do = (dy @ weight).view(B, L, H, d).permute(0, 2, 1, 3).contiguous()
        dw = dy.reshape(-1, N).t() @ o.permute(0, 2, 1, 3).reshape(-1, H * d)
        db = dy.sum((0, 1)) if ctx.has_bias else None
        return do, dw, db


class BigBirdSelfAttention(torch.nn.Module):
    """x [B, L, dim] -> [B, L, dim] with ``num_heads`` heads of 64.

    block (a multiple of 64), window, num_global, num_random and seed define the
    BigBird layout of each sequence length (see bsa_layout_build); it is built
    and uploaded on first use per (length, device).  ``key_mask`` in forward is
    uint8 [B, L], 1 = keep.  ``fused``: run the projections with the library's
    kernels (bf16 CUDA inputs and parameters only).  ``fp8``: run them and their gradients in
    8-bit floating point (bf16 CUDA inputs).  ``rope``: pairs of a head turned by each position
    axis (see bsa_rope_build; ``rope_base``, ``rope_per_axis`` and ``rope_interleave`` as there);
    ``positions`` in forward is then [axes, L] or [axes, B, L], by default 0 .. L - 1 on every
    axis.
    """

    HEAD_DIM = 64

    def __init__(self, dim: int, num_heads: int, window: int = 1, num_global: int = 2, num_random: int = 3,
                 seed: int = 0, bias: bool = True, out_proj: bool = True, block: int = 64, fused: bool = False,
                 fp8: bool = False, rope=None, rope_base: float = 10000.0, rope_per_axis: bool = False,
                 rope_interleave: bool = False):
        super().__init__()
        if dim != num_heads * self.HEAD_DIM:
            raise ValueError(f"dim must be num_heads * {self.HEAD_DIM}")
        if block < 64 or block % 64:
            raise ValueError("block must be a multiple of 64")
        if fused and fp8:
            raise ValueError("fused and fp8 are two ways to run the projections")
        self.num_heads, self.block, self.fused, self.fp8 = num_heads, block, fused, fp8
        self.rope = None
        if rope is not None:
            self.rope = bsa.bsa_rope_build(rope, rope_base, per_axis=rope_per_axis, interleave=rope_interleave)
            if 2 * self.rope.n_pairs > self.HEAD_DIM:
                raise ValueError(f"rope turns at most {self.HEAD_DIM // 2} pairs of a head")
        self.window, self.num_global, self.num_random, self.seed = window, num_global, num_random, seed
        self.qkv = torch.nn.Linear(dim, 3 * dim, bias=bias)
        self.proj = torch.nn.Linear(dim, dim, bias=bias) if out_proj else None
        self._layouts = {}

    def layout(self, L: int, device: torch.device) -> "bsa.Layout":
        key = (L, str(device))
        lay = self._layouts.get(key)
        if lay is None:
            lay = bsa.bsa_layout_build(self.num_heads, L, self.block, self.window, self.num_global,
                                       self.num_random, self.seed)
            with torch.cuda.device(device.index) if device.type == "cuda" else contextlib.nullcontext():
                bsa.bsa_layout_upload(lay)
            self._layouts[key] = lay
        return lay

    def __getstate__(self):  # copied and stored without the layouts, which are built again on first use
        return {**self.__dict__, "_layouts": {}}

    def _turn(self, q, k, positions):
        if positions is None:
            positions = torch.arange(q.shape[2], device=q.device).expand(self.rope.n_axes, -1)
        return rotary(q, k, positions, self.rope)

    def forward(self, x: torch.Tensor, key_mask: Optional[torch.Tensor] = None,
                positions: Optional[torch.Tensor] = None) -> torch.Tensor:
        B, L, C = x.shape
        H, d = self.num_heads, self.HEAD_DIM
        if positions is not None and self.rope is None:
            raise ValueError("positions without rope")
        if self.fused:
            if x.dtype != torch.bfloat16 or not x.is_cuda or self.qkv.weight.dtype != torch.bfloat16:
                raise ValueError("the fused layer takes bf16 CUDA inputs and parameters")
            q, k, v = _QKVProjection.apply(x, self.qkv.weight, self.qkv.bias, H)
            if self.rope is not None:
                q, k = self._turn(q, k, positions)
            o = block_sparse_attention(q, k, v, self.layout(L, x.device), key_mask=key_mask)
            if self.proj is None:
                return o.transpose(1, 2).reshape(B, L, C)
            return _OutProjection.apply(o, self.proj.weight, self.proj.bias)
        if self.fp8 and (x.dtype != torch.bfloat16 or not x.is_cuda):
            raise ValueError("the fp8 layer takes bf16 CUDA inputs")
        linear = (lambda t, m: fp8_linear(t, m.weight, m.bias)) if self.fp8 else (lambda t, m: m(t))
        # [B, L, 3C] -> three [B, H, L, d] contiguous tensors
        q, k, v = linear(x, self.qkv).view(B, L, 3, H, d).permute(2, 0, 3, 1, 4).unbind(0)
        if self.rope is not None:
            q, k = self._turn(q, k, positions)
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        o = block_sparse_attention(q, k, v, self.layout(L, x.device), key_mask=key_mask)
        o = o.transpose(1, 2).reshape(B, L, C)
        return linear(o, self.proj) if self.proj is not None else o


class BigBirdBlock(torch.nn.Module):
    """x -> stream_scale x + branch_scale gate N_post(attention(N_pre(x))).

    ``pre`` and ``post`` are "rms", "layer" or (``post``) None; layer norms have biases.  gate: a
    learned gate [dim], or False for none; a call may give its own, [dim] or [B, dim].  The other
    arguments are BigBirdSelfAttention's.

    The stream x is bf16.  The parameters of the norm before the attention are of one type, x's or
    fp32, and so are those of the norm after it, the gate and the following block's first norm.
    The projections' parameters are bf16, or of any type that fp8_linear takes with ``fp8`` (under
    autocast, of any that it casts).
    """

    def __init__(self, dim: int, num_heads: int, pre: str = "rms", post: Optional[str] = "rms", gate: bool = True,
                 branch_scale: float = 1.0, stream_scale: float = 1.0, eps: float = 1e-6, **attention):
        super().__init__()
        if pre not in ("rms", "layer") or post not in ("rms", "layer", None):
            raise ValueError('pre must be "rms" or "layer", post one of them or None')
        self.attention = BigBirdSelfAttention(dim, num_heads, **attention)
        self.pre, self.post, self.eps = pre, post, eps
        self.branch_scale, self.stream_scale = branch_scale, stream_scale
        one, zero = lambda: torch.nn.Parameter(torch.ones(dim)), lambda: torch.nn.Parameter(torch.zeros(dim))
        self.pre_weight, self.pre_bias = one(), zero() if pre == "layer" else None
        self.post_weight = one() if post is not None else None
        self.post_bias = zero() if post == "layer" else None
        self.gate = one() if gate else None

    def _check_types(self, x, gate, normed, following):
        """Refuses parameters that one of the steps below would, before the first runs."""
        layer = self.attention
        linear = [m for m in (layer.qkv, layer.proj) if type(m) is torch.nn.Linear]
        if layer.fused and any(m.weight.dtype != torch.bfloat16 for m in linear):
            raise ValueError("the fused projections take bf16 parameters")
        if not (layer.fused or layer.fp8 or torch.is_autocast_enabled(x.device.type)) and \
                any(m.weight.dtype != x.dtype for m in linear):
            raise ValueError("without fp8 or autocast the projections' parameters must be of the stream's type")
        after = [self.post_weight, self.post_bias, gate]
        if following is not None:
            after += [following.pre_weight, following.pre_bias]
        for params in ([self.pre_weight, self.pre_bias] if normed is None else [], after):
            types = {p.dtype for p in params if p is not None}
            if len(types) > 1 or not types <= {x.dtype, torch.float32}:
                raise ValueError("the norm parameters and gate of one pass must be all of the stream's type or all fp32")

    def forward(self, x: torch.Tensor, key_mask: Optional[torch.Tensor] = None,
                positions: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                normed: Optional[torch.Tensor] = None, following: Optional["BigBirdBlock"] = None):
        """The stream after the block; with ``following`` (stream, its normed input), to be passed
        to that block as ``normed`` (its eps must be this block's).  x: contiguous [B, L, dim].
        """
        if following is not None and following.eps != self.eps:
            raise ValueError("one pass takes both norms with one eps: the following block has another")
        gate = self.gate if gate is None else gate
        self._check_types(x, gate, normed, following)
        if normed is None:
            _, normed = block_norm(x, pre=self.pre, pre_weight=self.pre_weight, pre_bias=self.pre_bias, eps=self.eps)
        y = self.attention(normed, key_mask=key_mask, positions=positions)
        nxt = {"pre": None} if following is None else {"pre": following.pre, "pre_weight": following.pre_weight,
                                                      "pre_bias": following.pre_bias}
        stream, after = block_norm(x, y.contiguous(), post=self.post, post_weight=self.post_weight,
                                   post_bias=self.post_bias, gate=gate,
                                   branch_scale=self.branch_scale, stream_scale=self.stream_scale, eps=self.eps,
                                   **nxt)
        return stream if following is None else (stream, after)
