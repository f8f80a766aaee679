"""Autograd bindings of the fused Q+K rotation, alone and with the norm of queries and keys.

"How Unsloth Optimizes RoPE Embedding Computations in Triton Kernels",
Autograd Function Wrappers and Frequently Asked Questions: the rotation sits
in a ``torch.autograd.Function`` whose forward keeps the constants it needs
and whose backward runs the same kernel with the backward flag.  The
rotation is orthogonal, so the gradient of y = R(t) x is R(-t) applied to
dy; the pass-through tail and unrotated tokens pass their gradient through.

Here the forward is out of place (autograd keeps the inputs intact) and the
backward writes fresh gradient tensors; both are single launches of the
CUDA library.

``norm_rotary_qk`` is the same for ``norm_rotate_qk``, with gradients of both
weights; its node is csrc/serving_binding.cpp's.  Its backward reads the inputs
again: only they are kept.
"""
from __future__ import annotations

import torch

import rotary_position_embedding_rope_gb300 as _package

from . import rotate_qk


class RotaryQK(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, cos, sin, pos_idx, rotary_dim, layout, seq_before_head):
        q_out, k_out = rotate_qk(q.contiguous(), None if k is None else k.contiguous(), cos, sin,
                                 pos_idx, rotary_dim, layout, seq_before_head, backward=False)
        ctx.save_for_backward(cos, sin, pos_idx)
        ctx.cfg = (rotary_dim, layout, seq_before_head, k is not None)
        return q_out, k_out

    @staticmethod
    def backward(ctx, grad_q, grad_k):
        cos, sin, pos_idx = ctx.saved_tensors
        rotary_dim, layout, seq_before_head, has_k = ctx.cfg
        # an output that took no part in the loss arrives as None: rotate only the given ones
        gq = grad_q.contiguous() if grad_q is not None else None
        gk = grad_k.contiguous() if (has_k and grad_k is not None) else None
        dq = dk = None
        if gq is not None and gk is not None:
            dq, dk = rotate_qk(gq, gk, cos, sin, pos_idx, rotary_dim, layout, seq_before_head,
                               backward=True)
        elif gq is not None:
            dq, _ = rotate_qk(gq, None, cos, sin, pos_idx, rotary_dim, layout, seq_before_head,
                              backward=True)
        elif gk is not None:
            dk, _ = rotate_qk(gk, None, cos, sin, pos_idx, rotary_dim, layout, seq_before_head,
                              backward=True)
        return dq, dk, None, None, None, None, None, None


def rotary_qk(q: torch.Tensor, k: torch.Tensor | None, cos: torch.Tensor, sin: torch.Tensor,
              pos_idx: torch.Tensor | None = None, rotary_dim: int | None = None,
              layout: str = "split_half", seq_before_head: bool = False):
    """Differentiable fused rotation of q and k (k may be None): returns (q_rot, k_rot)."""
    rd = 2 * cos.shape[1] if rotary_dim is None else rotary_dim
    return RotaryQK.apply(q, k, cos, sin, pos_idx, rd, layout, seq_before_head)


def norm_rotary_qk(q: torch.Tensor | None, k: torch.Tensor | None, wq: torch.Tensor | None,
                   wk: torch.Tensor | None, cos: torch.Tensor, sin: torch.Tensor, eps: float = 1e-6,
                   pos_idx: torch.Tensor | None = None, rotary_dim: int | None = None,
                   layout: str = "split_half", seq_before_head: bool = False):
    """Differentiable norm and rotation of q and k (either may be None): (q_out, k_out), with
    gradients of q, k, wq and wk.  Arguments as ``norm_rotate_qk``; here q, k and weights whose
    strides or alignment that call does not take are copied.

    While a CUDA graph is captured, no other graph of the same leaves made on another
    stream may be alive (drop the outputs of eager calls first): the call refuses, because
    the captured backward pass could not run."""
    o = (_package._serving or _package._native()).norm_rotary_qk(
        q, k, wq, wk, cos, sin, eps, pos_idx, rotary_dim, _package._LAYOUT_CODE[layout], seq_before_head)
    if type(o) is int:
        raise _package.RopeError(o, "rope_norm_qk_fwd")
    return o
