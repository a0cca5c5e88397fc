"""PyTorch autograd for the chunked SSD forward, linear attention with a decay
for each head and layer norm.

The chunked SSD forward: y, final = ssd_autograd(...)
takes part in a torch graph, and its backward is the library's ssd_backward
(the gradients of sum(dy * y) + <dfinal, final> that autograd asks for).

The forward keeps only its inputs for the backward, which rebuilds the chunk
states from them instead of storing them during the forward (the memory
trade named on llms.blog "State Space Models and Mamba ...", section
"Hardware-Aware Parallel Associative Scan").  All arithmetic runs in the
library's kernels; this module only passes tensors.
"""
from __future__ import annotations

import torch

from . import ssd


class _Ops:
    """The two computations the function calls (tests without a GPU pass the
    fp64 oracle instead)."""

    @staticmethod
    def forward(x, a, Bm, Cm, D, chunk, init):
        return ssd.forward(x, a, Bm, Cm, D, chunk, initial_state=init)

    @staticmethod
    def backward(x, a, Bm, Cm, D, dy, chunk, dfinal, init):
        return ssd.backward(x, a, Bm, Cm, D, dy, chunk, dfinal=dfinal, initial_state=init)


class SSDFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, a, Bm, Cm, D, initial_state, chunk, ops):
        y, final = ops.forward(x, a, Bm, Cm, D, chunk, initial_state)
        ctx.save_for_backward(x, a, Bm, Cm, D, initial_state)
        ctx.chunk, ctx.ops = chunk, ops
        return y, final

    @staticmethod
    def backward(ctx, dy, dfinal):
        x, a, Bm, Cm, D, init = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(x)
        g = ctx.ops.backward(x, a, Bm, Cm, D, dy.contiguous().to(x.dtype), ctx.chunk,
                             None if dfinal is None else dfinal.contiguous().to(torch.float32), init)
        return (g["dx"], g["da"], g["dBm"], g["dCm"],
                g["dD"] if D is not None and ctx.needs_input_grad[4] else None,
                g["dinit"] if init is not None and ctx.needs_input_grad[5] else None,
                None, None)


def ssd_autograd(x, a, Bm, Cm, D=None, chunk=256, initial_state=None, *, ops=None):
    """(y, final_state) of the forward as a differentiable torch operation.
    Shapes and dtypes as for ssd.forward; gradients flow to x, a, Bm, Cm, D
    and initial_state (whichever require them)."""
    return SSDFunction.apply(x, a, Bm, Cm, D, initial_state, chunk, ops or _Ops)


def _aligned(t):
    """t contiguous and on a 16-byte boundary."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _LinearOps:
    @staticmethod
    def forward(q, k, v, decay, *, scale, initial_state, cu_seqlens):
        # rows of no sequence: zero, so that what follows in a graph can take all rows
        y = None if cu_seqlens is None else q.new_zeros(q.shape[:-1] + v.shape[-1:])
        return ssd.linear_attention(q, k, v, decay, scale=scale, initial_state=initial_state, cu_seqlens=cu_seqlens,
                                    y=y)

    backward = staticmethod(ssd.linear_attention_backward)


class LinearAttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, decay, initial_state, cu_seqlens, scale, ops):
        y, final = ops.forward(q, k, v, decay, scale=scale, initial_state=initial_state, cu_seqlens=cu_seqlens)
        ctx.save_for_backward(q, k, v, decay, initial_state, cu_seqlens)
        ctx.scale, ctx.ops = scale, ops
        ctx.set_materialize_grads(False)
        return y, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dfinal):
        q, k, v, decay, init, cu = ctx.saved_tensors
        if dy is None:
            dy = q.new_zeros(q.shape[:-1] + v.shape[-1:])
        want = init is not None and ctx.needs_input_grad[4]
        g = ctx.ops.backward(q, k, v, decay, _aligned(dy), scale=ctx.scale, initial_state=init,
                             dfinal=None if dfinal is None else _aligned(dfinal), cu_seqlens=cu, want_dinit=want)
        return g["dq"], g["dk"], g["dv"], None, g["dinit"] if want else None, None, None, None


def linear_attention_autograd(q, k, v, decay, *, scale=None, initial_state=None, cu_seqlens=None, ops=None):
    """(y, final_state) of ssd.linear_attention as a differentiable torch
    operation; gradients flow to q, k, v and initial_state.  The decay is a
    constant of the layer: one that requires a gradient is refused (a learned
    log-decay per token is what ssd_autograd takes).  Rows outside every packed
    sequence are zero, in y and in the gradients."""
    if decay.requires_grad:
        raise ValueError("decay has no gradient here; use ssd_autograd for a learned decay")
    return LinearAttentionFunction.apply(q, k, v, decay, initial_state, cu_seqlens, scale, ops or _LinearOps)


class _NormOps:
    forward = staticmethod(ssd.layer_norm)
    backward = staticmethod(ssd.layer_norm_backward)


class LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, gate, groups, eps, ops):
        y, stats = ops.forward(x, weight, bias, groups=groups, gate=gate, eps=eps)
        ctx.save_for_backward(x, weight, bias, gate, stats)
        ctx.groups, ctx.ops = groups, ops
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, bias, gate, stats = ctx.saved_tensors
        need = ctx.needs_input_grad
        g = ctx.ops.backward(x, weight, bias, dy.contiguous(), stats, groups=ctx.groups, gate=gate,
                             want_dweight=weight is not None and need[1], want_dbias=bias is not None and need[2])
        return g["dx"], g["dweight"], g["dbias"], g["dgate"], None, None, None


def layer_norm_autograd(x, weight=None, bias=None, *, groups=1, gate=None, eps=1e-5, ops=None):
    """y of ssd.layer_norm as a differentiable torch operation; gradients flow
    to x, weight, bias and gate."""
    return LayerNormFunction.apply(x, weight, bias, gate, groups, eps, ops or _NormOps)
