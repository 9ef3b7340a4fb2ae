"""torch autograd wrapper of the scan.

Mirrors the autodiff node of burn-mamba ``mamba3/quat_scan/backward.rs``
(``impl Mamba3QuatScanBackendExt for Autodiff``, ``quat_cumprod``, and the
``QuatScanBackward`` node with its ``State``): the forward runs the scan; when
gradients are tracked it keeps only the leaves ``q`` and ``init``, and the
backward recomputes from them (``quat_cumprod_bwd``).  Untracked calls keep
nothing.

``save_carries=True`` keeps the chunk carries as well (1/64 of ``q``): the
forward writes them (``quat_cumprod_fwd_carries``) and the backward starts
from them (``quat_cumprod_bwd_carries``) instead of recomputing the forward.
The page keeps only the leaves on purpose; this is the measured alternative.

``quat_cumprod_recalculated`` also returns the final carry ``cum[:, -1]`` as a
slice of ``cum``.  As in the page's module documentation, its cotangent then
reaches the node already added into ``d_cum[:, S-1]``; the node itself has a
single output.

``quat_norm_rotate`` and ``quat_delta`` are the differentiable forms of the
operators around the scan (:mod:`.mixer`).  Their gradients have none of their own: a
backward through them (``create_graph=True``) raises.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (
    quat_cumprod_bwd, quat_cumprod_bwd_carries, quat_cumprod_fwd, quat_cumprod_fwd_carries, quat_delta_bwd,
    quat_delta_fwd, quat_delta_fwd_carries, quat_norm_rotate_bwd, quat_norm_rotate_fwd)

__all__ = ["QuatCumprod", "quat_cumprod", "quat_cumprod_recalculated", "QuatNormRotate", "quat_norm_rotate",
           "QuatDelta", "quat_delta"]


class QuatCumprod(torch.autograd.Function):
    """``cum = quat_cumprod(q, init)``: forward and recompute backward in the CUDA library."""

    @staticmethod
    def forward(ctx, q, init, save_carries: bool, tracked: bool):
        # (Gradient mode is off inside forward: `tracked` is decided by the caller.)
        q = q.contiguous()
        init = init.contiguous()
        ctx.save_carries = bool(save_carries) and tracked
        if ctx.save_carries:
            cum, carries = quat_cumprod_fwd_carries(q, init)
            ctx.save_for_backward(q, carries)
        else:
            cum = quat_cumprod_fwd(q, init)
            if tracked:
                ctx.save_for_backward(q, init)
        return cum

    @staticmethod
    def backward(ctx, d_cum):
        d_cum = d_cum.contiguous()
        if ctx.save_carries:
            q, carries = ctx.saved_tensors
            d_q, d_init = quat_cumprod_bwd_carries(q, carries, d_cum)
        else:
            q, init = ctx.saved_tensors
            d_q, d_init = quat_cumprod_bwd(q, init, d_cum)
        return (d_q if ctx.needs_input_grad[0] else None,
                d_init if ctx.needs_input_grad[1] else None,
                None, None)


def quat_cumprod(q, init, *, save_carries: bool = False):
    """Differentiable scan: ``q`` [B,S,H,J,4] and ``init`` [B,H,J,4] fp32 CUDA -> ``cum``."""
    tracked = torch.is_grad_enabled() and (q.requires_grad or init.requires_grad)
    return QuatCumprod.apply(q, init, save_carries, tracked)


def quat_cumprod_recalculated(q, init, *, save_carries: bool = False):
    """``(cum, final_carry)`` with ``final_carry = cum[:, -1]`` (a slice of ``cum``)."""
    cum = quat_cumprod(q, init, save_carries=save_carries)
    return cum, cum[:, -1]


class QuatNormRotate(torch.autograd.Function):
    """Norm and rotation of queries and keys; the backward recomputes from the inputs."""

    @staticmethod
    def forward(ctx, q, k, cum, w_q, w_k, norm, eps):
        cum = cum.contiguous()
        ctx.norm, ctx.eps = norm, eps
        ctx.save_for_backward(q, k, cum, w_q, w_k)
        return quat_norm_rotate_fwd(q, k, cum, w_q, w_k, norm=norm, eps=eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_q_out, d_k_out):
        q, k, cum, w_q, w_k = ctx.saved_tensors
        d = quat_norm_rotate_bwd(q, k, cum, d_q_out.contiguous(), d_k_out.contiguous(), w_q, w_k,
                                 norm=ctx.norm, eps=ctx.eps)
        return (*[g if need else None for g, need in zip(d, ctx.needs_input_grad)], None, None)


def quat_norm_rotate(q, k, cum, w_q=None, w_k=None, *, norm="rms", eps=1e-6):
    """Differentiable :func:`quat_norm_rotate_fwd`: ``(q_out, k_out)``."""
    return QuatNormRotate.apply(q, k, cum, w_q, w_k, norm, eps)


def _own_rows(t):
    """``t``, or a contiguous copy of an expanded bfloat16 view (whose gradient autograd sums up)."""
    flat = t.dtype is torch.bfloat16 and any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride()))
    return t.contiguous() if flat else t


class QuatDelta(torch.autograd.Function):
    """Gated delta rule over whole sequences; tracked calls keep the carries and the errors."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, init, scale, offsets, tracked):
        g, beta = g.contiguous(), beta.contiguous()
        ctx.scale = scale
        ctx.set_materialize_grads(False)   # a cotangent that nobody has is None: no zeros are made and read for it
        if not tracked:
            return quat_delta_fwd(q, k, v, g, beta, init, scale=scale, offsets=offsets)
        o, final, carries, errors = quat_delta_fwd_carries(q, k, v, g, beta, init, scale=scale, offsets=offsets)
        ctx.save_for_backward(q, k, v, g, beta, carries, errors, offsets)
        return o, final

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o, d_final):
        *inputs, offsets = ctx.saved_tensors
        v = inputs[2]
        d_o = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if d_o is None else d_o.contiguous()
        d_final = None if d_final is None else d_final.contiguous()
        d = quat_delta_bwd(*inputs, d_o, d_final, scale=ctx.scale, offsets=offsets)
        return (*[g if need else None for g, need in zip(d, ctx.needs_input_grad)], None, None, None)


def quat_delta(q, k, v, g, beta, init=None, *, scale=None, offsets=None):
    """Differentiable :func:`quat_delta_fwd`: ``(o, final_state)``.  Expanded bfloat16 inputs are copied."""
    q, k, v = (_own_rows(t) for t in (q, k, v))
    inputs = [t for t in (q, k, v, g, beta, init) if t is not None]
    tracked = torch.is_grad_enabled() and any(t.requires_grad for t in inputs)
    init = None if init is None else init.contiguous()
    return QuatDelta.apply(q, k, v, g, beta, init, scale, offsets, tracked)
