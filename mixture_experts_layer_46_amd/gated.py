"""The gated half of the experts' feed-forward, grouped by expert (include/moe_ops.h):

    h = gated_mm(x, w_in, w_up, offsets)          SiLU(x W_in) * (x W_up); differentiable

gated_mm_grad is its gradient alone.  Checks, streams and given outputs as in ops.py.
"""
from __future__ import annotations

import torch

from .ops import _GroupedMM, _check, _dims, _given, _grad, gated_act, gated_act_grad, grouped_mm, grouped_mm_dw, grouped_mm_dx

__all__ = ["gated_mm", "gated_mm_grad"]


def _gated(x, w_in, w_up, offsets, out, keep):
    """(h, a, b)"""
    with torch.no_grad():
        a, b = grouped_mm(x, w_in, offsets), grouped_mm(x, w_up, offsets)
        return gated_act(a, b), a, b


class _GatedMM(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_in, w_up, offsets):
        h, a, b = _gated(x, w_in, w_up, offsets, None, True)
        ctx.save_for_backward(x, w_in, w_up, a, b, offsets)
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        x, w_in, w_up, a, b, offsets = ctx.saved_tensors
        return *gated_mm_grad(_grad(dh), x, w_in, w_up, a, b, offsets), None


def gated_mm(x, w_in, w_up, offsets, out=None):
    if torch.is_grad_enabled() and any(getattr(t, "requires_grad", False) for t in (x, w_in, w_up)):
        if out is not None:
            raise ValueError("out cannot be given where a gradient is recorded")
        return _GatedMM.apply(x, w_in, w_up, offsets)
    return _gated(x, w_in, w_up, offsets, out, False)[0]


def gated_mm_grad(dh, x, w_in, w_up, a, b, offsets):
    da, db = gated_act_grad(dh, a, b)
    dx = grouped_mm_dx(da, w_in, offsets)
    dx.add_(grouped_mm_dx(db, w_up, offsets))
    return dx, grouped_mm_dw(x, da, offsets), grouped_mm_dw(x, db, offsets)
