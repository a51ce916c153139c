"""The layer between its norms: one block of a residual stream.

    u    = norm(x, w_first)                                             before the first block
    x, u = forward_block(x, u, w_gate, experts, top_k, w_post, gate, scale, w_next)

A chain of blocks hands (x, u) on; the last one has the stack's final norm as its w_next.
"""
from __future__ import annotations

import torch

from . import _lib
from ._lib import MOE_FLAG_NO_RENORM
from .fp8 import Fp8Experts, forward_fp8
from .gated import gated_mm
from .norms import _number, residual_norm
from .ops import (QuantizedExperts, _Combine, _current, _Permute, _recorded, _Route, forward_int8, gated_act,
                  grouped_mm)

__all__ = ["forward_block"]


def _layer_train(u, w_gate, w_in, w_up, w_out, top_k, bias, flags, capacity_factor):
    """The layer, differentiable: forward_train's chain without dropout, its gated half in one
    kernel."""
    import mixture_experts_layer_46_amd as M
    T, H, E, F = M._check_layer(u, w_gate, bias, w_in, w_up, w_out, None, top_k)
    if flags & MOE_FLAG_NO_RENORM:
        raise ValueError("the gradient is that of renormalised gates only")
    if T == 0:
        raise ValueError("a recorded block needs at least one token")
    with _current(u=u, w_gate=w_gate, bias=bias, w_in=w_in, w_up=w_up, w_out=w_out):
        g, idx, _ = _Route.apply(u, w_gate, bias, top_k, flags)
        capacity = _lib.capacity_rows(capacity_factor, T, top_k, E)
        rows, offsets, row_of_pair = _Permute.apply(u, idx, E, capacity)
        h = gated_act(grouped_mm(rows, w_in, offsets)) if w_up is None else gated_mm(rows, w_in, w_up, offsets)
        return _Combine.apply(grouped_mm(h, w_out, offsets), row_of_pair, g, capacity == 0)


def forward_block(x, u, w_gate, experts, top_k, w_post=None, gate=None, scale=1.0, w_next=None, bias=None, flags=0,
                  capacity_factor=None, eps=1e-6):
    """(y, u_next): z = the layer of u, then residual_norm(x, z, w_post, gate, scale, w_next, eps).

    x, u [T, H]: the stream, and the layer's input (norm of it, or the block before's u_next).
    experts: (w_in, w_up, w_out) as forward takes them (w_up None for the two-layer SiLU FFN), or
    8-bit ones (quantize_ffn, quantize_ffn_fp8).  Differentiable in x, u, w_gate, bias, the
    experts' matrices (not 8-bit ones), w_post, gate and w_next."""
    import mixture_experts_layer_46_amd as M
    scale, eps = _number(scale, "scale"), _number(eps, "eps")
    if isinstance(experts, (QuantizedExperts, Fp8Experts)):
        if _recorded(u, w_gate, bias):
            raise ValueError("8-bit experts have no gradient: use torch.no_grad()")
        layer = forward_int8 if isinstance(experts, QuantizedExperts) else forward_fp8
        z = layer(u, w_gate, experts, top_k, bias=bias, flags=flags, capacity_factor=capacity_factor)
    else:
        w_in, w_up, w_out = experts
        if _recorded(u, w_gate, bias, w_in, w_up, w_out):
            z = _layer_train(u, w_gate, w_in, w_up, w_out, top_k, bias, flags, capacity_factor)
        elif M._check_layer(u, w_gate, bias, w_in, w_up, w_out, None, top_k)[0] == 0:
            z = torch.empty_like(u)
        else:
            with _current(u=u, w_gate=w_gate, bias=bias, w_in=w_in, w_up=w_up, w_out=w_out):
                z = M.forward(u, w_gate, w_in, w_up, w_out, top_k, bias=bias, flags=flags, capacity_factor=capacity_factor)
    return residual_norm(x, z, w_post, gate, scale, w_next, eps)
