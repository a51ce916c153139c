"""The norms before and after a block, fused with the block's gate and residual scale
(include/moe_ops.h):

    u       = norm(x, w)                                          before the first block
    y, u    = residual_norm(x, z, w_post, gate, scale, w_next)    behind a block, before the next

Both are differentiable; norm_grad and residual_norm_grad are the gradients alone.  Checks,
streams and given outputs as in ops.py.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import NormShape
from .ops import _apart, _code, _dims, _given, _grad, _launch, _on, _recorded, _row_stride, _wrote

__all__ = ["norm", "norm_grad", "residual_norm", "residual_norm_grad"]

_NONE, _CHANNEL, _TOKEN = 0, 1, 2


@functools.lru_cache(maxsize=512)
def _shape(T, ldx, ldz, H, code, gate, scale, eps):
    """(the C struct of a call's sizes, the gradient's bytes of workspace); read only and kept,
    since making them costs microseconds."""
    s = ctypes.byref(NormShape(T, ldx, ldz, H, code, gate, scale, eps))
    n = ctypes.c_size_t(0)
    # sizes out of range are refused by the operator itself
    return s, n.value if _lib.load().moe_residual_norm_grad_workspace(s, ctypes.byref(n)) == 0 else 0


def _gate_kind(gate, T, H, dev):
    if gate is None:
        return _NONE
    if isinstance(gate, torch.Tensor) and gate.dim() == 2:
        _given(gate, "gate", torch.float32, (T, 1), dev)
        return _TOKEN
    _given(gate, "gate", torch.float32, (H,), dev)
    return _CHANNEL


def _args(x, z, w_post, gate, scale, w_next, eps):
    """(T, H, GPU, C struct, workspace bytes)"""
    _dims(x, 2, "x")
    code = _code(x, "x")
    T, H = x.shape
    dev = x.get_device()
    ldz = H
    if z is not None:
        _dims(z, 2, "z")
        if z.dtype != x.dtype or z.shape != x.shape:
            raise ValueError(f"z must be {x.dtype} of shape {tuple(x.shape)}, got {z.dtype} {tuple(z.shape)}")
        if not z.is_contiguous():
            ldz = _row_stride(z, "z")
    if w_post is not None:
        _given(w_post, "w_post", torch.float32, (H,), dev)
    if w_next is not None:
        _given(w_next, "w_next", torch.float32, (H,), dev)
    kind = _gate_kind(gate, T, H, dev)
    ldx = H if x.is_contiguous() else _row_stride(x, "x")
    if z is not None and z.get_device() != dev:
        _on(z, "z", dev)
    s, ws = _shape(T, ldx, ldz, H, code, kind, scale, eps)
    return T, H, dev, s, ws


def _ptr(t):
    return None if t is None else t.data_ptr()


def _number(v, name):
    """A number of the caller's; not a tensor, whose gradient would be lost and whose value would
    have to be waited for."""
    if isinstance(v, torch.Tensor):
        raise ValueError(f"{name} must be a number, not a tensor (it has no gradient)")
    return float(v)


def _forward(x, z, w_post, gate, scale, w_next, eps, out):
    T, H, dev, s, _ = _args(x, z, w_post, gate, scale, w_next, eps)
    y = u = None
    if out is None:
        _on(x, "x", None)
        y = None if z is None else torch.empty_like(z)
        u = None if w_next is None else torch.empty_like(x)
    else:
        y, u = out
        for o, name, wanted in ((y, "y", z is not None), (u, "u", w_next is not None)):
            if not wanted:
                if o is not None:
                    raise ValueError(f"{name} is not made by this call")
                continue
            _given(o, name, x.dtype, (T, H), dev)
            _apart(o, name, x=x, z=z, w_post=w_post, gate=gate, w_next=w_next, u=u if o is y else None)
        _on(x, "x", None)
    if T > 0:
        _launch(dev, "moe_residual_norm", s, x.data_ptr(), _ptr(z), _ptr(w_post), _ptr(gate), _ptr(w_next), _ptr(y), _ptr(u))
    if out is not None:
        _wrote(y, u)
    return y, u


def _backward(dy, du, x, z, w_post, gate, scale, w_next, eps):
    T, H, dev, s, ws = _args(x, z, w_post, gate, scale, w_next, eps)
    if dy is not None:
        _given(dy, "dy", x.dtype, (T, H), dev)
    if w_next is not None:
        _given(du, "du", x.dtype, (T, H), dev)
    elif du is not None:
        raise ValueError("du needs w_next")
    _on(x, "x", None)
    dx = torch.empty_like(x)
    dz = None if z is None else torch.empty_like(z)
    dw_post, dgate, dw_next = (None if t is None else torch.empty_like(t) for t in (w_post, gate, w_next))
    part = x.new_empty(ws // 4, dtype=torch.float32)
    _launch(dev, "moe_residual_norm_grad", s, _ptr(dy), _ptr(du), x.data_ptr(), _ptr(z), _ptr(w_post), _ptr(gate),
            _ptr(w_next), dx.data_ptr(), _ptr(dz), _ptr(dw_post), _ptr(dgate), _ptr(dw_next), part.data_ptr(), ws)
    return dx, dz, dw_post, dgate, dw_next


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, w_post, gate, scale, w_next, eps):
        ctx.save_for_backward(x, z, w_post, gate, w_next)
        ctx.scale, ctx.eps = scale, eps
        ctx.set_materialize_grads(False)
        return _forward(x, z, w_post, gate, scale, w_next, eps, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, du):
        x, z, w_post, gate, w_next = ctx.saved_tensors
        dy = None if dy is None else _grad(dy)
        if w_next is not None:                              # u without a use: zeros
            du = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if du is None else _grad(du)
        dx, dz, dw_post, dgate, dw_next = _backward(dy, du, x, z, w_post, gate, ctx.scale, w_next, ctx.eps)
        return dx, dz, dw_post, dgate, None, dw_next, None


def _run(x, z, w_post, gate, scale, w_next, eps, out):
    if _recorded(x, z, w_post, gate, w_next):
        if out is not None:
            raise ValueError("out cannot be given where a gradient is recorded")
        return _Norm.apply(x, z, w_post, gate, scale, w_next, eps)
    return _forward(x, z, w_post, gate, scale, w_next, eps, out)


def norm(x, w, eps=1e-6, out=None):
    """u = x r(x) w, r(x) = 1 / sqrt(mean of the row's squares + eps): the norm of rows.

    x [T, H] bf16 or fp32, dense along H, rows may be apart; w [H] fp32; u [T, H] in x's type,
    computed in fp32 and rounded once.  H a multiple of 8, at most 16384.  Differentiable in x
    and w (without `out`)."""
    if w is None:
        raise ValueError("w is required")
    return _run(x, None, None, None, 1.0, w, _number(eps, "eps"), None if out is None else (None, out))[1]


def norm_grad(du, x, w, eps=1e-6):
    """(dx, dw) of norm for the gradient du [T, H]."""
    if w is None:
        raise ValueError("w is required")
    dx, _, _, _, dw = _backward(None, du, x, None, None, None, 1.0, w, _number(eps, "eps"))
    return dx, dw


def residual_norm(x, z, w_post=None, gate=None, scale=1.0, w_next=None, eps=1e-6, out=None):
    """(y, u): the stream behind a block, and the next block's input.

        v = z r(z) w_post    y = scale x + gate v    u = y r(y) w_next

    x, z [T, H] bf16 or fp32 (the stream and the block's output), dense along H, rows may be
    apart; w_post, w_next [H] fp32; gate fp32, [H] (a number per channel) or [T, 1] (per
    token); scale a number, not a tensor.  Without w_post v = z, without gate it is 1, without
    w_next u is None.  All in fp32, u from the unrounded y; y and u [T, H] in x's type, each
    rounded once.  H a multiple of 8, at most 16384.  `out` = (y, u): tensors to write.
    Differentiable in x, z, w_post, gate and w_next (without `out`)."""
    if z is None:
        raise ValueError("z is required")
    return _run(x, z, w_post, gate, _number(scale, "scale"), w_next, _number(eps, "eps"), out)


def residual_norm_grad(dy, du, x, z, w_post=None, gate=None, scale=1.0, w_next=None, eps=1e-6):
    """(dx, dz, dw_post, dgate, dw_next) of residual_norm for the gradients dy [T, H] (None: zeros)
    and du [T, H] (None without w_next); None for a parameter that is not there."""
    if z is None:
        raise ValueError("z is required")
    return _backward(dy, du, x, z, w_post, gate, _number(scale, "scale"), w_next, _number(eps, "eps"))
