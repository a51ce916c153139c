"""The gated half of the experts' feed-forward, grouped by expert (include/moe_ops.h):

    h = gated_mm(x, w_in, w_up, offsets)            SiLU(x W_in) * (x W_up), one kernel; differentiable
    dx, dw_in, dw_up = gated_mm_grad(dh, x, w_in, w_up, a, b, offsets)

With one group (offsets [0, R]) they are those of a dense gated feed-forward.  Checks, streams and
given outputs as in ops.py.
"""
from __future__ import annotations

import torch

from .ops import _apart, _code, _dense, _dims, _given, _grad, _launch, _mm_shape, _recorded, _spec, _wrote

__all__ = ["gated_mm", "gated_mm_grad"]


def _check_matrices(w_in, w_up, offsets, dtype, dev):
    _dims(w_in, 3, "w_in")
    E, K, N = w_in.shape
    _given(w_in, "w_in", dtype, (E, K, N), dev)
    _given(w_up, "w_up", dtype, (E, K, N), dev)
    _given(offsets, "offsets", torch.int32, (E + 1,), dev)
    return E, K, N


def _gated(x, w_in, w_up, offsets, out, keep):
    """(h, a, b), the projections a and b None unless they are to be kept"""
    _dims(x, 2, "x")
    code = _code(x, "x")
    dev = x.get_device()
    E, K, N = _check_matrices(w_in, w_up, offsets, x.dtype, dev)
    R = x.shape[0]
    _given(x, "x", x.dtype, (R, K), dev)
    if out is not None:
        _given(out, "out", x.dtype, (R, N), dev)
        _apart(out, "out", x=x, w_in=w_in, w_up=w_up, offsets=offsets)
    _dense(x, "x")
    h = x.new_empty((R, N)) if out is None else out
    a, b = (x.new_empty((R, N)), x.new_empty((R, N))) if keep else (None, None)
    _launch(dev, "moe_gated_mm", _mm_shape(R, E, K, N, code, code, out is None), x.data_ptr(), w_in.data_ptr(),
            w_up.data_ptr(), offsets.data_ptr(), h.data_ptr(), a.data_ptr() if keep else None, b.data_ptr() if keep else None)
    if out is not None:
        _wrote(out)
    return h, a, b


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
        return *_gated_grad(_grad(dh), x, w_in, w_up, a, b, offsets, ctx.needs_input_grad), None


def gated_mm(x, w_in, w_up, offsets, out=None):
    """h[r] = SiLU(x[r] @ w_in[e]) * (x[r] @ w_up[e]) for the rows r of every group e, the rows
    [offsets[e], offsets[e+1]).

    x [R, K], w_in and w_up [E, K, N] bf16 or fp32, offsets [E+1] int32 (permute's); h [R, N] in x's
    type, computed in fp32 and rounded once.  Rows that lie in no group are zeros, or with `out`
    given left as they were.  K and N multiples of 8.  Differentiable in x, w_in and w_up (without
    `out`); the two projections are then kept, in x's type, for the gradient."""
    if _recorded(x, w_in, w_up):
        if out is not None:
            raise ValueError("out cannot be given where a gradient is recorded")
        return _GatedMM.apply(x, w_in, w_up, offsets)
    return _gated(x, w_in, w_up, offsets, out, False)[0]


def gated_mm_grad(dh, x, w_in, w_up, a, b, offsets):
    """(dx, dw_in, dw_up) of gated_mm for the gradient dh [R, N], given the projections a = x @ w_in
    and b = x @ w_up [R, N] in x's type.  The projections' gradients between are rounded to x's type
    (what the matrix instructions take).  Rows of dx that lie in no group are zeros."""
    return _gated_grad(dh, x, w_in, w_up, a, b, offsets, (True, True, True))


def _gated_grad(dh, x, w_in, w_up, a, b, offsets, needed):
    _dims(x, 2, "x")
    code = _code(x, "x")
    dev = x.get_device()
    E, K, N = _check_matrices(w_in, w_up, offsets, x.dtype, dev)
    R = x.shape[0]
    _given(x, "x", x.dtype, (R, K), dev)
    for name, t in (("dh", dh), ("a", a), ("b", b)):
        _given(t, name, x.dtype, (R, N), dev)
    _dense(x, "x")
    # the operators without their wrappers' checks, which are done: with the two
    # weight gradients in one launch 36 -> 23 us of the host's time a call
    da, db = x.new_empty((R, N)), x.new_empty((R, N))
    _launch(dev, "moe_gated_act_grad", code, R, N, _spec(0.0, 0, 0, dev), dh.data_ptr(), a.data_ptr(), N, b.data_ptr(), N,
            da.data_ptr(), N, db.data_ptr(), N)
    dx, dw = None, [torch.empty_like(w) if n else None for w, n in zip((w_in, w_up), needed[1:])]
    if needed[0]:
        dx = torch.empty_like(x)
        _launch(dev, "moe_gated_mm_dx", _mm_shape(R, E, K, N, code, code, True), da.data_ptr(), db.data_ptr(),
                w_in.data_ptr(), w_up.data_ptr(), offsets.data_ptr(), dx.data_ptr())
    shape = _mm_shape(R, E, K, N, code, code, False)
    if needed[1] and needed[2]:
        _launch(dev, "moe_gated_mm_dw", shape, x.data_ptr(), da.data_ptr(), db.data_ptr(), offsets.data_ptr(),
                dw[0].data_ptr(), dw[1].data_ptr())
    else:
        for d, w in zip((da, db), dw):
            if w is not None:
                _launch(dev, "moe_grouped_mm_dw", shape, x.data_ptr(), d.data_ptr(), offsets.data_ptr(), w.data_ptr())
    return dx, *dw
