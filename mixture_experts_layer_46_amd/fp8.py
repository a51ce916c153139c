"""Experts in 8-bit floating point (e4m3) with a power-of-two scale for each block of 128
(include/moe_ops.h):

    q, scale = quantize_rows_fp8(x)                 a scale for each 128 elements of a row
    q, scale = quantize_experts_fp8(w)              a scale for each 128 x 128 of an expert
    y        = grouped_mm_fp8(xq, x_scale, wq, w_scale, offsets)

and the layer made of them:

    forward_fp8(x, w_gate, experts, top_k, ...)     experts = quantize_ffn_fp8(w_in, w_up, w_out)

Scales are torch.float8_e8m0fnu (a biased exponent), which the matrix instructions apply
themselves.  Checks, streams and given outputs as in ops.py.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from ._lib import MOE_BF16
from .ops import _CODES, _apart, _check, _code, _current, _dense, _dims, _given, _launch, _mm_shape, _on, _wrote, gated_act

__all__ = ["quantize_rows_fp8", "quantize_experts_fp8", "grouped_mm_fp8", "Fp8Experts", "quantize_ffn_fp8",
           "grouped_ffn_fp8", "forward_fp8"]

_Q, _S = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _scales(K):
    """Bytes of a row of scales over K elements: one per 128, in whole fours."""
    return (K + 511) // 512 * 4


def quantize_rows_fp8(x):
    """8-bit floating-point rows of x [R, K] (bf16 or fp32): (q [R, K] float8_e4m3fn, scale [R, S]
    float8_e8m0fnu), S = 4 ceil(K / 512), of which scale[r, i] is that of q[r, 128 i : 128 i + 128]:
    the least power of two 2^e, e >= -127, for which the block's largest magnitude is at most
    448 2^e.  A block with an infinity or a NaN gets scale NaN and q 0.  K a multiple of 16."""
    _dims(x, 2, "x")
    code = _code(x, "x")
    R, K = x.shape
    dev = _dense(x, "x")
    q = torch.empty_like(x, dtype=_Q)                       # (the quickest of torch's calls: the host's time counts)
    scale = x.new_empty((R, _scales(K)), dtype=_S)
    _launch(dev, "moe_quantize_rows_fp8", code, R, K, x.data_ptr(), q.data_ptr(), scale.data_ptr())
    return q, scale


def quantize_experts_fp8(w):
    """8-bit floating-point expert matrices of w [E, K, N] (bf16 or fp32), made once:
    (q [E, N, K] float8_e4m3fn, scale [E, ceil(N / 128), S] float8_e8m0fnu), S = 4 ceil(K / 512):
    a scale for each block of 128 x 128, as quantize_rows_fp8 has one for 128 elements.  K a
    multiple of 16, N of 8."""
    _dims(w, 3, "w")
    code = _code(w, "w")
    E, K, N = w.shape
    dev = _dense(w, "w")
    q = torch.empty((E, N, K), dtype=_Q, device=w.device)
    scale = torch.empty((E, (N + 127) // 128, _scales(K)), dtype=_S, device=w.device)
    _launch(dev, "moe_quantize_experts_fp8", code, E, K, N, w.data_ptr(), q.data_ptr(), scale.data_ptr())
    return q, scale


def grouped_mm_fp8(xq, x_scale, wq, w_scale, offsets, dtype=torch.bfloat16, out=None):
    """y[r] = (xq[r] x_scale[r]) @ (wq[e] w_scale[e])^T, each block of 128 times its scale, for the
    rows r of every group e: summed in fp32, one rounding to `dtype` (bf16 or fp32).

    xq [R, K] and x_scale [R, S] as quantize_rows_fp8 makes them, wq [E, N, K] and w_scale
    [E, ceil(N / 128), S] as quantize_experts_fp8 does, offsets [E+1] int32 -> [R, N].  Rows
    that lie in no group are zeros, or with `out` given left as they were.

    With bf16 output the 8-bit matrix instruction adds 8 consecutive products of the contraction at
    a time and drops of them what lies below 2^-13 of the largest, before the sum goes on in fp32:
    a result is off by at most 2^-10 of the sum of these largest magnitudes (over random values by
    1.5e-5 of the result's norm, where the rounding to bf16 is 1.7e-3 of it).  Where large products
    cancel and the small ones between them count, take dtype=torch.float32, with which every product
    is exact and all are summed in fp32: up to 2.4 times the time where matrix instructions bound
    the call, 3% more where reading the experts does."""
    _dims(xq, 2, "xq")
    _dims(wq, 3, "wq")
    R, K = xq.shape
    E, N, _ = wq.shape
    dev = xq.get_device()
    _given(xq, "xq", _Q, (R, K), dev)
    _given(x_scale, "x_scale", _S, (R, _scales(K)), dev)
    _given(wq, "wq", _Q, (E, N, K), dev)
    _given(w_scale, "w_scale", _S, (E, (N + 127) // 128, _scales(K)), dev)
    _given(offsets, "offsets", torch.int32, (E + 1,), dev)
    rest = out is None
    if not rest:
        dtype = out.dtype
    if dtype not in _CODES:
        raise TypeError(f"unsupported output type {dtype}")
    if not rest:
        _given(out, "out", dtype, (R, N), dev)
        _apart(out, "out", xq=xq, x_scale=x_scale, wq=wq, w_scale=w_scale, offsets=offsets)
    _on(xq, "xq", None)
    if rest:
        out = xq.new_empty((R, N), dtype=dtype)
    _launch(dev, "moe_grouped_mm_fp8", _mm_shape(R, E, K, N, MOE_BF16, _CODES[dtype], rest), xq.data_ptr(),
            x_scale.data_ptr(), wq.data_ptr(), w_scale.data_ptr(), offsets.data_ptr(), out.data_ptr())
    if not rest:
        _wrote(out)
    return out


# ------------------------------------------------------------------------- the layer
class Fp8Experts(NamedTuple):
    """The experts' matrices (quantize_ffn_fp8): (q [E, N, K], scale [E, ceil(N / 128), S]) each."""
    w_in: tuple
    w_up: Optional[tuple]
    w_out: tuple


def quantize_ffn_fp8(w_in, w_up, w_out) -> Fp8Experts:
    """The experts of forward (w_in, w_up [E, H, F], w_up None for the two-layer SiLU FFN;
    w_out [E, F, H]) in 8-bit floating point, made once.  H and F multiples of 16."""
    _dims(w_in, 3, "w_in")
    E, H, F = w_in.shape
    if w_up is not None:
        _check(w_up, "w_up", w_in.dtype, (E, H, F))
    _check(w_out, "w_out", w_in.dtype, (E, F, H))
    return Fp8Experts(quantize_experts_fp8(w_in), None if w_up is None else quantize_experts_fp8(w_up),
                      quantize_experts_fp8(w_out))


def _check_experts(experts, E, H):
    """Raises unless the matrices are those of E experts between rows of H and hidden rows of one
    width."""
    _dims(experts.w_in[0], 3, "w_in")
    F = experts.w_in[0].shape[1]
    for name, pair, (n, k) in (("w_in", experts.w_in, (F, H)), ("w_up", experts.w_up, (F, H)), ("w_out", experts.w_out, (H, F))):
        if pair is not None or name != "w_up":
            _check(pair[0], f"{name}, 8-bit,", _Q, (E, n, k))
            _check(pair[1], f"{name}'s scale", _S, (E, (n + 127) // 128, _scales(k)))


def grouped_ffn_fp8(x_perm, offsets, experts: Fp8Experts):
    """The grouped expert FFN on 8-bit floating-point experts: the rows x_perm [R, H] and the
    activated hidden rows are quantised, with a scale for each 128 elements.  Returns [R, H] in
    x_perm's type, which is that of the products' output, too (see grouped_mm_fp8); rows that lie
    in no group are zeros."""
    _dims(x_perm, 2, "x_perm")
    _dims(offsets, 1, "offsets")
    _check_experts(experts, offsets.shape[0] - 1, x_perm.shape[1])
    q, s = quantize_rows_fp8(x_perm)
    a = grouped_mm_fp8(q, s, *experts.w_in, offsets, dtype=x_perm.dtype)
    b = None if experts.w_up is None else grouped_mm_fp8(q, s, *experts.w_up, offsets, dtype=x_perm.dtype)
    q, s = quantize_rows_fp8(gated_act(a, b))
    return grouped_mm_fp8(q, s, *experts.w_out, offsets, dtype=x_perm.dtype)


def forward_fp8(x, w_gate, experts: Fp8Experts, top_k, bias=None, flags=0, capacity_factor=None, out=None):
    """The whole layer (forward) with 8-bit floating-point experts (quantize_ffn_fp8); the routing
    stays fp32."""
    import mixture_experts_layer_46_amd as M
    T, H, E, _ = M._check_layer(x, w_gate, bias, out=out, top_k=top_k, experts=False)
    _check_experts(experts, E, H)
    given = out
    if out is None:
        out = torch.empty_like(x)
    if T == 0:
        return out
    with _current(x=x, w_gate=w_gate, bias=bias, out=out):
        _, idx, w = M.route(x, w_gate, top_k, bias=bias, flags=flags)
        g = M.permute(idx, E, x=x, capacity=_lib.capacity_rows(capacity_factor, T, top_k, E))
        y = grouped_ffn_fp8(g["x_perm"], g["offsets"], experts)
        M.combine(y, g["row_of_pair"], w, out=out)
    if given is not None:
        _wrote(given)
    return out
