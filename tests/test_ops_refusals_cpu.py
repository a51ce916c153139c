"""Calls that the wrappers refuse on the host, before anything is enqueued (CPU tensors: a call
that passes every check ends at "on the GPU")."""
import pytest
import torch

import mixture_experts_layer_46_amd as M

bf, f32, i32, i8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


def z(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("out,msg", [
    (z(3, 24), "out must have shape"), (z(3, 8), "out must have shape"), (z(4, 16), "out must have shape"),
    (z(3, 16, dtype=f32), "out must be torch.bfloat16")])
def test_combine_refuses_an_out_of_another_shape(out, msg):
    """combine writes T rows of y_perm's width wherever `out` points."""
    with pytest.raises(ValueError, match=msg):
        M.combine(z(6, 16), z(6, dtype=i32), z(3, 2, dtype=f32), out=out)


T, H, E, F, K = 4, 32, 4, 48, 2


def _experts(h=H, e=E, f=F, up=True):
    """8-bit experts as quantize_ffn lays them out: q [E, N, K], scale [E, N]."""
    pair = lambda n, k: (z(e, n, k, dtype=i8), z(e, n, dtype=f32))
    return M.QuantizedExperts(pair(f, h), pair(f, h) if up else None, pair(h, f))


GOOD, WIDE, NARROW, FEW, THIN = _experts(), _experts(h=64), _experts(h=16), _experts(e=3), _experts(f=32)

MISFITS = [
    (GOOD._replace(w_out=WIDE.w_out), "w_out, 8-bit, must have shape"),          # more columns than a token has
    (GOOD._replace(w_out=NARROW.w_out), "w_out, 8-bit, must have shape"),        # fewer
    (GOOD._replace(w_out=THIN.w_out), "w_out, 8-bit, must have shape"),          # another hidden width
    (GOOD._replace(w_out=FEW.w_out), "w_out, 8-bit, must have shape"),           # fewer experts
    (GOOD._replace(w_up=THIN.w_up), "w_up, 8-bit, must have shape"), (GOOD._replace(w_up=WIDE.w_up), "w_up, 8-bit, must have"),
    (GOOD._replace(w_in=NARROW.w_in), "w_in, 8-bit, must have shape"), (FEW, "w_in, 8-bit, must have shape"),
    (GOOD._replace(w_out=(GOOD.w_out[0], z(E, H + 1, dtype=f32))), "w_out's scale must have shape"),
    (GOOD._replace(w_out=(GOOD.w_out[0], z(E, H))), "w_out's scale must be torch.float32"),
    (GOOD._replace(w_in=(z(E, F, H), GOOD.w_in[1])), "w_in, 8-bit, must be torch.int8"),
    (GOOD._replace(w_out=(None, GOOD.w_out[1])), "w_out, 8-bit, is required"),
]


@pytest.mark.parametrize("experts,msg", MISFITS)
def test_8bit_layer_refuses_experts_that_do_not_fit(experts, msg):
    """Experts of another width than the tokens' would have the combine write past `out`."""
    with pytest.raises(ValueError, match=msg):
        M.forward_int8(z(T, H), z(H, E, dtype=f32), experts, K)
    with pytest.raises(ValueError, match=msg):
        M.forward_int8(z(0, H), z(H, E, dtype=f32), experts, K)
    with pytest.raises(ValueError, match=msg):
        M.grouped_ffn_int8(z(T * K, H), z(E + 1, dtype=i32), experts)


def test_8bit_layer_takes_experts_that_fit():
    """... as far as the checks go: what is left to refuse is the host's memory."""
    for experts in (GOOD, _experts(up=False)):
        with pytest.raises(ValueError, match="on the GPU"):
            M.forward_int8(z(T, H), z(H, E, dtype=f32), experts, K)
        with pytest.raises(ValueError, match="on the GPU"):
            M.grouped_ffn_int8(z(T * K, H), z(E + 1, dtype=i32), experts)


@pytest.mark.parametrize("w_in,w_up,w_out,msg", [
    (z(E, H, F), z(E, H, F), z(E, F, 2 * H), "w_out must have shape"), (z(E, H, F), None, z(E, H, F), "w_out must have shape"),
    (z(E, H, F), z(E, H, 2 * F), z(E, F, H), "w_up must have shape"), (z(E, H, F), None, z(3, F, H), "w_out must have shape"),
    (z(E, H, F), None, z(E, F, H, dtype=f32), "w_out must be torch.bfloat16"), (z(H, F), None, z(E, F, H), "w_in must be a tensor")])
def test_quantize_ffn_refuses_matrices_that_do_not_fit(w_in, w_up, w_out, msg):
    with pytest.raises(ValueError, match=msg):
        M.quantize_ffn(w_in, w_up, w_out)
