"""Calls that the wrappers refuse on the host, before anything is enqueued (CPU tensors: a call
that passes every check ends at "on the GPU", which no case here expects)."""
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
