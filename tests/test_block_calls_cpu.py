"""Calls of the block's operators that would lose something silently, refused on the host (CPU tensors: a
call that passes every check ends at "on the GPU")."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_46_amd as M

bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
T, H, E, F, K = 4, 32, 4, 48, 2


def z(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


W = z(H, dtype=f32)
EXPERTS = (z(E, H, F), z(E, H, F), z(E, F, H))
GATE = z(H, E, dtype=f32)


@pytest.mark.parametrize("value", [torch.tensor(0.5), torch.nn.Parameter(torch.tensor(0.5)), torch.ones(1)],
                         ids=["tensor", "parameter", "one element"])
@pytest.mark.parametrize("name,call", [
    ("scale", lambda v: M.residual_norm(z(T, H), z(T, H), W, None, v, W)),
    ("scale", lambda v: M.residual_norm_grad(z(T, H), z(T, H), z(T, H), z(T, H), W, None, v, W)),
    ("scale", lambda v: M.forward_block(z(T, H), z(T, H), GATE, EXPERTS, K, W, None, v, W)),
    ("eps", lambda v: M.residual_norm(z(T, H), z(T, H), W, None, 1.0, W, eps=v)),
    ("eps", lambda v: M.residual_norm_grad(z(T, H), z(T, H), z(T, H), z(T, H), W, None, 1.0, W, eps=v)),
    ("eps", lambda v: M.forward_block(z(T, H), z(T, H), GATE, EXPERTS, K, W, None, 1.0, W, eps=v)),
    ("eps", lambda v: M.norm(z(T, H), W, v)), ("eps", lambda v: M.norm_grad(z(T, H), z(T, H), W, v))])
def test_scale_and_eps_are_numbers(name, call, value):
    """A tensor would lose its gradient (a learnable scale never moves), and its value would be read
    back from the GPU, which no captured call may do."""
    with pytest.raises(ValueError, match=f"{name} must be a number"):
        call(value)


@pytest.mark.parametrize("value", [1, 0.5, np.float32(0.5), np.float64(0.5)])
def test_numbers_of_any_kind_pass(value):
    with pytest.raises(ValueError, match="on the GPU"):
        M.residual_norm(z(T, H), z(T, H), W, None, value, W, eps=value)


def _dual(*shape, dtype=f32):
    return torch.autograd.forward_ad.make_dual(z(*shape, dtype=dtype), z(*shape, dtype=dtype))


OFF = torch.zeros(E + 1, dtype=i32)
FP8 = M.Fp8Experts(*((torch.zeros(E, n, k, dtype=torch.uint8).view(torch.float8_e4m3fn),
                      torch.zeros(E, 1, 4, dtype=torch.uint8).view(torch.float8_e8m0fnu)) for n, k in ((F, H), (F, H), (H, F))))


@pytest.mark.parametrize("call", [
    lambda: M.norm(_dual(T, H), W), lambda: M.norm(z(T, H), _dual(H)),
    lambda: M.residual_norm(z(T, H), _dual(T, H, dtype=bf)), lambda: M.residual_norm(z(T, H), z(T, H), W, _dual(H), 1.0, W),
    lambda: M.residual_norm(z(T, H), z(T, H), _dual(H)), lambda: M.residual_norm(z(T, H), z(T, H), w_next=_dual(H)),
    lambda: M.gated_mm(_dual(T, H, dtype=bf), EXPERTS[0], EXPERTS[1], OFF),
    lambda: M.gated_mm(z(T, H), _dual(E, H, F, dtype=bf), EXPERTS[1], OFF),
    lambda: M.gated_mm(z(T, H), EXPERTS[0], _dual(E, H, F, dtype=bf), OFF),
    lambda: M.grouped_mm(_dual(T, H, dtype=bf), EXPERTS[0], OFF), lambda: M.grouped_mm(z(T, H), _dual(E, H, F, dtype=bf), OFF),
    lambda: M.gated_act(_dual(T, F, dtype=bf), z(T, F)), lambda: M.gated_act(z(T, F), _dual(T, F, dtype=bf)),
    lambda: M.dropout(_dual(T, F, dtype=bf), 0.5, 1),
    lambda: M.forward_block(z(T, H), _dual(T, H, dtype=bf), GATE, EXPERTS, K),
    lambda: M.forward_block(z(T, H), z(T, H), _dual(H, E), EXPERTS, K),
    lambda: M.forward_block(z(T, H), z(T, H), GATE, (EXPERTS[0], EXPERTS[1], _dual(E, F, H, dtype=bf)), K),
    lambda: M.forward_block(z(T, H), z(T, H), GATE, EXPERTS, K, bias=_dual(E)),
    lambda: M.forward_block(z(T, H), _dual(T, H, dtype=bf), GATE, FP8, K),
    lambda: M.forward_block(z(T, H), z(T, H), _dual(H, E), FP8, K),
    lambda: M.forward_train(_dual(T, H, dtype=bf), GATE, *EXPERTS, K)])
@pytest.mark.parametrize("recorded", [True, False])
def test_forward_mode_tangents_are_refused(call, recorded):
    """No operator has a forward-mode derivative: a tangent that came in would be missing from what goes
    out, with no sign of it."""
    with torch.autograd.forward_ad.dual_level(), torch.set_grad_enabled(recorded):
        with pytest.raises(ValueError, match="forward-mode"):
            call()
        with pytest.raises(ValueError, match="on the GPU"):               # without a tangent nothing is refused
            M.norm(z(T, H), W)
        with pytest.raises(ValueError, match="on the GPU"):
            M.gated_mm(z(T, H).requires_grad_(), EXPERTS[0], EXPERTS[1], OFF)


def test_jvp_is_refused():
    for f in (lambda t: M.norm(t, W), lambda t: M.residual_norm(t, t)[0], lambda t: M.gated_act(t, t)):
        with pytest.raises(ValueError, match="forward-mode"):
            torch.func.jvp(f, (z(T, H),), (z(T, H),))


@pytest.mark.parametrize("T_", [T, 0])
def test_served_block_runs_on_its_tensors_gpu(monkeypatch, T_):
    """The layer's own stages take the current device's stream: forward_block makes the tensors' GPU the
    current one around them (whatever kind of experts), and refuses tensors of two GPUs.  Without a second
    GPU: the context is a mark, the layer a look at it."""
    from contextlib import contextmanager

    from mixture_experts_layer_46_amd import block
    inside, seen = [], []

    @contextmanager
    def current(**ts):
        inside.append({n for n, t in ts.items() if t is not None})
        yield
        inside.pop()

    def layer(x, *args, **kw):
        seen.append(set(inside[-1]) if inside else None)
        return x

    monkeypatch.setattr(block, "_current", current, raising=False)
    monkeypatch.setattr(M, "forward", layer)
    monkeypatch.setattr(block, "residual_norm", lambda *a: a[:2])
    u = z(T_, H)
    M.forward_block(z(T_, H), u, GATE, EXPERTS, K, bias=z(E, dtype=f32))
    assert seen == ([{"u", "w_gate", "bias", "w_in", "w_up", "w_out"}] if T_ else [])
