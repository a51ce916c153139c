"""The norms and their gradients with more rows than a launch has places for, at every shape of their
kernels, so that each workgroup goes round several times; parameters' gradients over all those
rows.  Formulas and tolerances are those of test_norms_gpu.py.
"""
import pytest
import torch

from gpu_util import say
from test_norms_gpu import check, formulas, gpu, make

pytestmark = pytest.mark.gpu
bf, f32, f64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def M():
    import mixture_experts_layer_46_amd as M
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M._lib.load()
    return M


# on 256 CUs: forward 4 rows a workgroup of 256 threads to 512 columns, else a row each, 1024 threads
# a CU; gradient 512 workgroups of up to 512 threads to 4096 columns, else 256
SIZES = [(4500, 64), (9001, 512), (5000, 520), (1500, 2056), (1100, 4096), (600, 4104), (700, 8192), (530, 9224), (517, 16384)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("post,gate,nxt", [(True, "channel", True), (False, "token", True)])
def test_residual_norm_and_gradient(M, T, H, dtype, post, gate, nxt):
    say("residual_norm", T, H, dtype, post, gate, nxt)
    d = make(T, H, dtype, post, gate, nxt)
    ref, tol = formulas(d, 0.75)
    c = gpu(d)
    args = (c["x"], c["z"], c["w_post"], c["gate"], 0.75, c["w_next"])
    for name, t in zip(("y", "u"), M.residual_norm(*args)):
        check(t, ref[name], tol[name], name)
    got = M.residual_norm_grad(c["dy"], c["du"], *args)
    for name, t in zip(("dx", "dz", "dw_post", "dgate", "dw_next"), got):
        if name in ref:
            check(t, ref[name], tol[name], name)
        else:
            assert t is None, name
    again = M.residual_norm_grad(c["dy"], c["du"], *args)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again)), "the same call, other bits"


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
def test_norm_and_gradient(M, T, H, dtype):
    say("norm", T, H, dtype)
    d = make(T, H, dtype, False, None, True)
    d["z"] = d["dy"] = None
    ref, tol = formulas(d, 1.0)
    c = gpu(d)
    check(M.norm(c["x"], c["w_next"]), ref["u"], tol["u"], "u")
    dx, dw = M.norm_grad(c["du"], c["x"], c["w_next"])
    check(dx, ref["dx"], tol["dx"], "dx")
    check(dw, ref["dw_next"], tol["dw_next"], "dw")
