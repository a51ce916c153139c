"""A trained block against the chain of the public operators that it stands for, outputs and
gradients bit for bit: each operator is held to 64 bits by its own tests, this holds how they are
joined far closer than a tolerance of the whole block can.

Only the router's part meets sums of its own: u's gradient is one rounded term of the permute's and
one of the gate's, added and rounded, eps / 2 each; the gate's products are n fp32 terms, off by at
most n 2^-23 of their magnitudes.
"""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
bf, f32, f64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def M():
    import mixture_experts_layer_46_amd as M
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M._lib.load()
    return M


def within(got, ref, tol):
    assert bool(((got.to(f64) - ref).abs() <= tol).all()), float(((got.to(f64) - ref).abs() - tol).max())


@pytest.mark.parametrize("capacity", [None, 1.0])
@pytest.mark.parametrize("T,H,E,k,F,gate", [(1, 64, 4, 2, 96, None), (333, 256, 8, 2, 384, "channel"), (500, 136, 5, 3, 72, "token")])
@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
def test_trained_block_is_its_chain(M, T, H, E, k, F, gate, dtype, capacity):
    say("chain", T, H, E, k, F, gate, dtype, capacity)
    g = torch.Generator().manual_seed(T + H)
    r = lambda *s, f=1.0, t=dtype: (torch.randn(*s, generator=g) * f).to(t).cuda()
    x, u, dy, du = (r(T, H) for _ in range(4))
    wg = r(H, E, f=H ** -0.5, t=f32)
    w_in, w_up, w_out = r(E, H, F, f=H ** -0.5), r(E, H, F, f=H ** -0.5), r(E, F, H, f=F ** -0.5)
    w_post, w_next = 1 + r(H, f=0.1, t=f32), 1 + r(H, f=0.1, t=f32)
    gate = r(H, f=0.5, t=f32) if gate == "channel" else 0.5 + r(T, 1, f=0.1, t=f32) if gate == "token" else None

    leaves = [None if t is None else t.clone().requires_grad_() for t in (x, u, wg, w_in, w_up, w_out, w_post, gate, w_next)]
    lx, lu, lg, li, lp, lo, l1, lt, l2 = leaves
    out = M.forward_block(lx, lu, lg, (li, lp, lo), k, l1, lt, 0.9, l2, capacity_factor=capacity)
    grads = iter(torch.autograd.grad(out, [t for t in leaves if t is not None], (dy, du)))
    dx_, du_, dwg_, di_, dp_, do_, d1_, dt_, d2_ = (None if t is None else next(grads) for t in leaves)

    _, idx, w = M.route(u, wg, k)
    rows = 0 if capacity is None else M.capacity_rows(capacity, T, k, E)
    p = M.permute(idx, E, x=u, capacity=rows)
    xp, off, where = p["x_perm"], p["offsets"], p["row_of_pair"]
    assert (rows == 0 or T == 1) == bool((where >= 0).all()), "the capacity drops pairs"
    h, a, b = M.gated._gated(xp, w_in, w_up, off, None, True)
    yp = M.grouped_mm(h, w_out, off)
    z = M.combine(yp, where, w)
    for got, want in zip(out, M.residual_norm(x, z, w_post, gate, 0.9, w_next)):
        assert torch.equal(got, want)

    dx, dz, d1, dt, d2 = M.residual_norm_grad(dy, du, x, z, w_post, gate, 0.9, w_next)
    dyp, dw = M.combine_grad(dz, yp, where, w)
    d_out = M.grouped_mm_dw(h, dyp, off)
    dxp, d_in, d_up = M.gated_mm_grad(M.grouped_mm_dx(dyp, w_out, off), xp, w_in, w_up, a, b, off)
    for name, got, want in (("x", dx_, dx), ("w_in", di_, d_in), ("w_up", dp_, d_up), ("w_out", do_, d_out), ("w_post", d1_, d1),
                            ("gate", dt_, dt), ("w_next", d2_, d2)):
        assert (got is None and want is None) or torch.equal(got, want), name

    # the softmax's gradient: a few fp32 operations on each number
    w64, dw64 = w.to(f64), dw.to(f64)
    dl, ml = torch.zeros(T, E, dtype=f64, device="cuda"), torch.zeros(T, E, dtype=f64, device="cuda")
    dl.scatter_(1, idx.long(), w64 * (dw64 - (w64 * dw64).sum(1, keepdim=True)))
    ml.scatter_(1, idx.long(), w64 * (dw64.abs() + (w64 * dw64).abs().sum(1, keepdim=True)))
    few = (k + 4) * 2.0 ** -24
    u64, wg64 = u.to(f64), wg.to(f64)
    within(dwg_, u64.T.contiguous() @ dl, (T * 2.0 ** -23 + few) * (u64.abs().T.contiguous() @ ml) + 1e-38)
    half = torch.finfo(dtype).eps / 2
    ones = torch.ones(T, k, device="cuda")
    first, second = M.combine(dxp, where, ones).to(f64), dl @ wg64.T.contiguous()
    acc = ((E + 8) * 2.0 ** -23 + few) * (ml @ wg64.abs().T.contiguous())
    acc = acc + half * (second.abs() + acc)
    within(du_, first + second, acc + half * ((first + second).abs() + acc) + 1e-38)
