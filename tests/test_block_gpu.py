"""Blocks as they are used: norms, routing, the gated half, the experts' products, the combine
and the residual norm in a chain, trained and served.

Tolerances, normwise (largest difference over largest value): fp32: each of the at most ten
stages of a block sums n <= 128 random terms in fp32, off by at most n 2^-23 of its magnitudes,
two blocks and their gradients: 40 stages, 40 * 128 * 2^-23 / sqrt(128) (random signs) = 6e-5;
the bar is 1e-3 as for the layer.  bf16: every stored tensor is rounded once, 2^-9 of the value
at worst half a step; ten stored tensors a block forward, as many back: 40 roundings, 40 2^-9 in
the worst sum, 8e-2.
"""
import pytest
import torch

from gpu_util import normwise, say

pytestmark = pytest.mark.gpu
bf, f32, f64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def M():
    import mixture_experts_layer_46_amd as M
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M._lib.load()
    return M


def block(H, E, F, dtype, swiglu, gate, T, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return dict(w_gate=r(H, E) * H ** -0.5, w_in=(r(E, H, F) * H ** -0.5).to(dtype),
                w_up=(r(E, H, F) * H ** -0.5).to(dtype) if swiglu else None, w_out=(r(E, F, H) * F ** -0.5).to(dtype),
                w_post=1 + 0.1 * r(H), w_next=1 + 0.1 * r(H),
                gate=0.5 + 0.1 * r(H) if gate == "channel" else 0.5 + 0.1 * r(T, 1) if gate == "token" else None)


def ref_norm(t, w, eps=1e-6):
    return t / torch.sqrt((t * t).mean(1, keepdim=True) + eps) * w


def ref_block(x, u, p, idx, k):
    logits = u @ p["w_gate"]
    gates = torch.softmax(torch.gather(logits, 1, idx), dim=1)
    z = torch.zeros_like(x)
    for j in range(k):
        for e in range(p["w_gate"].shape[1]):
            t = torch.nonzero(idx[:, j] == e).flatten()
            a = u[t] @ p["w_in"][e]
            h = a * torch.sigmoid(a)
            if p["w_up"] is not None:
                h = h * (u[t] @ p["w_up"][e])
            z = z.index_add(0, t, (h @ p["w_out"][e]) * gates[t, j, None])
    y = 0.9 * x + (1.0 if p["gate"] is None else p["gate"]) * ref_norm(z, p["w_post"])
    return y, ref_norm(y, p["w_next"])


@pytest.mark.parametrize("T,H,E,k,F,swiglu,gate,dtype", [
    (60, 64, 4, 2, 96, True, "channel", f32), (1, 72, 4, 2, 40, True, "token", f32), (33, 128, 5, 3, 64, False, None, f32),
    (60, 64, 4, 2, 96, True, "channel", bf), (130, 128, 8, 2, 128, True, "token", bf)])
def test_two_blocks_trained(M, T, H, E, k, F, swiglu, gate, dtype):
    """Every gradient of two blocks in a row against 64-bit autograd with the same experts chosen."""
    say("two blocks", T, H, E, k, F, swiglu, gate, dtype)
    g = torch.Generator().manual_seed(T)
    x0, w0 = torch.randn(T, H, generator=g).to(dtype), 1 + 0.1 * torch.randn(H, generator=g)
    dy, du = torch.randn(T, H, generator=g).to(dtype), torch.randn(T, H, generator=g).to(dtype)
    blocks = [block(H, E, F, dtype, swiglu, gate, T, s) for s in (1, 2)]
    leaf = lambda t, f: None if t is None else f(t).requires_grad_()
    gp = [{n: leaf(t, lambda v: v.cuda()) for n, t in b.items()} for b in blocks]
    gx, gw = x0.cuda().requires_grad_(), w0.cuda().requires_grad_()
    x, u, chosen = gx, M.norm(gx, gw), []
    for p in gp:
        chosen.append(M.route(u.detach(), p["w_gate"].detach(), k)[1].cpu().long())
        x, u = M.forward_block(x, u, p["w_gate"], (p["w_in"], p["w_up"], p["w_out"]), k, p["w_post"], p["gate"], 0.9, p["w_next"])
    leaves = [gx, gw] + [t for p in gp for t in p.values() if t is not None]
    grads = torch.autograd.grad((x, u), leaves, (dy.cuda(), du.cuda()))
    rp = [{n: leaf(t, lambda v: v.to(f64)) for n, t in b.items()} for b in blocks]
    rx, rw = x0.to(f64).requires_grad_(), w0.to(f64).requires_grad_()
    a, b = rx, ref_norm(rx, rw)
    for p, idx in zip(rp, chosen):
        a, b = ref_block(a, b, p, idx, k)
    refs = [rx, rw] + [t for p in rp for t in p.values() if t is not None]
    want = torch.autograd.grad((a, b), refs, (dy.to(f64), du.to(f64)))
    tol = 1e-3 if dtype == f32 else 8e-2
    assert normwise(x.detach().cpu().to(f64), a.detach()) <= tol and normwise(u.detach().cpu().to(f64), b.detach()) <= tol
    for i, (got, w) in enumerate(zip(grads, want)):
        assert got.dtype == leaves[i].dtype
        assert normwise(got.cpu().to(f64), w) <= tol, i


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["full", "int8", "fp8"])
def test_served(M, kind, dtype):
    """The served block is the layer and the norm one after the other, bit by bit."""
    T, H, E, k, F = 50, 256, 4, 2, 128
    p = {n: None if t is None else t.cuda() for n, t in block(H, E, F, dtype, True, "channel", T, 3).items()}
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    u = M.norm(x, p["w_post"])
    ex = (p["w_in"], p["w_up"], p["w_out"])
    if kind == "full":
        z = M.forward(u, p["w_gate"], *ex, k)
    else:
        ex = (M.quantize_ffn if kind == "int8" else M.quantize_ffn_fp8)(*ex)
        z = (M.forward_int8 if kind == "int8" else M.forward_fp8)(u, p["w_gate"], ex, k)
    want = M.residual_norm(x, z, p["w_post"], p["gate"], 0.5, p["w_next"])
    got = M.forward_block(x, u, p["w_gate"], ex, k, p["w_post"], p["gate"], 0.5, p["w_next"])
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_captured_training_block(M):
    """A block and its gradients captured, replayed with eager work in between."""
    T, H, E, k, F = 200, 128, 8, 2, 256
    p = {n: None if t is None else t.cuda().requires_grad_() for n, t in block(H, E, F, bf, True, "channel", T, 5).items()}
    r = lambda s: torch.randn(T, H, generator=torch.Generator().manual_seed(s)).to(bf).cuda()
    x, dy, du = r(1).requires_grad_(), r(2), r(3)
    w0 = torch.ones(H, device="cuda")
    leaves = [x] + [t for t in p.values() if t is not None]

    def run():
        y, u = M.forward_block(x, M.norm(x, w0), p["w_gate"], (p["w_in"], p["w_up"], p["w_out"]), k, p["w_post"], p["gate"],
                               0.9, p["w_next"])
        return [t.detach() for t in (y, u, *torch.autograd.grad((y, u), leaves, (dy, du)))]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        with torch.no_grad():
            x.copy_(r(10 + i))
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["full", "int8", "fp8"])
def test_no_tokens_served(M, kind):
    p = {n: None if t is None else t.cuda() for n, t in block(64, 4, 96, bf, True, "channel", 0, 6).items()}
    x = torch.zeros(0, 64, dtype=bf, device="cuda")
    ex = (p["w_in"], p["w_up"], p["w_out"])
    if kind != "full":
        ex = (M.quantize_ffn if kind == "int8" else M.quantize_ffn_fp8)(*ex)
    y, u = M.forward_block(x, x, p["w_gate"], ex, 2, p["w_post"], p["gate"], 1.0, p["w_next"])
    assert y.shape == u.shape == (0, 64)
