"""The differentiable operators inside larger autograd programs: what the engine hands to their
backward passes, and what they leave behind for it."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def M():
    import mixture_experts_layer_46_amd as M
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M._lib.load()
    return M


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def _layer(dtype, T=64, H=64, E=4, F=64):
    return dict(x=rand((T, H), dtype, 1), w_gate=rand((H, E), f32, 2, H ** -0.5), w_in=rand((E, H, F), dtype, 3, H ** -0.5),
                w_up=rand((E, H, F), dtype, 4, H ** -0.5), w_out=rand((E, F, H), dtype, 5, F ** -0.5),
                bias=rand((E,), f32, 6))


def _train(M, d, dout, **kw):
    g = {n: t.clone().requires_grad_() for n, t in d.items()}
    out = M.forward_train(g["x"], g["w_gate"], g["w_in"], g["w_up"], g["w_out"], 2, bias=g["bias"], dropout_p=0.1, seed=3,
                          **kw)
    return [out.detach(), *torch.autograd.grad(out, list(g.values()), dout)]


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
def test_dropped_pairs_leave_no_unset_gradients(M, dtype, monkeypatch):
    """Rows that a capacity left without a pair get a gradient of zeros: torch's anomaly
    detection, which looks at whole gradients, finds no stray NaN of unwritten memory there."""
    say(f"anomaly detection, dropped pairs {dtype}")
    d, dout = _layer(dtype), rand((64, 64), dtype, 7)
    want = _train(M, d, dout, capacity_factor=0.6)
    empty_like = torch.empty_like
    monkeypatch.setattr(torch, "empty_like",
                        lambda t, **kw: empty_like(t, **kw).fill_(float("nan")) if t.is_floating_point() else empty_like(t, **kw))
    with torch.autograd.detect_anomaly(check_nan=True):
        got = _train(M, d, dout, capacity_factor=0.6)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def _shifted(y, dy):
    """y's gradient dy as the engine hands it over behind a concatenation: a dense view that
    starts one element into its storage."""
    flat = torch.cat([torch.zeros(1, dtype=y.dtype, device=y.device), y.reshape(-1)])
    return flat, torch.cat([torch.zeros(1, dtype=dy.dtype, device=dy.device), dy.reshape(-1)])


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
def test_gradients_at_any_address(M, dtype):
    """Gradients that are views off the kernels' 16 bytes (slices of a concatenation's or a
    stack's gradient) give the same results as aligned ones."""
    say(f"misaligned gradients {dtype}")
    R, K, N = 40, 64, 72
    off = torch.tensor([0, 25, 25, 40], dtype=torch.int32).cuda()
    x, w, dy = rand((R, K), dtype, 1), rand((3, K, N), dtype, 2, K ** -0.5), rand((R, N), dtype, 3)
    a, b = rand((R, N), dtype, 4), rand((R, N), dtype, 5)
    d = _layer(dtype)
    layer = lambda *t: M.forward_train(*t[:5], 2, bias=t[5], dropout_p=0.1, seed=3)
    for name, fn, inputs, g in (
            ("grouped_mm", lambda x, w: M.grouped_mm(x, w, off), (x, w), dy),
            ("gated_act", lambda a, b: M.gated_act(a, b, 0.1, 5, 6), (a, b), dy),
            ("dropout", lambda a: M.dropout(a, 0.1, 5, 6), (a,), dy),
            ("forward_train", layer, tuple(d.values()), rand((64, 64), dtype, 7))):
        t = [v.clone().requires_grad_() for v in inputs]
        want = torch.autograd.grad(fn(*t), t, g)
        flat, gflat = _shifted(fn(*t), g)
        got = torch.autograd.grad(flat, t, gflat)
        assert all(torch.equal(p, q) for p, q in zip(got, want)), name
    # a stack of odd tensors: the second one's gradient starts 35 elements in
    u, v = rand((5, 7), dtype, 8).requires_grad_(), rand((5, 7), dtype, 9).requires_grad_()
    g = rand((2, 5, 7), dtype, 10)
    du, dv = torch.autograd.grad(torch.stack([M.dropout(u, 0.3, 1, 1), M.dropout(v, 0.3, 1, 2)]), (u, v), g)
    assert torch.equal(du, M.dropout(g[0].clone(), 0.3, 1, 1)) and torch.equal(dv, M.dropout(g[1].clone(), 0.3, 1, 2))


def test_given_outputs_count_as_written(M):
    """A tensor written through `out` counts as modified: a backward pass that had kept its old
    contents raises, as behind any other in-place operation, instead of using the new ones."""
    say("out and autograd's version counters")
    a, b = rand((8, 16), bf, 1).requires_grad_(), rand((8, 16), bf, 2)
    h = M.gated_act(a, b)
    with torch.no_grad():
        M.dropout(b, 0.5, 1, 2, out=b)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        h.sum().backward()
    off = torch.tensor([0, 8], dtype=torch.int32).cuda()
    x, w, dy = rand((8, 16), bf, 3), rand((1, 16, 24), bf, 4), rand((8, 24), bf, 5)
    q, s = M.quantize_rows(x)
    wq, ws = M.quantize_experts(w)
    gate, experts = rand((16, 2), f32, 6), M.quantize_ffn(rand((2, 16, 32), bf, 7), None, rand((2, 32, 16), bf, 8))
    e = lambda *shape: torch.empty(*shape, dtype=bf, device="cuda")
    for call, out in ((lambda o: M.grouped_mm(x, w, off, out=o), e(8, 24)), (lambda o: M.grouped_mm_dx(dy, w, off, out=o), e(8, 16)),
                      (lambda o: M.grouped_mm_dw(x, dy, off, out=o), e(1, 16, 24)),
                      (lambda o: M.grouped_mm_int8(q, s, wq, ws, off, out=o), e(8, 24)),
                      (lambda o: M.dropout(x, 0.1, 1, out=o), e(8, 16)), (lambda o: M.gated_act(x, x, out=o), e(8, 16)),
                      (lambda o: M.gated_act_grad(x, x, b, out=(o, e(8, 16))), e(8, 16)),
                      (lambda o: M.gated_act_grad(x, x, b, out=(e(8, 16), o)), e(8, 16)),
                      (lambda o: M.forward_int8(x, gate, experts, 1, out=o), e(8, 16))):
        before = out._version
        call(out)
        assert out._version > before
    # tensors of inference mode have no counter; they are written all the same
    with torch.inference_mode():
        o = e(8, 16)
        M.dropout(x, 0.0, 1, out=o)
        assert torch.equal(o, x)


def test_activation_outputs_over_inputs_are_refused(M):
    """Refused on the host, before a launch; halves of one packed tensor are no overlap."""
    say("gated_act, overlapping outputs")
    buf = rand((8, 96), bf, 1)
    a, b, dh = buf[:, :24], buf[:, 24:48], rand((8, 24), bf, 2)
    flat = buf.view(-1)[:8 * 24].view(8, 24)
    for call, msg in ((lambda: M.gated_act(a, b, out=flat), "out overlaps a"), (lambda: M.gated_act(dh, b, out=dh), "out overlaps a"),
                      (lambda: M.gated_act_grad(dh, a, b, out=(buf[:, 48:72], buf[:, 56:80])), "db overlaps da"),
                      (lambda: M.gated_act_grad(dh, a, b, out=(dh, buf[:, 56:80])), "da overlaps dh"),
                      (lambda: M.gated_act_grad(dh, a, b, out=(buf[:, 8:32], buf[:, 56:80])), "da overlaps a"),
                      (lambda: M.gated_act_grad(dh, a, b, out=(buf[:, 56:80], buf[:, 32:56])), "db overlaps b")):
        with pytest.raises(ValueError, match=msg):
            call()
    want = M.gated_act_grad(dh, a, b)
    M.gated_act_grad(dh, a, b, out=(buf[:, 48:72], buf[:, 72:]))
    assert torch.equal(buf[:, 48:72], want[0]) and torch.equal(buf[:, 72:], want[1])
