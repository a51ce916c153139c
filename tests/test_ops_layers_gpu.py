"""The training and 8-bit operators run together, as the layer uses them: the differentiable
layer against 64-bit autograd, the 8-bit layer against its formula, and the calls under
streams and captured graphs."""
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


def layer(T, H, E, F, dtype, swiglu, bias, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    d = dict(x=r(T, H).to(dtype), w_gate=r(H, E) * H ** -0.5, w_in=(r(E, H, F) * H ** -0.5).to(dtype),
             w_up=(r(E, H, F) * H ** -0.5).to(dtype) if swiglu else None,
             w_out=(r(E, F, H) * F ** -0.5).to(dtype), bias=r(E) * 0.5 if bias else None)
    return d, (r(T, H)).to(dtype)


def ref_layer(d, idx, k, keep, c, row_of_pair, flags):
    """The layer in 64 bits for given experts: per token, the weighted sum of its experts."""
    p = {n: (None if t is None else t.to(f64).requires_grad_()) for n, t in d.items()}
    T, H = p["x"].shape
    logits = p["x"] @ p["w_gate"]
    if p["bias"] is not None and not flags & 1:
        logits = logits + p["bias"]
    gates = torch.softmax(torch.gather(logits, 1, idx), dim=1)
    out = torch.zeros(T, H, dtype=f64)
    for j in range(k):
        for e in range(d["w_gate"].shape[1]):
            t = torch.nonzero((idx[:, j] == e) & (row_of_pair[:, j] >= 0)).flatten()
            if t.numel() == 0:
                continue
            xe = p["x"][t]
            a = xe @ p["w_in"][e]
            h = a * torch.sigmoid(a)
            if p["w_up"] is not None:
                h = h * (xe @ p["w_up"][e])
            h = h * keep[row_of_pair[t, j]].to(f64) * c
            out = out.index_add(0, t, (h @ p["w_out"][e]) * gates[t, j, None])
    return out, p


TRAIN = [  # T, H, E, k, F, swiglu, bias, p, capacity factor, flags, dtype
    (70, 64, 8, 2, 96, True, False, 0.0, None, 0, f32), (70, 64, 8, 2, 96, True, True, 0.1, None, 0, f32),
    (33, 72, 5, 3, 40, False, True, 0.2, None, 0, f32), (64, 64, 4, 2, 64, True, True, 0.1, 0.6, 1, f32),
    (1, 64, 8, 2, 96, True, False, 0.1, None, 0, f32), (300, 128, 8, 2, 256, True, False, 0.1, None, 0, bf),
    (500, 264, 3, 2, 328, True, True, 0.1, None, 0, bf), (64, 64, 4, 2, 64, False, True, 0.1, 0.6, 0, bf),
]


@pytest.mark.parametrize("T,H,E,k,F,swiglu,bias,p,cf,flags,dtype", TRAIN)
def test_forward_train_gradients(M, T, H, E, k, F, swiglu, bias, p, cf, flags, dtype):
    """Every gradient against 64-bit autograd of the same experts and the same mask.

    Normwise bounds.  fp32: each product of the chain is off by at most n 2^-23 sum |a||b|,
    for n <= 360 random terms below n 2^-23 sqrt(n) of its norm, 8e-4 at 360 and in practice
    its square root's share; the bar is 1e-3 for the at most seven products.  bf16: x, a, b,
    h, y, dy, dh, da, db and dx are each rounded once (2^-8 of the value), ten roundings that
    reach a gradient at worst in sum: 4e-2."""
    say(f"forward_train T={T} H={H} E={E} k={k} F={F} swiglu={swiglu} p={p} cf={cf} flags={flags} {dtype}")
    from test_ops_gpu import keep_ref
    d, dout = layer(T, H, E, F, dtype, swiglu, bias, T + H)
    g = {n: (None if t is None else t.cuda().requires_grad_()) for n, t in d.items()}
    out = M.forward_train(g["x"], g["w_gate"], g["w_in"], g["w_up"], g["w_out"], k, bias=g["bias"], dropout_p=p,
                          seed=5, step=9, flags=flags, capacity_factor=cf)
    names = [n for n, t in g.items() if t is not None]
    grads = dict(zip(names, torch.autograd.grad(out, [g[n] for n in names], dout.cuda())))
    _, idx, _ = M.route(g["x"].detach(), g["w_gate"].detach(), k, bias=None if g["bias"] is None else g["bias"].detach(),
                        flags=flags)
    cap = M.capacity_rows(cf, T, k, E)
    rop = M.permute(idx, E, capacity=cap)["row_of_pair"].view(T, k).cpu().long()
    keep, c = keep_ref(5, 9, T * k * F, p)
    ref, q = ref_layer(d, idx.cpu().long(), k, keep.view(T * k, F), c, rop, flags)
    ref.backward(dout.to(f64))
    tol = 1e-3 if dtype == f32 else 4e-2
    assert normwise(out.detach().cpu().to(f64), ref.detach()) <= tol
    for n in names:
        want = q[n].grad if q[n].grad is not None else torch.zeros_like(q[n])
        assert grads[n].dtype == g[n].dtype
        err = normwise(grads[n].cpu().to(f64), want)
        assert err <= tol, (n, err)


def test_forward_train_matches_forward(M):
    """Without dropout the differentiable layer computes the layer's forward (h and y rounded
    the same, other than gate and up before the activation: one more bf16 rounding each)."""
    say("forward_train against forward")
    for dtype, tol in ((f32, 2e-5), (bf, 2e-2)):
        d, _ = layer(300, 128, 8, 256, dtype, True, True, 1)
        g = {n: t.cuda() for n, t in d.items()}
        a = M.forward(g["x"], g["w_gate"], g["w_in"], g["w_up"], g["w_out"], 2, bias=g["bias"])
        b = M.forward_train(g["x"], g["w_gate"], g["w_in"], g["w_up"], g["w_out"], 2, bias=g["bias"])
        assert normwise(b.cpu().to(f64), a.cpu().to(f64)) <= tol


def test_forward_train_parameter_step(M):
    """A training step through .backward(): every parameter gets a finite gradient."""
    say("forward_train backward()")
    d, dout = layer(64, 64, 8, 96, bf, True, True, 2)
    g = {n: t.cuda().requires_grad_() for n, t in d.items()}
    for step in range(2):
        M.forward_train(g["x"], g["w_gate"], g["w_in"], g["w_up"], g["w_out"], 2, bias=g["bias"], dropout_p=0.1,
                        seed=1, step=step).backward(dout.cuda())
    for n, t in g.items():
        assert t.grad is not None and bool(torch.isfinite(t.grad).all()), n


def int8_layer_ref(x, idx, gates, q, E, k, swiglu, dtype):
    """The 8-bit layer in 64 bits from the same 8-bit experts, each stored tensor rounded to
    `dtype` as the path does (the quantised rows are made from the rounded ones)."""
    from test_ops_gpu import quant_ref
    out = torch.zeros(x.shape, dtype=f64)
    for j in range(k):
        for e in range(E):
            t = torch.nonzero(idx[:, j] == e).flatten()
            if t.numel() == 0:
                continue
            def mm(rows, w):
                rq, rs = quant_ref(rows)
                return ((rq.to(f64) @ w[0][e].cpu().to(f64).T) * rs.to(f64)[:, None] * w[1][e].cpu().to(f64)).to(dtype)
            a = mm(x[t], q.w_in).to(f64)
            h = a * torch.sigmoid(a)
            if swiglu:
                h = h * mm(x[t], q.w_up).to(f64)
            y = mm(h.to(dtype), q.w_out).to(f64)
            out[t] += y * gates[t, j, None].to(f64)
    return out


@pytest.mark.parametrize("T,H,E,k,F,swiglu,dtype", [(1, 64, 8, 2, 96, True, bf), (70, 144, 5, 3, 80, False, bf),
                                                   (300, 256, 8, 2, 512, True, bf), (64, 128, 4, 2, 64, True, f32)])
def test_forward_int8(M, T, H, E, k, F, swiglu, dtype):
    """The 8-bit layer against its formula.  A hidden value whose rounding to bf16 falls the
    other way (a fp32 against a 64-bit activation) moves by 2^-8 of itself, and its 8-bit
    integer by at most one step of 1/127 of its row's largest: normwise 2e-2 covers the two
    roundings of y and out and such steps; in fp32 a step is as rare and as large: 1e-2."""
    say(f"forward_int8 T={T} H={H} E={E} k={k} F={F} swiglu={swiglu} {dtype}")
    d, _ = layer(T, H, E, F, dtype, swiglu, True, T + F)
    g = {n: (None if t is None else t.cuda()) for n, t in d.items()}
    q = M.quantize_ffn(g["w_in"], g["w_up"], g["w_out"])
    out = M.forward_int8(g["x"], g["w_gate"], q, k, bias=g["bias"])
    _, idx, gates = M.route(g["x"], g["w_gate"], k, bias=g["bias"])
    ref = int8_layer_ref(d["x"], idx.cpu().long(), gates.cpu(), q, E, k, swiglu, dtype)
    assert normwise(out.cpu().to(f64), ref) <= (2e-2 if dtype == bf else 1e-2)
    # and near the layer it stands for: two quantised projections of 1/254 of the largest
    # value per term, averaged over the contraction
    full = M.forward(g["x"], g["w_gate"], g["w_in"], g["w_up"], g["w_out"], k, bias=g["bias"])
    assert normwise(out.cpu().to(f64), full.cpu().to(f64)) <= 6e-2


def _chain(M, s):
    """One pass of every operator on the tensors of s; returns the outputs."""
    y = M.grouped_mm(s["x"], s["w"], s["off"])
    h = M.gated_act(y, y, 0.1, 3, s["step"])
    da, db = M.gated_act_grad(h, y, y, 0.1, 3, s["step"])
    dx = M.grouped_mm_dx(da, s["w"], s["off"])
    dw = M.grouped_mm_dw(s["x"], da, s["off"])
    q, sc = M.quantize_rows(s["x"])
    z = M.grouped_mm_int8(q, sc, s["wq"], s["ws"], s["off"])
    d = M.dropout(z, 0.2, 4, s["step"])
    cy, cw = M.combine_grad(s["dout"], y, s["rop"], s["tw"])
    return [y, h, da, db, dx, dw, q, sc, z, d, cy, cw]


def _chain_state(M, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    counts = torch.tensor([40, 0, 300, 7, 53])
    R, K, N = 400, 256, 264
    w = (r(5, K, N) * K ** -0.5).to(bf).cuda()
    wq, ws = M.quantize_experts(w)
    off = torch.cat([torch.zeros(1), counts.cumsum(0)]).to(torch.int32).cuda()
    return dict(x=r(R, K).to(bf).cuda(), w=w, wq=wq, ws=ws, off=off, dout=r(200, N).to(bf).cuda(),
                rop=torch.randperm(R, generator=g).to(torch.int32).cuda(), tw=torch.rand(200, 2, generator=g).cuda(),
                step=torch.zeros(1, dtype=torch.int64, device="cuda"))


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_captured_graphs(M):
    """Two captured passes replayed in turn, with eager work between, give the eager results on
    new contents each time; the mask follows the step word."""
    say("captured graphs")
    s1, s2 = _chain_state(M, 1), _chain_state(M, 2)
    _chain(M, s1), _chain(M, s2)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in (s1, s2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_chain(M, s))
        graphs.append(gr)
    for i in range(4):
        for s in (s1, s2):
            s["x"].copy_(torch.randn(s["x"].shape, generator=torch.Generator().manual_seed(i)).to(bf))
            s["step"].fill_(i)
        eager = [_chain(M, s1), _chain(M, s2)]
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert _same(outs[0], eager[0]) and _same(outs[1], eager[1]), i


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
def test_captured_training_pass(M, dtype):
    """The whole layer with all its gradients in one graph: every replay, on new contents and a
    new mask, with eager passes (over leaves of their own) between, equals the eager pass."""
    say(f"captured forward_train {dtype}")
    T, H, E, k, F = 4100, 128, 8, 2, 96               # rows enough for sums over many blocks
    d, dout = layer(T, H, E, F, dtype, True, True, 3)
    dout, step = dout.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda")

    def leaves():
        return {n: t.cuda().requires_grad_() for n, t in d.items()}

    def run(g):
        out = M.forward_train(g["x"], g["w_gate"], g["w_in"], g["w_up"], g["w_out"], k, bias=g["bias"], dropout_p=0.1,
                              seed=7, step=step, capacity_factor=1.1)
        return [t.detach() for t in (out, *torch.autograd.grad(out, list(g.values()), dout))]

    run(leaves())
    torch.cuda.synchronize()
    g, gr = leaves(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        outs = run(g)
    for i in range(4):
        step.fill_(i)
        x = torch.randn(T, H, generator=torch.Generator().manual_seed(i)).to(dtype).cuda()
        e = leaves()
        with torch.no_grad():
            e["x"].copy_(x)
            g["x"].copy_(x)
        want = run(e)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert _same(outs, want), [bool(torch.equal(a, b)) for a, b in zip(outs, want)]


def test_gate_gradients_of_many_tokens(M):
    """The gate's and its bias's gradients, whose sums over the tokens are cut into groups.
    Bound: the three fp32 steps (dl, a partial sum, the sum of those) are each off by at most
    n 2^-23 of the magnitudes' sum, n <= T terms, plus 8 2^-24 for the terms themselves."""
    say("gate gradients, many tokens")
    from mixture_experts_layer_46_amd.ops import _tall_dw
    for T, K, N in ((1, 8, 8), (255, 16, 24), (513, 136, 64), (5000, 264, 8), (70001, 8, 256)):
        x, dy = torch.randn(T, K, generator=torch.Generator().manual_seed(T)), torch.randn(T, N,
                                                                                           generator=torch.Generator().manual_seed(K))
        got = _tall_dw(x.cuda(), dy.cuda()).cpu().to(f64)
        a, b = x.to(f64), dy.to(f64)
        assert got.shape == (K, N)
        assert bool(((got - a.T @ b).abs() <= T * 2.0 ** -23 * (a.abs().T @ b.abs())).all()), (T, K, N)


def test_two_streams(M):
    """The operators need no workspace: passes on two streams at once do not disturb each other."""
    say("two streams")
    s1, s2 = _chain_state(M, 3), _chain_state(M, 4)
    want = [_chain(M, s1), _chain(M, s2)]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        with torch.cuda.stream(a):
            g1 = _chain(M, s1)
        with torch.cuda.stream(b):
            g2 = _chain(M, s2)
        torch.cuda.synchronize()
        got.append((g1, g2))
    for g1, g2 in got:
        assert _same(g1, want[0]) and _same(g2, want[1])


def test_many_rows_past_32_bits(M):
    """Row offsets past 2^32 bytes: the last rows of a tall activation, a tall product and a
    tall dropout are right."""
    say("past 32 bits")
    R, K, N = 530000, 4096, 8                      # x: 4.3 GB
    x = torch.empty((R, K), dtype=bf, device="cuda").normal_()
    w = torch.empty((2, K, N), dtype=bf, device="cuda").normal_()
    dy = torch.empty((R, N), dtype=bf, device="cuda").normal_()
    off = torch.tensor([0, R - 100, R], dtype=torch.int32, device="cuda")
    tail = torch.tensor([0, 0, 100], dtype=torch.int32, device="cuda")
    # the rows alone may take another form of the kernel, whose sums run in another order: the
    # float products are held to the 64-bit ones, by the bounds of the products' own tests
    from test_ops_gpu import check
    xt, dyt, w1 = x[-100:].cpu().to(f64), dy[-100:].cpu().to(f64), w[1].cpu().to(f64)
    y = M.grouped_mm(x, w, off)
    check(y[-100:], xt @ w1, K * 2.0 ** -23 * (xt.abs() @ w1.abs()), "y")
    dx = M.grouped_mm_dx(dy, w, off)
    check(dx[-100:], dyt @ w1.T, N * 2.0 ** -23 * (dyt.abs() @ w1.T.abs()), "dx")
    dw = M.grouped_mm_dw(x, dy, off)
    check(dw[1], xt.T @ dyt, 100 * 2.0 ** -23 * (xt.T.abs() @ dyt.abs()), "dw")
    q, s = M.quantize_rows(x)
    q2, s2 = M.quantize_rows(x[-100:].contiguous())
    assert torch.equal(q[-100:], q2) and torch.equal(s[-100:], s2)
    wq, ws = M.quantize_experts(w)
    z = M.grouped_mm_int8(q, s, wq, ws, off)
    assert torch.equal(z[-100:], M.grouped_mm_int8(q2, s2, wq, ws, tail))
    d = M.dropout(x, 0.1, 1, 2)
    n = 64 * K                                     # the mask goes by the element's index
    i = x.numel() - n
    import numpy as np
    blocks = np.arange(i // 8, (i + n) // 8, dtype=np.uint64)
    assert int(blocks[0]) * 8 > 1 << 31
    keep = torch.from_numpy(_philox_at(blocks, 1, 2).reshape(-1) >= round(0.1 * 65536))
    tail_d = d.view(-1)[i:].cpu()
    assert torch.equal(tail_d != 0, keep & (x.view(-1)[i:].cpu() != 0))


def _philox_at(b, seed, step):
    import numpy as np
    u = np.uint64
    m32 = u(0xFFFFFFFF)
    c = [b & m32, b >> u(32), np.full_like(b, step), np.zeros_like(b)]
    k = [seed, 0]
    for _ in range(10):
        p0, p1 = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(p1 >> u(32)) ^ c[1] ^ u(k[0]), p1 & m32, (p0 >> u(32)) ^ c[3] ^ u(k[1]), p0 & m32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    w = np.stack(c, 1)
    return np.stack([w & u(0xFFFF), w >> u(16)], 2).reshape(-1, 8)
