"""The norms around a block and their gradients against the formulas in 64 bits.

Tolerances: with e = 2^-24, a row's sum of squares (a few sequential terms per lane, then a
tree over lanes and wavefronts: less than 24 additions deep, all terms positive) is off by at
most 24 e, its root's reciprocal by half of that and 2 e of its own, and every product or sum
after it by e: K = 32 e of the magnitudes that enter covers y.  An error of y of K M, M = |scale x|
+ |gate v|, moves r(y) by K rms(M) / rms(y) = K rho of its value.  A gradient takes two such
steps and a sum over the row of signed terms, whose magnitudes are added: 3 K (1 + rho) of the
magnitudes.  Sums over T rows add T e.  Each output is rounded once, eps / 2.
"""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
bf, f32, f64 = torch.bfloat16, torch.float32, torch.float64
E24 = 2.0 ** -24
K = 32 * E24


@pytest.fixture(scope="module", autouse=True)
def M():
    import mixture_experts_layer_46_amd as M
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M._lib.load()
    return M


def half_eps(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, ref, acc, what):
    """|got - ref| <= acc + eps/2 (|ref| + acc), and NaN exactly where the reference has it."""
    got = got.cpu()
    assert got.shape == ref.shape, what
    tol = acc + half_eps(got.dtype) * (ref.abs() + acc) + 1e-38
    err = (got.to(f64) - ref).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at flat {i}: "
                             f"{got.flatten()[i].item()} for {ref.flatten()[i].item()} (tolerance {tol.flatten()[i].item():.3g})")


def make(T, H, dtype, post, gate, nxt, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + T * 7 + H)
    r = lambda *s: torch.randn(*s, generator=g)
    d = dict(x=(r(T, H) * torch.exp(0.5 * r(H))).to(dtype), z=(0.3 * r(T, H)).to(dtype), dy=r(T, H).to(dtype),
             du=r(T, H).to(dtype) if nxt else None, w_post=1 + 0.2 * r(H) if post else None,
             w_next=1 + 0.2 * r(H) if nxt else None,
             gate=0.5 * r(H) if gate == "channel" else 0.2 + torch.rand(T, 1, generator=g) if gate == "token" else None)
    return d


def formulas(d, scale, eps=1e-6):
    """Every output in 64 bits, and the magnitude that its error is held to."""
    v = {k: None if t is None else t.to(f64) for k, t in d.items()}
    x, z, w1, gate, w2 = (v[k] for k in ("x", "z", "w_post", "gate", "w_next"))
    T, H = x.shape
    one = torch.ones(1, 1, dtype=f64)
    gate_ = one if gate is None else gate
    w1_ = one if w1 is None else w1
    out, mag = {}, {}
    rz = one
    y, m = scale * x, (scale * x).abs()
    if z is not None:
        if w1 is not None:
            rz = 1 / torch.sqrt((z * z).mean(1, keepdim=True) + eps)
        zh = z * rz
        vv = zh * w1_
        y = y + gate_ * vv
        m = m + (gate_ * vv).abs()
        out["y"], mag["y"] = y, K * m
    g = v["dy"] if v["dy"] is not None else torch.zeros_like(x)
    gm, rho = g.abs(), torch.zeros(T, 1, dtype=f64)
    if w2 is not None:
        ry = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        yh, mh = y * ry, m * ry
        rho = (m * m).mean(1, keepdim=True).sqrt() * ry
        out["u"], mag["u"] = yh * w2, K * (mh * w2.abs() + (yh * w2).abs() * (1 + rho))
        if v["du"] is not None:
            t = v["du"] * w2
            g = g + ry * (t - yh * (t * yh).mean(1, keepdim=True))
            gm = gm + ry * (t.abs() + mh * (t.abs() * mh).mean(1, keepdim=True))
            out["dw_next"] = (v["du"] * yh).sum(0)
            mag["dw_next"] = ((3 * K * (1 + rho) + T * E24) * v["du"].abs() * mh).sum(0)
    f = 3 * K * (1 + rho)
    out["dx"], mag["dx"] = scale * g, f * abs(scale) * gm
    if z is not None:
        p, pm = g * gate_ * w1_, gm * (gate_ * w1_).abs()
        if w1 is None:
            out["dz"], mag["dz"] = p, f * pm
        else:
            out["dz"] = rz * (p - zh * (p * zh).mean(1, keepdim=True))
            mag["dz"] = 2 * f * rz * (pm + zh.abs() * (pm * zh.abs()).mean(1, keepdim=True))
            out["dw_post"] = (g * gate_ * zh).sum(0)
            mag["dw_post"] = ((f + T * E24) * gm * (gate_ * zh).abs()).sum(0)
        if gate is not None:
            dim = 0 if gate.dim() == 1 else 1
            out["dgate"] = (g * vv).sum(dim, keepdim=dim == 1)
            mag["dgate"] = ((2 * f + T * E24) * gm * vv.abs()).sum(dim, keepdim=dim == 1)
    return out, mag


def gpu(d):
    return {k: None if t is None else t.cuda() for k, t in d.items()}


# one row; rows of one chunk; around a wavefront's, a workgroup's and two chunks' lengths; more rows
# than workgroups; odd counts
SIZES = [(1, 8), (3, 64), (9, 504), (5, 512), (4, 520), (7, 1032), (2, 4096), (3, 8192), (2, 8200), (1, 16384), (260, 12288), (259, 12296), (3, 10240), (2100, 256),
         (1300, 1048), (1030, 520)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("post,gate,nxt", [(True, "channel", True), (True, "token", True), (False, None, True),
                                           (True, None, False), (False, "channel", False), (False, "token", True),
                                           (False, None, False)])
def test_residual_norm_and_gradient(M, T, H, dtype, post, gate, nxt):
    say("residual_norm", T, H, dtype, post, gate, nxt)
    d = make(T, H, dtype, post, gate, nxt)
    ref, tol = formulas(d, 0.75)
    c = gpu(d)
    args = (c["x"], c["z"], c["w_post"], c["gate"], 0.75, c["w_next"])
    y, u = M.residual_norm(*args)
    check(y, ref["y"], tol["y"], "y")
    if nxt:
        check(u, ref["u"], tol["u"], "u")
    else:
        assert u is None
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


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
def test_rows_apart(M, dtype):
    """x and z as the halves of a packed tensor."""
    d = make(37, 264, dtype, True, "channel", True)
    ref, tol = formulas(d, 1.25)
    c = gpu(d)
    packed = torch.cat([c["x"], c["z"]], dim=1)
    x, z = packed[:, :264], packed[:, 264:]
    y, u = M.residual_norm(x, z, c["w_post"], c["gate"], 1.25, c["w_next"])
    check(y, ref["y"], tol["y"], "y")
    check(u, ref["u"], tol["u"], "u")
    for name, t in zip(("dx", "dz", "dw_post", "dgate", "dw_next"),
                       M.residual_norm_grad(c["dy"], c["du"], x, z, c["w_post"], c["gate"], 1.25, c["w_next"])):
        check(t, ref[name], tol[name], name)


@pytest.mark.parametrize("H", [256, 1032])
def test_no_rows(M, H):
    z = lambda *s: torch.zeros(*s, device="cuda")
    w = z(H) + 1
    x = z(0, H)
    y, u = M.residual_norm(x, x, w, w, 1.0, w)
    assert y.shape == u.shape == (0, H)
    dx, dz, d1, dg, d2 = M.residual_norm_grad(x, x, x, x, w, w, 1.0, w)
    assert dx.shape == dz.shape == (0, H) and not bool(d1.any() or dg.any() or d2.any())
    dx, dz, d1, dg, d2 = M.residual_norm_grad(x, x, x, x, w, z(0, 1), 1.0, w)
    assert dg.shape == (0, 1) and not bool(d1.any() or d2.any())


def test_rows_of_zeros_and_non_finite_rows(M):
    """A row of zeros is zeros; a row with an infinity or a NaN does not reach its neighbours."""
    d = make(12, 520, f32, True, "channel", True)
    d["z"][3] = 0.0
    d["x"][3] = 0.0
    clean, _ = M.residual_norm(*(gpu(d)[k] for k in ("x", "z", "w_post", "gate")), 0.5, d["w_next"].cuda())
    bad = {k: None if t is None else t.clone() for k, t in d.items()}
    bad["z"][5, 7] = float("inf")
    bad["x"][8, 9] = float("nan")
    c, o = gpu(bad), gpu(d)
    keep = [i for i in range(12) if i not in (5, 8)]
    for s in (c, o):
        s["out"] = M.residual_norm(s["x"], s["z"], s["w_post"], s["gate"], 0.5, s["w_next"])
        s["grad"] = M.residual_norm_grad(s["dy"], s["du"], s["x"], s["z"], s["w_post"], s["gate"], 0.5, s["w_next"])
    for a, b in zip(c["out"] + c["grad"][:2], o["out"] + o["grad"][:2]):
        assert torch.equal(a[keep], b[keep])
    assert bool((o["out"][0][3] == 0).all()) and bool((o["out"][1][3] == 0).all())
    assert torch.isnan(c["out"][0][5]).any() and torch.isnan(c["out"][1][8]).all()


@pytest.mark.parametrize("gate", ["channel", "token"])
def test_autograd(M, gate):
    """Through autograd, with gradients of y or u alone, and of views at odd addresses."""
    d = make(33, 136, f32, True, gate, True)
    names = ("x", "z", "w_post", "gate", "w_next")
    for dy, du in ((True, True), (True, False), (False, True)):
        e = dict(d, dy=d["dy"] if dy else None, du=d["du"] if du else torch.zeros_like(d["du"]))
        ref, tol = formulas(e, 0.5)
        c = {k: t.cuda().requires_grad_(k in names) for k, t in d.items()}
        y, u = M.residual_norm(c["x"], c["z"], c["w_post"], c["gate"], 0.5, c["w_next"])
        odd = torch.zeros(33 * 136 + 1, device="cuda")[1:].view(33, 136).copy_(d["dy"])
        outs = ([y] if dy else []) + ([u] if du else [])
        grads = torch.autograd.grad(outs, [c[k] for k in names], ([odd] if dy else []) + ([c["du"].detach()] if du else []))
        for name, t in zip(names, grads):
            key = {"x": "dx", "z": "dz", "gate": "dgate"}.get(name, "d" + name)
            check(t, ref[key], tol[key], key)


def test_gradient_against_differences(M):
    """The forward's own differences along a direction: with step h the third derivative leaves
    O(h^2) of the loss's scale, fp32 rounding 2^-23 |loss terms| / h."""
    d = make(6, 264, f32, True, "channel", True)
    c = gpu(d)
    names = ("x", "z", "w_post", "gate", "w_next")
    g = torch.Generator().manual_seed(5)
    for name, grad in zip(names, M.residual_norm_grad(c["dy"], c["du"], c["x"], c["z"], c["w_post"], c["gate"], 0.75, c["w_next"])):
        way = torch.randn(d[name].shape, generator=g).cuda()
        h, terms = 2.0 ** -7, 0.0
        loss = []
        for sign in (1, -1):
            e = dict(c)
            e[name] = c[name] + sign * h * way
            y, u = M.residual_norm(e["x"], e["z"], e["w_post"], e["gate"], 0.75, e["w_next"])
            t = torch.cat([y.double() * c["dy"], u.double() * c["du"]])
            loss.append(t.sum())
            terms = float(t.abs().sum())
        slope, want = float((loss[0] - loss[1]) / (2 * h)), float((grad.double() * way).sum())
        bound = 2.0 ** -23 * terms / h + 30 * h * h * float((grad.double() * way).abs().sum())
        assert abs(slope - want) <= bound, (name, slope, want, bound)


def test_given_outputs_and_streams(M):
    d = make(64, 512, bf, True, "channel", True)
    c = gpu(d)
    args = (c["x"], c["z"], c["w_post"], c["gate"], 0.75, c["w_next"])
    y, u = M.residual_norm(*args)
    yo, uo = torch.full_like(y, float("nan")), torch.full_like(u, float("nan"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        M.residual_norm(*args, out=(yo, uo))
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, yo) and torch.equal(u, uo)


def test_captured(M):
    d = make(700, 1032, bf, True, "channel", True)
    c = gpu(d)
    args = (c["x"], c["z"], c["w_post"], c["gate"], 0.75, c["w_next"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        M.residual_norm_grad(c["dy"], c["du"], *args)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = M.residual_norm(*args)
        grads = M.residual_norm_grad(c["dy"], c["du"], *args)
    for i in range(3):
        c["x"].copy_(make(700, 1032, bf, True, "channel", True, seed=i + 1)["x"])
        want = M.residual_norm(*args) + M.residual_norm_grad(c["dy"], c["du"], *args)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out + grads, want):
            assert torch.equal(a, b)
