"""8-bit floating-point rows, experts and their grouped product against 64 bits.

Quantisation is exact arithmetic but for one rounding to e4m3, so that its results are compared
for equality.  A sum of n products kept in fp32 is off by at most n 2^-23 sum |a||b| (2^-23: a
matrix instruction may truncate where an fma rounds), a rounding to the output type by eps / 2.
Products with bf16 output run on the 8-bit instruction, which adds groups of 8 consecutive
products and drops of each what lies below 2^-13 of the group's largest: at most 8 2^-13 of it
for every group.
"""
import numpy as np
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
bf, f32, f64 = torch.bfloat16, torch.float32, torch.float64
E4, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module", autouse=True)
def M():
    import mixture_experts_layer_46_amd as M
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M._lib.load()
    return M


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def offs(counts, start=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + start, dtype=torch.int32)


def check(got, ref, acc, what):
    """|got - ref| <= acc + eps/2 (|ref| + acc), and NaN exactly where the reference has it."""
    got = got.cpu()
    tol = acc + torch.finfo(got.dtype).eps / 2 * (ref.abs() + acc) + 1e-38
    err = (got.to(f64) - ref).abs()
    bad = ~(err <= tol) & ~(torch.isnan(got) & torch.isnan(ref))
    if bool(bad.any()):
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at flat {i}: "
                             f"{got.flatten()[i].item()} for {ref.flatten()[i].item()} (tolerance {tol.flatten()[i].item():.3g})")


def block_exponent(amax):
    """The least e >= -127 with amax <= 448 2^e, by trying them (64 bits)."""
    e = torch.full_like(amax, -127.0)
    for _ in range(260):
        e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    return e


def to_e4m3(v):
    """|v| <= 448 in 64 bits to the nearest e4m3 number, ties to even, as its value."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def rows_ref(x):
    """(values of q, exponents [R, S] of 128-element blocks, padding 0) in 64 bits."""
    R, K = x.shape
    nb, S = -(-K // 128), -(-K // 512) * 4
    xp = torch.zeros(R, nb * 128, dtype=f64)
    xp[:, :K] = x.to(f64)
    xp = xp.view(R, nb, 128)
    e = block_exponent(xp.abs().amax(dim=2))
    q = to_e4m3(xp / torch.exp2(e)[:, :, None]).view(R, nb * 128)[:, :K]
    pad = torch.zeros(R, S, dtype=f64)
    pad[:, :nb] = e
    return q, pad


def exps(scale):
    return scale.cpu().view(torch.uint8).to(f64) - 127


QUANT = [(1, 16), (3, 112), (2, 128), (5, 144), (4, 512), (3, 528), (2, 1040), (7, 2048), (3, 4112), (2, 8208), (1000, 64), (33, 128), (31, 256), (130, 208), (17, 272)]


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,K", QUANT)
def test_quantize_rows(M, R, K, dtype):
    say("quantize_rows_fp8", R, K, dtype)
    x = rand((R, K), f32, R + K) * torch.exp2(torch.randint(-20, 20, (R, K // 16), generator=torch.Generator().manual_seed(1))
                                              .float()).repeat_interleave(16, 1)
    x = x.to(dtype)
    q, s = M.quantize_rows_fp8(x.cuda())
    assert q.dtype == E4 and s.dtype == E8
    rq, re = rows_ref(x)
    assert torch.equal(exps(s), re)
    assert torch.equal(q.cpu().to(f64), rq)


def test_quantize_borders(M):
    """Largest magnitudes at, just below and just above 448 2^e; ties between e4m3 numbers; zeros;
    the smallest and largest fp32 numbers."""
    x = torch.zeros(12, 128)
    up = lambda v: float(np.nextafter(np.float32(v), np.float32(np.inf)))
    x[0, :4] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10])           # ties to even: 16, 20; below half the smallest: 0
    x[1, 0], x[1, 1] = up(448.0), 1.0
    x[2, 0] = -448.0 * 2.0 ** -100
    x[3, 0], x[3, 1] = 3.4e38, -1e30
    x[4, 0], x[4, 1] = 2.0 ** -149, -2.0 ** -130
    x[5, 127] = 2.0 ** -126
    x[6] = torch.linspace(-448, 448, 128)
    x[7, 5] = 449.0
    x[8, :3] = torch.tensor([1.75, 1.0, 1.0625])
    x[9, :3] = torch.tensor([up(1.75), 1.0, 1.0625])
    x[10, 0] = 448.0 * 2.0 ** -127
    q, s = M.quantize_rows_fp8(x.cuda())
    rq, re = rows_ref(x)
    assert torch.equal(exps(s)[:, :1], re[:, :1])
    assert torch.equal(q.cpu().to(f64), rq)
    assert bool((s.cpu().view(torch.uint8)[:, 1:] == 127).all()), "padding"


def test_quantize_not_finite(M):
    """An infinity or a NaN spoils its own block of 128 alone."""
    x = rand((4, 512), f32, 3)
    want_q, want_s = (t.cpu().view(torch.uint8) for t in M.quantize_rows_fp8(x.cuda()))
    x[1, 130], x[2, 511] = float("inf"), float("nan")
    q, s = (t.cpu().view(torch.uint8) for t in M.quantize_rows_fp8(x.cuda()))
    want_s[1, 1], want_s[2, 3] = 255, 255
    want_q[1, 128:256], want_q[2, 384:] = 0, 0
    assert torch.equal(q, want_q) and torch.equal(s, want_s)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("E,K,N", [(1, 16, 8), (2, 128, 128), (3, 144, 136), (1, 528, 264), (2, 1040, 72), (2, 48, 1000)])
def test_quantize_experts(M, E, K, N, dtype):
    w = (rand((E, K, N), f32, K + N) * torch.exp2(torch.arange(N) % 7 - 3.0)).to(dtype)
    q, s = M.quantize_experts_fp8(w.cuda())
    nk, nn = -(-K // 128), -(-N // 128)
    wp = torch.zeros(E, nk * 128, nn * 128, dtype=f64)
    wp[:, :K, :N] = w.to(f64)
    wp = wp.view(E, nk, 128, nn, 128)
    e = block_exponent(wp.abs().amax(dim=(2, 4)))
    rq = to_e4m3(wp / torch.exp2(e)[:, :, None, :, None]).view(E, nk * 128, nn * 128)[:, :K, :N].transpose(1, 2)
    assert torch.equal(q.cpu().to(f64), rq)
    assert torch.equal(exps(s)[:, :, :nk], e.transpose(1, 2)) and bool((exps(s)[:, :, nk:] == 0).all())


def operands(R, E, K, N, seed=0, spread=3):
    """Random 8-bit operands with scales of many sizes, NaN in the padding of every row of scales."""
    g = torch.Generator().manual_seed(seed + R + 3 * K + 7 * N)
    S, nb, nk = -(-K // 512) * 4, -(-N // 128), -(-K // 128)
    xq = (torch.randn(R, K, generator=g) * 60).clamp(-448, 448).to(E4)
    wq = (torch.randn(E, N, K, generator=g) * 60).clamp(-448, 448).to(E4)
    xs = torch.randint(120 - spread, 121 + spread, (R, S), generator=g, dtype=torch.uint8)
    ws = torch.randint(117 - spread, 118 + spread, (E, nb, S), generator=g, dtype=torch.uint8)
    xs[:, nk:], ws[:, :, nk:] = 255, 255
    return xq, xs.view(E8), wq, ws.view(E8)


def open_rows(q, s, K):
    """Rows q [..., K] times the scales of their blocks, in 64 bits."""
    nk = -(-K // 128)
    f = torch.exp2(s.view(torch.uint8)[..., :nk].to(f64) - 127)
    f = torch.where(s.view(torch.uint8)[..., :nk] == 255, float("nan"), f)
    return q.to(f64) * f.repeat_interleave(128, -1)[..., :K]


def product_ref(xq, xs, wq, ws, off, dtype):
    """(product in 64 bits, what it may be off by before the rounding to dtype)"""
    R, K = xq.shape
    E, N, _ = wq.shape
    x = open_rows(xq, xs, K).cuda()
    y, m = torch.zeros(R, N, dtype=f64, device="cuda"), torch.zeros(R, N, dtype=f64, device="cuda")
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a == b:
            continue
        w = open_rows(wq[e], ws[e].view(torch.uint8).repeat_interleave(128, 0)[:N].view(E8), K).cuda()
        xa, wa = x[a:b].abs(), w.abs()
        y[a:b], m[a:b] = x[a:b] @ w.T.contiguous(), K * 2.0 ** -23 * (xa @ wa.T.contiguous())
        if dtype == bf:
            xa, wa, drop = xa.float(), wa.float(), torch.zeros(b - a, N, device="cuda")
            for k in range(0, K, 8):
                top = torch.zeros(b - a, N, device="cuda")
                for i in range(k, min(k + 8, K)):
                    top = torch.maximum(top, xa[:, i, None] * wa[None, :, i])
                drop += top
            m[a:b] += 8 * 2.0 ** -13 * drop.double()
    return y.cpu(), m.cpu()


# form, rows, groups, K, N: sizes that leave a remainder on every side, groups without rows and of one
FORMS = [("16x64 thin", f32, 1, 1, 880, 40), ("16x64 thin", f32, 2, 2, 864, 40),
         ("32x64 thin", f32, 352, 1, 1040, 784), ("32x64 thin", f32, 2219, 5, 1232, 80),
         ("64x64", f32, 4961, 1, 496, 80), ("64x64", f32, 5, 5, 528, 3304),
         ("128x128", f32, 2150, 1, 432, 1112), ("128x128", f32, 696, 5, 432, 2832),
         ("128x128", bf, 1975, 1, 432, 1160), ("128x128", bf, 634, 5, 432, 2976),
         ("256x256", bf, 2655, 1, 432, 3576), ("256x256", bf, 4543, 5, 432, 1888),
         ("32x64 thin", bf, 1, 1, 1456, 40), ("32x64 thin", bf, 2, 2, 1440, 40),
         ("64x64", bf, 1, 1, 816, 40), ("64x64", bf, 2, 2, 624, 40)]
each_form = pytest.mark.parametrize("form,dtype,R,E,K,N", FORMS, ids=lambda v: {bf: "bf16", f32: "fp32"}.get(v, str(v)))


def groups_of(R, E):
    rest = 3 if R > 100 else 0
    n = R - 2 * rest
    counts = np.full(E, n // E)
    if E > 2:
        counts[1], counts[2] = 0, 1
    counts[0] += n - counts.sum()
    return offs(counts, rest), rest


@each_form
def test_product_forms(M, form, dtype, R, E, K, N):
    say("grouped_mm_fp8", form, R, E, K, N, dtype)
    code = M._lib.MOE_F32 if dtype == f32 else M._lib.MOE_BF16
    assert M._lib.grouped_mm_form("fp8", R, E, K, N, dtype=code, cus=256) == form
    xq, xs, wq, ws = operands(R, E, K, N)
    off, rest = groups_of(R, E)
    ref, tol = product_ref(xq, xs, wq, ws, off, dtype)
    args = [t.cuda() for t in (xq, xs, wq, ws, off)]
    y = M.grouped_mm_fp8(*args, dtype=dtype)
    assert y.dtype == dtype
    check(y, ref, tol, form)
    out = torch.full((R, N), 7.0, dtype=dtype, device="cuda")
    M.grouped_mm_fp8(*args, out=out)
    assert torch.equal(out[rest:R - rest], y[rest:R - rest]) and bool((out[:rest] == 7).all() and (out[R - rest:] == 7).all())


CASES = [([1], 16, 8), ([0, 1, 0], 32, 64), ([3, 0, 0, 5, 2], 48, 72), ([15, 16, 17, 31, 32, 33], 64, 136),
         ([63, 64, 65, 1], 144, 264), ([0, 127, 128, 129], 256, 256), ([255, 256, 257, 0], 112, 512), ([320, 2, 511], 528, 264),
         ([2] * 100 + [0] * 56 + [5] * 100, 48, 40), ([0, 0, 0], 32, 16), ([1300], 1040, 328), ([1], 4112, 520)]


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_product(M, counts, K, N, dtype):
    R = sum(counts)
    xq, xs, wq, ws = operands(R, len(counts), K, N)
    off = offs(counts)
    ref, tol = product_ref(xq, xs, wq, ws, off, dtype)
    y = M.grouped_mm_fp8(*(t.cuda() for t in (xq, xs, wq, ws, off)), dtype=dtype)
    check(y, ref, tol, "product")


@pytest.mark.parametrize("form,dtype,R,E,K,N", [c for c in FORMS if c[1] == f32], ids=str)
def test_scales_of_any_size(M, form, dtype, R, E, K, N):
    """Scales whose product lies in or out of fp32's range, each row of xq with one of its own: the
    products of positive numbers against 64 bits, where they overflow infinite, where they are
    subnormal off by at most the least step for each 64 products."""
    g = torch.Generator().manual_seed(R + K)
    xq, wq = ((torch.rand(*s, generator=g) + 0.5).to(E4) for s in ((R, K), (E, N, K)))
    S = 4 * ((K + 511) // 512)
    xs = torch.randint(0, 255, (R, 1), generator=g).expand(R, S).contiguous().to(torch.uint8).view(E8)
    ws = torch.randint(0, 255, (E, (N + 127) // 128, 1), generator=g).expand(-1, -1, S).contiguous().to(torch.uint8).view(E8)
    off, _ = groups_of(R, E)
    y = M.grouped_mm_fp8(*(t.cuda() for t in (xq, xs, wq, ws, off)), dtype=dtype).double().cpu()
    ref, tol = product_ref(xq, xs, wq, ws, off, dtype)
    top = ref > torch.finfo(f32).max * 1.01
    assert bool(torch.isinf(y[top]).all())
    rest = ref < torch.finfo(f32).max * 0.99
    bad = (y - ref).abs() > tol + (K + 63) // 64 * 2.0 ** -149
    assert not bool(bad[rest].any())


@each_form
def test_not_finite_stays(M, form, dtype, R, E, K, N):
    """A NaN scale or value spoils its row; one of an expert its block of columns (scale) or its
    column (value); nothing else changes."""
    xq, xs, wq, ws = operands(R, E, K, N)
    off, rest = groups_of(R, E)
    a = [t.cuda() for t in (xq, xs, wq, ws, off)]
    clean = M.grouped_mm_fp8(*a, dtype=dtype)
    r, r2, n = rest + 1 if R > rest + 1 else 0, R - rest - 1, N - 1
    a[0].view(torch.uint8)[r, K - 1] = 0x7F
    a[1].view(torch.uint8)[r2, 0] = 255
    a[2].view(torch.uint8)[0, n, 3] = 0xFF
    y = M.grouped_mm_fp8(*a, dtype=dtype)
    bad = torch.zeros(R, N, dtype=torch.bool, device="cuda")
    bad[r], bad[r2] = True, True
    bad[int(off[0]):int(off[1]), n] = True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("off", [[5, 3, 9], [-4, 2, 100], [0, 100, 2], [9, 9, 9], [100, 100, 100], [-1, -1, -1]])
@pytest.mark.parametrize("dtype,R,K,N", [(bf, 9, 144, 136), (f32, 9, 144, 136), (bf, 700, 464, 1912), (bf, 2815, 400, 3152),
                                        (f32, 1343, 400, 488), (f32, 2150, 432, 1112)], ids=str)
def test_malformed_offsets_stay_inside(M, off, dtype, R, K, N):
    """Whatever the offsets hold, guard rows around the output keep what they held."""
    off = [v * R // 9 for v in off]
    xq, xs, wq, ws = (t.cuda() for t in operands(R, 2, K, N))
    buf = torch.full((R + 64, N), 3.0, device="cuda", dtype=dtype)
    M.grouped_mm_fp8(xq, xs, wq, ws, torch.tensor(off, dtype=torch.int32, device="cuda"), out=buf[32:32 + R])
    assert bool((buf[:32] == 3).all() and (buf[32 + R:] == 3).all())


def test_no_rows(M):
    xq, xs, wq, ws = (t.cuda() for t in operands(1, 2, 48, 24))
    q, s = M.quantize_rows_fp8(torch.zeros(0, 48, device="cuda"))
    assert q.shape == (0, 48) and s.shape == (0, 4)
    assert M.grouped_mm_fp8(q, s, wq, ws, torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 24)


def test_captured(M):
    x, off = rand((300, 528), bf, 9).cuda(), offs([100, 0, 200]).cuda()
    _, _, wq, ws = (t.cuda() for t in operands(1, 3, 528, 264))
    run = lambda: M.grouped_mm_fp8(*M.quantize_rows_fp8(x), wq, ws, off)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    for i in range(3):
        x.copy_(rand((300, 528), bf, 20 + i))
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("up", [True, False])
def test_layer(M, dtype, up):
    """forward_fp8 is its stages, and near the layer in the experts' own precision: each of the four
    roundings to e4m3 (x, w, h, w again) is off by at most 2^-4 of a value, in the norm over many
    independent ones well inside the sum 4 2^-4."""
    T, H, E, F, k = 96, 256, 8, 384, 2
    x = rand((T, H), dtype, 1).cuda()
    wg = rand((H, E), f32, 2, H ** -0.5).cuda()
    w_in, w_up, w_out = (rand(s, dtype, i, s[1] ** -0.5).cuda() for i, s in ((3, (E, H, F)), (4, (E, H, F)), (5, (E, F, H))))
    w_up = w_up if up else None
    ex = M.quantize_ffn_fp8(w_in, w_up, w_out)
    out = M.forward_fp8(x, wg, ex, k)
    _, idx, w = M.route(x, wg, k)
    g = M.permute(idx, E, x=x)
    y = M.grouped_ffn_fp8(g["x_perm"], g["offsets"], ex)
    assert torch.equal(out, M.combine(y, g["row_of_pair"], w))
    full = M.forward(x, wg, w_in, w_up, w_out, k)
    rel = float((out.double() - full.double()).norm() / full.double().norm())
    assert rel <= 4 * 2.0 ** -4, rel
