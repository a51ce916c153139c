"""The training and 8-bit operators against plain implementations in 64 bits.

Tolerances are element by element and follow from the arithmetic: a sum of n products kept
in fp32 is off by at most n 2^-23 sum |a||b| (2^-23: a matrix instruction may truncate where
an fma rounds), a rounding to the output type by eps / 2 of the value.
"""
import numpy as np
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


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def offs(counts, start=0):
    o = np.concatenate([[0], np.cumsum(counts)]) + start
    return torch.tensor(o, dtype=torch.int32)


def half_eps(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, ref, acc, what):
    """|got - ref| <= acc + eps/2 (|ref| + acc), and NaN exactly where the reference has it."""
    got = got.cpu()
    e = half_eps(got.dtype)
    tol = acc + e * (ref.abs() + acc) + 1e-38          # below the least normal value: no relative bound
    err = (got.to(f64) - ref).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements off, first at flat {i}: "
                             f"{got.flatten()[i].item()} for {ref.flatten()[i].item()} (tolerance {tol.flatten()[i].item():.3g})")


def mm_ref(x, w, off, transposed=False):
    """(product, sum of magnitudes) in 64 bits; rows in no group are zeros."""
    x, w = x.to(f64), w.to(f64)
    J = w.shape[1] if transposed else w.shape[2]
    y, m = torch.zeros(x.shape[0], J, dtype=f64), torch.zeros(x.shape[0], J, dtype=f64)
    for e in range(w.shape[0]):
        a, b = int(off[e]), int(off[e + 1])
        we = w[e].T if transposed else w[e]
        y[a:b], m[a:b] = x[a:b] @ we, x[a:b].abs() @ we.abs()
    return y, m


def dw_ref(x, dy, off, K, N):
    E = off.numel() - 1
    d, m = torch.zeros(E, K, N, dtype=f64), torch.zeros(E, K, N, dtype=f64)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        d[e] = x[a:b].to(f64).T @ dy[a:b].to(f64)
        m[e] = x[a:b].to(f64).abs().T @ dy[a:b].to(f64).abs()
    return d, m


# counts, K, N: one row; empty groups first, last and between; rows around every tile
# height; sizes of one chunk, of part of a tile, and of several tiles with a tail
MM_CASES = [
    ([1], 8, 8), ([1], 264, 520), ([0, 1, 0], 32, 64), ([3, 0, 0, 5, 2], 40, 72),
    ([15, 16, 17, 31, 32, 33], 64, 136), ([63, 64, 65, 1], 136, 264), ([0, 127, 128, 129], 256, 256),
    ([255, 256, 257, 0], 96, 512), ([320, 2, 511], 520, 264), ([700, 1, 0, 40], 72, 1032), ([1300], 1032, 328),
    ([2] * 100 + [0] * 56 + [5] * 100, 48, 40), ([0, 0, 0], 24, 16), ([600, 0, 300, 64, 65, 16, 17, 1], 768, 776),
]
MM_IDS = [f"{sum(c)}rows-{len(c)}groups-{k}x{n}" for c, k, n in MM_CASES]


def mm_inputs(counts, K, N, dtype, tail):
    """Operands with `tail` rows of NaN before the first and behind the last group."""
    R = sum(counts)
    off = offs(counts, start=tail)
    x, dy = rand((R + 2 * tail, K), dtype, 1), rand((R + 2 * tail, N), dtype, 2)
    w = rand((len(counts), K, N), dtype, 3, K ** -0.5)
    for t in (x, dy):
        if tail:
            t[:tail] = float("nan")
            t[R + tail:] = float("nan")
    return x, dy, w, off


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tail", [0, 3])
@pytest.mark.parametrize("counts,K,N", MM_CASES, ids=MM_IDS)
def test_grouped_mm_and_gradients(M, counts, K, N, dtype, tail):
    say(f"grouped_mm counts={counts[:8]} K={K} N={N} {dtype} tail={tail}")
    x, dy, w, off = mm_inputs(counts, K, N, dtype, tail)
    R = x.shape[0]
    xd, dyd, wd, od = x.cuda(), dy.cuda(), w.cuda(), off.cuda()
    y = M.grouped_mm(xd, wd, od)
    dx = M.grouped_mm_dx(dyd, wd, od)
    dw = M.grouped_mm_dw(xd, dyd, od)
    torch.cuda.synchronize()
    live = torch.zeros(R, dtype=torch.bool)
    live[tail:R - tail] = True
    x0, dy0 = torch.where(live[:, None], x, 0), torch.where(live[:, None], dy, 0)
    ref, mag = mm_ref(x0, w, off)
    check(y, ref, K * 2.0 ** -23 * mag, "y")
    ref, mag = mm_ref(dy0, w, off, True)
    check(dx, ref, N * 2.0 ** -23 * mag, "dx")
    ref, mag = dw_ref(x0, dy0, off, K, N)
    check(dw, ref, max(counts) * 2.0 ** -23 * mag, "dw")
    if dtype == bf:
        check(M.grouped_mm_dw(xd, dyd, od, dtype=f32), ref, max(counts) * 2.0 ** -23 * mag, "dw in fp32")
    # the same call gives the same bits
    assert torch.equal(y.view(torch.uint8), M.grouped_mm(xd, wd, od).view(torch.uint8))
    assert torch.equal(dw.view(torch.uint8), M.grouped_mm_dw(xd, dyd, od).view(torch.uint8))


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
def test_groups_do_not_mix(M, dtype):
    """A NaN in one group's rows, or in one expert's matrix, stays with that group: nothing read
    past a tile's rows, columns or contraction reaches a result, not even times zero."""
    counts, K, N = [70, 33, 300, 1, 40], 200, 344
    say(f"groups do not mix {dtype}")
    x, dy, w, off = mm_inputs(counts, K, N, dtype, 0)
    for bad in (1, 3):
        a, b = int(off[bad]), int(off[bad + 1])
        xb, dyb, wb = x.clone(), dy.clone(), w.clone()
        xb[a:b], dyb[a:b], wb[bad] = float("nan"), float("nan"), float("inf")
        y, dx, dw = (M.grouped_mm(xb.cuda(), wb.cuda(), off.cuda()), M.grouped_mm_dx(dyb.cuda(), wb.cuda(), off.cuda()),
                     M.grouped_mm_dw(xb.cuda(), dyb.cuda(), off.cuda()))
        clean = (M.grouped_mm(x.cuda(), w.cuda(), off.cuda()), M.grouped_mm_dx(dy.cuda(), w.cuda(), off.cuda()),
                 M.grouped_mm_dw(x.cuda(), dy.cuda(), off.cuda()))
        rows = torch.ones(sum(counts), dtype=torch.bool)
        rows[a:b] = False
        es = [e for e in range(len(counts)) if e != bad]
        assert torch.equal(y.cpu()[rows], clean[0].cpu()[rows])
        assert torch.equal(dx.cpu()[rows], clean[1].cpu()[rows])
        assert torch.equal(dw.cpu()[es], clean[2].cpu()[es])
        assert bool(y.cpu()[~rows].isnan().all()) and bool(dx.cpu()[~rows].isnan().all())
        assert bool(dw.cpu()[bad].isnan().all())


def test_rows_outside_groups_are_left(M):
    say("rows outside the groups with out given")
    counts, K, N, tail = [20, 0, 70], 64, 72, 5
    for dtype in (bf, f32):
        x, dy, w, off = mm_inputs(counts, K, N, dtype, tail)
        R = x.shape[0]
        y = torch.full((R, N), 7.0, dtype=dtype, device="cuda")
        dx = torch.full((R, K), 7.0, dtype=dtype, device="cuda")
        assert M.grouped_mm(x.cuda(), w.cuda(), off.cuda(), out=y) is y
        M.grouped_mm_dx(dy.cuda(), w.cuda(), off.cuda(), out=dx)
        for t in (y, dx):
            assert bool((t[:tail] == 7).all()) and bool((t[R - tail:] == 7).all())
            assert not bool((t[tail:R - tail] == 7).all(1).any())


def test_offsets_are_held_in_bounds(M):
    """Offsets below 0 or above the row count are clamped: nothing outside is touched."""
    say("offsets out of range")
    K, N, R = 64, 72, 40
    x, w = rand((R, K), bf, 1), rand((3, K, N), bf, 3, K ** -0.5)
    off = torch.tensor([-7, 10, 30, 100000], dtype=torch.int32)
    y = M.grouped_mm(x.cuda(), w.cuda(), off.cuda())
    good = M.grouped_mm(x.cuda(), w.cuda(), torch.tensor([0, 10, 30, 40], dtype=torch.int32).cuda())
    assert torch.equal(y, good)


@pytest.mark.parametrize("off", [[0, 60, 10, 40, 20], [70, 0, 70, 0, 70], [100, 80, 60, 40, 20],
                                 [-5, 1 << 30, -(1 << 31), (1 << 31) - 1, 3]])
def test_offsets_that_decrease_stay_in_bounds(M, off):
    """Decreasing offsets name no groups; the results mean nothing, but nothing outside the
    output is written: guard rows around it keep their values."""
    say(f"decreasing offsets {off}")
    o = torch.tensor(off, dtype=torch.int32).cuda()
    R, K, N, G = 70, 72, 264, 64
    for dtype in (bf, f32):
        x, dy, w = rand((R, K), dtype, 1).cuda(), rand((R, N), dtype, 2).cuda(), rand((4, K, N), dtype, 3).cuda()
        y = torch.full((R + 2 * G, N), 7.0, dtype=dtype, device="cuda")
        dx = torch.full((R + 2 * G, K), 7.0, dtype=dtype, device="cuda")
        dw = torch.full((6, K, N), 7.0, dtype=dtype, device="cuda")
        M.grouped_mm(x, w, o, out=y[G:G + R])
        M.grouped_mm_dx(dy, w, o, out=dx[G:G + R])
        M.grouped_mm_dw(x, dy, o, out=dw[1:5])
        for t in (y, dx):
            assert bool((t[:G] == 7).all()) and bool((t[G + R:] == 7).all())
        assert bool((dw[0] == 7).all()) and bool((dw[5] == 7).all())
    K = 80
    xq, wq = torch.ones(R, K, dtype=torch.int8).cuda(), torch.ones(4, N, K, dtype=torch.int8).cuda()
    y = torch.full((R + 2 * G, N), 7.0, dtype=bf, device="cuda")
    M.grouped_mm_int8(xq, torch.ones(R).cuda(), wq, torch.ones(4, N).cuda(), o, out=y[G:G + R])
    assert bool((y[:G] == 7).all()) and bool((y[G + R:] == 7).all())


def test_no_rows(M):
    say("no rows")
    for dtype in (bf, f32):
        w = rand((4, 16, 24), dtype, 1).cuda()
        off = torch.zeros(5, dtype=torch.int32).cuda()
        assert M.grouped_mm(torch.empty(0, 16, dtype=dtype).cuda(), w, off).shape == (0, 24)
        assert M.grouped_mm_dx(torch.empty(0, 24, dtype=dtype).cuda(), w, off).shape == (0, 16)
        dw = M.grouped_mm_dw(torch.empty(0, 16, dtype=dtype).cuda(), torch.empty(0, 24, dtype=dtype).cuda(), off)
        assert dw.shape == (4, 16, 24) and not bool(dw.any())


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
def test_grouped_mm_autograd_and_differences(M, dtype):
    """autograd gives the gradients of the functional calls; the product is linear in x and in
    w, so <dy, y(x + v) - y(x)> = <dx, v> up to rounding."""
    say(f"grouped_mm autograd {dtype}")
    counts, K, N = [70, 0, 33, 5], 72, 136
    x, dy, w, off = mm_inputs(counts, K, N, dtype, 0)
    xd, wd, od, dyd = x.cuda().requires_grad_(), w.cuda().requires_grad_(), off.cuda(), dy.cuda()
    y = M.grouped_mm(xd, wd, od)
    dx, dw = torch.autograd.grad(y, (xd, wd), dyd)
    assert torch.equal(dx, M.grouped_mm_dx(dyd, wd.detach(), od))
    assert torch.equal(dw, M.grouped_mm_dw(xd.detach(), dyd, od))
    v, u = rand(x.shape, dtype, 11), rand(w.shape, dtype, 12)
    # each of the two products and the gradient is off by at most eps/2 of its elements plus
    # its sum's error; |<a, b>| <= sum |a||b| element by element
    e = half_eps(dtype)
    for moved, grad, var in (((x.to(f64) + v.to(f64)).to(dtype), dx, "x"), ((w.to(f64) + u.to(f64)).to(dtype), dw, "w")):
        y2 = M.grouped_mm(moved.cuda(), w.cuda(), od) if var == "x" else M.grouped_mm(x.cuda(), moved.cuda(), od)
        step = moved.to(f64) - (x if var == "x" else w).to(f64)       # what the sum of two rounded to
        y2, y1 = y2.cpu().to(f64), y.detach().cpu().to(f64)
        lhs = float((dy.to(f64) * (y2 - y1)).sum())
        rhs = float((grad.cpu().to(f64) * step).sum())
        tol = float((dy.to(f64).abs() * (y2.abs() + y1.abs())).sum()) * (e + 2.0 ** -18)
        tol += float((grad.cpu().to(f64).abs() * step.abs()).sum()) * (e + 2.0 ** -18)
        assert abs(lhs - rhs) <= tol, (var, lhs, rhs, tol)


# ------------------------------------------------------------------------------ int8
def quant_ref(x):
    """(q, scale) of rows: scale = fp32(max|x| / 127), the exact ratio rounded to even."""
    x = x.to(f64)
    amax = x.abs().amax(dim=-1)
    s = (amax.to(f32) / 127.0)
    ok = torch.isfinite(amax) & (s > 0)
    q = torch.where(ok[..., None], torch.round(x / torch.where(ok, s, 1.0).to(f64)[..., None]), 0.0).clamp(-127, 127)
    return q.to(torch.int8), torch.where(torch.isfinite(amax), s, float("nan"))


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,K", [(1, 8), (3, 24), (70, 264), (33, 1040), (9, 2048), (5, 2056), (4, 16392)])
def test_quantize_rows_exact(M, R, K, dtype):
    say(f"quantize_rows {R}x{K} {dtype}")
    x = rand((R, K), dtype, R + K)
    x[0, ::2] = 0
    if R > 2:
        x[1] = 0                                          # a row of zeros
        x[2] = (torch.arange(K) % 255 - 127).to(dtype)    # on the integers
    if R > 4:
        x[3] = ((torch.arange(K) % 254 - 127) + 0.5).to(dtype) * 2    # many exact borders for a scale of 2
        x[3, 0] = 254
    q, s = M.quantize_rows(x.cuda())
    rq, rs = quant_ref(x)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq)


def test_quantize_rows_nonfinite_and_tiny(M):
    say("quantize_rows, rows with inf, nan, subnormals")
    x = rand((6, 64), f32, 5)
    x[0, 7], x[1, 9], x[2, 3] = float("inf"), float("nan"), float("-inf")
    x[3] = 2.0 ** -149 * torch.arange(64)
    x[4] *= 2.0 ** 120
    x[5] *= 2.0 ** -126
    q, s = M.quantize_rows(x.cuda())
    q, s = q.cpu(), s.cpu()
    assert bool(s[:3].isnan().all()) and not bool(q[:3].any())
    rq, rs = quant_ref(x)
    assert torch.equal(s[3:], rs[3:]) and torch.equal(q[3:], rq[3:])


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("E,K,N", [(1, 16, 8), (3, 80, 72), (5, 144, 200), (2, 1040, 64)])
def test_quantize_experts_exact(M, E, K, N, dtype):
    say(f"quantize_experts {E}x{K}x{N} {dtype}")
    w = rand((E, K, N), dtype, E + K + N, K ** -0.5)
    w[0, :, 3] = 0
    q, s = M.quantize_experts(w.cuda())
    rq, rs = quant_ref(w.transpose(1, 2).contiguous())
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


I8_CASES = [([1], 16, 8), ([0, 1, 0], 48, 64), ([3, 0, 0, 5, 2], 80, 72), ([15, 16, 17, 31, 32, 33], 64, 136),
            ([63, 64, 65, 1], 144, 264), ([255, 256, 257, 0], 96, 520), ([700, 1, 0, 40], 1040, 328),
            ([2] * 100 + [0] * 56 + [5] * 100, 48, 40), ([1], 4112, 1032), ([600, 64, 65, 16, 17, 0], 768, 776)]


@pytest.mark.parametrize("out", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,K,N", I8_CASES, ids=[f"{sum(c)}rows-{len(c)}groups-{k}x{n}" for c, k, n in I8_CASES])
def test_grouped_mm_int8(M, counts, K, N, out):
    say(f"grouped_mm_int8 counts={counts[:8]} K={K} N={N} {out}")
    g = torch.Generator().manual_seed(K + N)
    tail, R, E = 2, sum(counts), len(counts)
    off = offs(counts, tail)
    xq = torch.randint(-127, 128, (R + 2 * tail, K), dtype=torch.int8, generator=g)
    wq = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, generator=g)
    xq[tail], wq[0, 0] = 127, -127                        # the largest sum there is
    xs, ws = torch.rand(R + 2 * tail, generator=g) + 0.01, torch.rand(E, N, generator=g) * 1e-3
    xs[:tail] = float("nan")
    y = M.grouped_mm_int8(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), off.cuda(), dtype=out)
    ref = torch.zeros(R + 2 * tail, N, dtype=f64)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        ref[a:b] = (xq[a:b].to(f64) @ wq[e].to(f64).T) * xs[a:b, None].to(f64) * ws[e].to(f64)
    # the conversion and the two scales round once each in fp32, then the output type
    check(y, ref, 3.1 * 2.0 ** -24 * ref.abs(), "y")
    keep = torch.full_like(y, 7.0)
    M.grouped_mm_int8(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), off.cuda(), out=keep)
    assert torch.equal(keep[tail:R + tail], y[tail:R + tail])
    assert bool((keep[:tail] == 7).all()) and bool((keep[R + tail:] == 7).all())


# Calls with enough work for the large tiles, whose kernels the cases above never reach:
# several rounds of 256 x 256 tiles, a workgroup per tile and a stream of tiles (a weight
# gradient of many and of few rows a group), and 128 x 128 tiles, with empty groups, groups of
# one row, and tiles that end early on both sides.
BIG_CASES = [([1000, 257, 0, 2200, 1, 1542], 2064, 2056), ([0, 700, 1, 5, 2294, 0], 1040, 1032), ([1500, 128, 0, 1, 371], 4112, 1032),
             ([0, 1, 0, 12, 2, 0, 7], 4112, 216), ([400, 40, 1, 18, 0, 0], 144, 7336), ([3] * 8 + [0] * 20 + [9] * 36, 304, 440),
             ([60] * 30 + [0] * 4 + [200] * 30, 304, 440), ([45, 0, 33, 64] * 16, 80, 984), ([71], 528, 16184), ([75] * 4, 1872, 2144),
             ([190, 0, 33, 1, 257, 64, 100, 31, 0, 5, 300, 16, 17, 128, 129, 90, 0, 250, 200, 179], 1040, 1032),
             # (a long contraction for few output tiles)
             ([1654], 328, 440), ([900, 0, 1, 700], 264, 136), ([5003], 40, 8)]
BIG_IDS = [f"{sum(c)}rows-{len(c)}groups-{k}x{n}" for c, k, n in BIG_CASES]


def on_gpu64(a, b):
    """a @ b and |a| @ |b| in 64 bits (the references' sizes would take the CPU seconds each)."""
    a, b = a.to(f64), b.to(f64)
    return (a @ b).cpu(), (a.abs() @ b.abs()).cpu()


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,K,N", BIG_CASES, ids=BIG_IDS)
def test_grouped_mm_large_tiles(M, counts, K, N, dtype):
    say(f"grouped_mm large counts={counts[:8]} K={K} N={N} {dtype}")
    tail = 5
    x, dy, w, off = mm_inputs(counts, K, N, dtype, tail)
    xd, dyd, wd, od = x.cuda(), dy.cuda(), w.cuda(), off.cuda()
    y, dx = torch.full_like(dyd, 7.0), torch.full_like(xd, 7.0)
    M.grouped_mm(xd, wd, od, out=y)
    M.grouped_mm_dx(dyd, wd, od, out=dx)
    dw = torch.full((len(counts) + 2, K, N), 7.0, dtype=dtype, device="cuda")
    M.grouped_mm_dw(xd, dyd, od, out=dw[1:-1])
    dw32 = M.grouped_mm_dw(xd, dyd, od, dtype=f32)
    torch.cuda.synchronize()
    for t in (y, dx):
        assert bool((t[:tail] == 7).all()) and bool((t[tail + sum(counts):] == 7).all())
    assert bool((dw[0] == 7).all()) and bool((dw[-1] == 7).all())
    for e, c in enumerate(counts):
        a, b = int(off[e]), int(off[e + 1])
        if c == 0:
            assert not bool(dw[e + 1].any()) and not bool(dw32[e].any())
            continue
        ref, mag = on_gpu64(xd[a:b], wd[e])
        check(y[a:b], ref, K * 2.0 ** -23 * mag, f"y of group {e}")
        ref, mag = on_gpu64(dyd[a:b], wd[e].T)
        check(dx[a:b], ref, N * 2.0 ** -23 * mag, f"dx of group {e}")
        ref, mag = on_gpu64(xd[a:b].T, dyd[a:b])
        check(dw[e + 1], ref, c * 2.0 ** -23 * mag, f"dw of group {e}")
        check(dw32[e], ref, c * 2.0 ** -23 * mag, f"dw in fp32 of group {e}")
    assert torch.equal(dw[1:-1].reshape(-1).view(torch.uint8), M.grouped_mm_dw(xd, dyd, od).reshape(-1).view(torch.uint8))


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
def test_large_tiles_do_not_mix_groups(M, dtype):
    """NaN in one group's rows or matrix reaches that group's results and no other's."""
    say(f"large tiles, NaN in groups {dtype}")
    counts, K, N = [500, 700, 0, 259, 1200], 2056, 2056
    x, dy, w, off = mm_inputs(counts, K, N, dtype, 0)
    x[500:1200:50, 7] = float("nan")
    dy[:500:100, 9] = float("nan")
    w[3, 100, 200] = float("inf")
    x, dy, w, od = x.cuda(), dy.cuda(), w.cuda(), off.cuda()
    y, dx, dw = M.grouped_mm(x, w, od), M.grouped_mm_dx(dy, w, od), M.grouped_mm_dw(x, dy, od)
    rows = torch.zeros(sum(counts), dtype=torch.bool, device="cuda")
    rows[500:1200:50] = True
    assert bool(y[rows].isnan().all()) and bool(y[~rows][:, :200].isfinite().all()) and bool(y[~rows][:, 201:].isfinite().all())
    assert not bool(y[1200:1459, 200].isfinite().any()) and bool(y[1459:].isfinite().all())
    rows[:] = False
    rows[:500:100] = True
    assert bool(dx[rows].isnan().all()) and bool(dx[~rows][:, :100].isfinite().all()) and bool(dx[~rows][:, 101:].isfinite().all())
    assert bool(dw[1, 7].isnan().all()) and bool(dw[0, :, 9].isnan().all())
    dw[1, 7], dw[0, :, 9] = 0, 0
    assert bool(dw.isfinite().all()) and not bool(dw[2].any())


@pytest.mark.parametrize("off", [[0, 3000, 500, 2000, 1000], [5000, 0, 5000, 0, 5000], [5000, 4000, 3000, 2000, 1000]])
def test_large_tiles_with_offsets_that_decrease(M, off):
    """As the small tiles: the results mean nothing, guard rows keep their values."""
    say(f"large tiles, decreasing offsets {off}")
    o = torch.tensor(off, dtype=torch.int32).cuda()
    R, K, N, G = 5000, 2064, 2056, 300
    for dtype in (bf, f32):
        x, dy, w = rand((R, K), dtype, 1).cuda(), rand((R, N), dtype, 2).cuda(), rand((4, K, N), dtype, 3).cuda()
        y = torch.full((R + 2 * G, N), 7.0, dtype=dtype, device="cuda")
        dx = torch.full((R + 2 * G, K), 7.0, dtype=dtype, device="cuda")
        dw = torch.full((6, K, N), 7.0, dtype=dtype, device="cuda")
        M.grouped_mm(x, w, o, out=y[G:G + R])
        M.grouped_mm_dx(dy, w, o, out=dx[G:G + R])
        M.grouped_mm_dw(x, dy, o, out=dw[1:5])
        for t in (y, dx):
            assert bool((t[:G] == 7).all()) and bool((t[G + R:] == 7).all())
        assert bool((dw[0] == 7).all()) and bool((dw[5] == 7).all())
    xq, wq = torch.ones(R, K, dtype=torch.int8).cuda(), torch.ones(4, N, K, dtype=torch.int8).cuda()
    y = torch.full((R + 2 * G, N), 7.0, dtype=bf, device="cuda")
    M.grouped_mm_int8(xq, torch.ones(R).cuda(), wq, torch.ones(4, N).cuda(), o, out=y[G:G + R])
    assert bool((y[:G] == 7).all()) and bool((y[G + R:] == 7).all())


@pytest.mark.parametrize("out", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,K,N", [BIG_CASES[i] for i in (0, 1, 2, 5, 6, 8)], ids=[BIG_IDS[i] for i in (0, 1, 2, 5, 6, 8)])
def test_grouped_mm_int8_large_tiles(M, counts, K, N, out):
    say(f"grouped_mm_int8 large counts={counts[:8]} K={K} N={N} {out}")
    g = torch.Generator().manual_seed(K + N)
    tail, R, E = 2, sum(counts), len(counts)
    off = offs(counts, tail)
    xq = torch.randint(-127, 128, (R + 2 * tail, K), dtype=torch.int8, generator=g).cuda()
    wq = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, generator=g).cuda()
    xs, ws = (torch.rand(R + 2 * tail, generator=g) + 0.01).cuda(), (torch.rand(E, N, generator=g) * 1e-3).cuda()
    y = torch.full((R + 2 * tail, N), 7.0, dtype=out, device="cuda")
    M.grouped_mm_int8(xq, xs, wq, ws, off.cuda(), out=y)
    assert bool((y[:tail] == 7).all()) and bool((y[R + tail:] == 7).all())
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        ref = ((xq[a:b].to(f64) @ wq[e].to(f64).T) * xs[a:b, None].to(f64) * ws[e].to(f64)).cpu()
        check(y[a:b], ref, 3.1 * 2.0 ** -24 * ref.abs(), f"y of group {e}")


# --------------------------------------------------------------------------- dropout
def philox(seed, step, blocks):
    """[blocks, 8] 16-bit numbers of Philox4x32-10, in numpy's unsigned 64-bit integers."""
    u = np.uint64
    m32 = u(0xFFFFFFFF)
    b = np.arange(blocks, dtype=np.uint64)
    c = [b & m32, b >> u(32), np.full_like(b, step & 0xFFFFFFFF), np.full_like(b, step >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(p1 >> u(32)) ^ c[1] ^ u(k[0]), p1 & m32, (p0 >> u(32)) ^ c[3] ^ u(k[1]), p0 & m32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    w = np.stack(c, 1)
    return np.stack([w & u(0xFFFF), w >> u(16)], 2).reshape(blocks, 8)


def test_philox_reference_known_answers():
    """The published known-answer vectors of Philox4x32-10 (counter and key all zeros, all ones)."""
    w = philox(0, 0, 1)[0].astype(np.uint64)
    words = [int(w[2 * i] | (w[2 * i + 1] << np.uint64(16))) for i in range(4)]
    assert words == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def keep_ref(seed, step, n, p):
    t = int(round(p * 65536))
    keep = torch.from_numpy((philox(seed, step, (n + 7) // 8).reshape(-1)[:n] >= t))
    return keep, (65536.0 / (65536 - t) if t < 65536 else 0.0)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,p", [(1, 0.5), (7, 0.3), (8, 0.9), (1000, 0.1), (4099, 0.0), (4099, 1.0), (65536 + 3, 0.25),
                                 (300, 1e-9), (4096, 0.99999)])
def test_dropout(M, n, p, dtype):
    say(f"dropout n={n} p={p} {dtype}")
    seed, step = 0x123456789ABCDEF0, (7 << 32) + 5
    x = rand((n,), dtype, n)
    keep, c = keep_ref(seed, step, n, p)
    x[~keep] = float("nan")                               # what is dropped may hold anything
    ref = torch.where(keep, x.to(f64) * c, 0.0)
    y = M.dropout(x.cuda(), p, seed, step)
    check(y, ref, 2.0 ** -23 * ref.abs(), "y")            # the scale's and the product's fp32 roundings
    z = x.cuda()
    M.dropout(z, p, seed, step, out=z)
    assert torch.equal(z, y)
    # the gradient draws the same mask
    xd = x.cuda().requires_grad_()
    dy = rand((n,), dtype, n + 1).cuda()
    (dx,) = torch.autograd.grad(M.dropout(xd, p, seed, step), xd, dy)
    assert torch.equal(dx, M.dropout(dy, p, seed, step))
    # the step as a device word
    word = torch.tensor([step], dtype=torch.int64, device="cuda")
    assert torch.equal(M.dropout(x.cuda(), p, seed, word), y)


def act_ref(a, b, dh, keep, c):
    a, dh = a.to(f64), dh.to(f64)
    b = torch.ones_like(a) if b is None else b.to(f64)
    s = torch.sigmoid(a)
    d = dh * c
    h = torch.where(keep, a * s * b * c, 0.0)
    da = torch.where(keep, d * b * (s + a * s * (1 - s)), 0.0)
    mag = torch.where(keep, (d * b).abs() * (s + a.abs() * s * (1 - s)), 0.0)
    db = torch.where(keep, d * a * s, 0.0)
    return h, da, mag, db


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,F,p,packed,gate", [(1, 8, 0.5, False, True), (5, 24, 0.0, True, True), (33, 264, 0.1, True, True),
                                               (64, 128, 0.4, False, False), (7, 2056, 0.1, False, True),
                                               (3, 40, 1.0, False, True), (130, 72, 0.0, False, False)])
def test_gated_act_and_gradient(M, R, F, p, packed, gate, dtype):
    say(f"gated_act {R}x{F} p={p} packed={packed} gate={gate} {dtype}")
    seed, step = 99, 3
    ab, dh = rand((R, 2 * F), dtype, R, 2.0), rand((R, F), dtype, R + F)
    ab[0, :4] = torch.tensor([-90.0, 90.0, -1.28, 0.0]).to(dtype)
    keep, c = keep_ref(seed, step, R * F, p)
    keep = keep.view(R, F)
    ab[:, :F][~keep] = float("inf")                       # under the mask: anything
    ab[:, F:][~keep] = float("nan")
    a, b = ab[:, :F], ab[:, F:] if gate else None
    abd = ab.cuda()
    ad, bd = abd[:, :F], abd[:, F:] if gate else None
    if not packed:
        ad, bd = ad.contiguous(), None if bd is None else bd.contiguous()
    # the exponential, the reciprocal and up to six products: 16 roundings of 2^-24, and the
    # exponential's argument, |a| <= 90 times log2 e, rounded once: 90 2^-24 more
    u = (16 + 130) * 2.0 ** -24
    h, da, mag, db = act_ref(a, b, dh, keep, c)
    check(M.gated_act(ad, bd, p, seed, step), h, u * h.abs(), "h")
    gda, gdb = M.gated_act_grad(dh.cuda(), ad, bd, p, seed, step)
    check(gda, da, u * mag, "da")
    if gate:
        check(gdb, db, u * db.abs(), "db")
    else:
        assert gdb is None
    # packed gradients
    if gate:
        buf = torch.full((R, 2 * F + 8), 7.0, dtype=dtype, device="cuda")
        M.gated_act_grad(dh.cuda(), ad, bd, p, seed, step, out=(buf[:, :F], buf[:, F:2 * F]))
        assert torch.equal(buf[:, :F], gda) and torch.equal(buf[:, F:2 * F], gdb) and bool((buf[:, 2 * F:] == 7).all())
    # autograd
    ar, br = ad.detach().requires_grad_(), None if bd is None else bd.detach().requires_grad_()
    out = M.gated_act(ar, br, p, seed, step)
    grads = torch.autograd.grad(out, (ar, br) if gate else (ar,), dh.cuda())
    assert torch.equal(grads[0], gda) and (not gate or torch.equal(grads[1], gdb))


def test_gated_act_differences(M):
    """Central differences of the kernel itself, in fp32: with a step of 2^-5 the truncation is
    at most h^2/6 |f'''| <= 2^-12 |b| c per element (|SiLU'''| < 1) and the rounding of the two
    values 2^-22 |f| / h; summed against the gradient's direction both stay below 1e-3 of the
    sum of magnitudes."""
    say("gated_act against differences")
    R, F, p, h = 40, 64, 0.2, 2.0 ** -5
    a, b, dh = rand((R, F), f32, 1).cuda(), rand((R, F), f32, 2).cuda(), rand((R, F), f32, 3).cuda()
    da, db = M.gated_act_grad(dh, a, b, p, 5, 6)
    f = lambda x, y: M.gated_act(x, y, p, 5, 6).to(f64)
    for grad, up, dn in ((da, f(a + h, b), f(a - h, b)), (db, f(a, b + h), f(a, b - h))):
        num = dh.to(f64) * (up - dn) / (2 * h)
        assert float((num - grad.to(f64)).abs().sum()) <= 1e-3 * float((dh.abs() * (1 + b.abs()) * 1.25).sum())


# --------------------------------------------------------------------------- combine
@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,k,H,drop", [(1, 1, 8, 0), (5, 3, 40, 2), (33, 8, 264, 30), (64, 2, 2056, 0), (9, 4, 4104, 5),
                                        (17, 6, 16392, 0), (3, 2, 64, 6), (200, 1, 512, 0)])
def test_combine_grad(M, T, k, H, drop, dtype):
    say(f"combine_grad T={T} k={k} H={H} drop={drop} {dtype}")
    g = torch.Generator().manual_seed(T + k + H)
    P = T * k
    perm = torch.randperm(P, generator=g)
    kept = perm[: P - drop]
    rop = torch.full((P,), -1, dtype=torch.int32)
    rop[kept] = torch.arange(P - drop, dtype=torch.int32)
    dout, y = rand((T, H), dtype, 1), rand((P - drop + 1, H), dtype, 2)    # one row no pair names
    w = torch.rand(T, k, generator=g)
    dy, dw = M.combine_grad(dout.cuda(), y.cuda(), rop.cuda(), w.cuda())
    d = dout.to(f64)[kept // k]
    ref = d * w.flatten()[kept].to(f64)[:, None]
    check(dy[: P - drop], ref, 2.0 ** -24 * ref.abs(), "dy_perm")
    rw, mag = torch.zeros(P, dtype=f64), torch.zeros(P, dtype=f64)
    rw[kept], mag[kept] = (d * y[:-1].to(f64)).sum(1), (d * y[:-1].to(f64)).abs().sum(1)
    check(dw, rw.view(T, k), H * 2.0 ** -24 * mag.view(T, k), "dtopk_w")


def test_combine_grad_leaves_unnamed_rows(M):
    say("combine_grad, rows no pair names, rows out of range")
    T, k, H = 4, 2, 64
    dout, y = rand((T, H), bf, 1).cuda(), rand((8, H), bf, 2).cuda()
    rop = torch.tensor([0, 1, -1, 100000, 4, 5, 6, -5], dtype=torch.int32).cuda()
    w = torch.rand(T, k).cuda()
    from mixture_experts_layer_46_amd import _lib
    dy = torch.full((8, H), 7.0, dtype=bf, device="cuda")
    dw = torch.full((T, k), 7.0, device="cuda")
    _lib.call("moe_combine_grad", _lib.MOE_BF16, T, k, H, 8, dout.data_ptr(), y.data_ptr(), rop.data_ptr(), w.data_ptr(),
              dy.data_ptr(), dw.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert bool((dy[[2, 3, 7]] == 7).all()) and not bool((dy[[0, 1, 4, 5, 6]] == 7).all(1).any())
    assert dw.flatten()[[2, 3, 7]].tolist() == [0.0, 0.0, 0.0]
