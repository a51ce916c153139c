"""Every form of the grouped products' kernels, at sizes that leave a remainder on every side.

The library picks a form from the sizes; the cases here name the one they are meant for, and
the host-side test holds the picker to that, so that a change of its constants cannot take a
form out of the tests unnoticed."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_46_amd import _lib

bf, f32, f64, i8 = torch.bfloat16, torch.float32, torch.float64, torch.int8
gpu = pytest.mark.gpu
CUS = 256                                             # compute units of an MI355X

# product, type of the operands, form, rows, groups, K, N
CASES = [
    ("y", bf, "256x256", 3499, 1, 248, 3568), ("y", bf, "256x256", 5406, 3, 232, 1808),
    ("y", bf, "128x128", 1345, 1, 296, 1672), ("y", bf, "128x128", 1438, 2, 232, 1360),
    ("y", bf, "64x64", 627, 1, 248, 872), ("y", bf, "64x64", 1126, 2, 208, 464),
    ("y", bf, "32x64 thin", 12, 1, 232, 72), ("y", bf, "32x64 thin", 4, 2, 368, 72),
    ("y", bf, "16x64 thin", 1, 1, 1528, 88), ("y", bf, "16x64 thin", 27, 2, 1232, 72),
    ("y", f32, "64x64", 128, 1, 112, 2088), ("y", f32, "64x64", 2098, 2, 104, 112),
    ("y", f32, "32x64 thin", 304, 1, 376, 880), ("y", f32, "32x64 thin", 1347, 2, 120, 208),
    ("y", f32, "16x64 thin", 2, 1, 104, 88), ("y", f32, "16x64 thin", 8, 2, 144, 112),
    ("dx", bf, "256x256", 4467, 1, 2344, 344), ("dx", bf, "256x256", 5247, 5, 1656, 240),
    ("dx", bf, "128x128", 4612, 1, 528, 232), ("dx", bf, "128x128", 3258, 3, 584, 216),
    ("dx", bf, "64x64", 115, 1, 72, 208), ("dx", bf, "64x64", 142, 3, 72, 216),
    ("dx", bf, "32x64 thin", 1492, 1, 184, 1304), ("dx", bf, "32x64 thin", 832, 2, 368, 1560),
    ("dx", bf, "16x64 thin", 4, 1, 72, 856), ("dx", bf, "16x64 thin", 12, 2, 80, 720),
    ("dx", f32, "64x64", 2503, 1, 104, 104), ("dx", f32, "64x64", 2290, 19, 152, 104),
    ("dx", f32, "32x64 thin", 619, 1, 536, 232), ("dx", f32, "32x64 thin", 1393, 2, 200, 120),
    ("dx", f32, "16x64 thin", 1, 1, 80, 104), ("dx", f32, "16x64 thin", 39, 2, 80, 104),
    ("dw", bf, "256x256", 1152, 1, 3080, 3016), ("dw", bf, "256x256", 1882, 2, 1136, 3656),
    ("dw", bf, "256x256 stream", 1067, 5, 1432, 1128),
    ("dw", bf, "256x256 stream", 4785, 33, 1800, 392),    # 528 tiles on 256 workgroups: three rounds
    ("dw", bf, "128x128", 404, 1, 1624, 1544), ("dw", bf, "128x128", 2922, 7, 944, 280),
    ("dw", bf, "64x64", 212, 1, 944, 560), ("dw", bf, "64x64", 2603, 12, 368, 72),
    ("dw", bf, "32x64 thin", 223, 1, 40, 88), ("dw", bf, "32x64 thin", 638, 2, 56, 72),
    ("dw", f32, "64x64", 136, 1, 1912, 568), ("dw", f32, "64x64", 2556, 19, 432, 80),
    ("dw", f32, "32x64 thin", 151, 1, 48, 72), ("dw", f32, "32x64 thin", 401, 2, 40, 152),
    ("int8", i8, "256x256", 4322, 1, 656, 2408), ("int8", i8, "256x256", 2815, 2, 400, 3152),
    ("int8", i8, "128x128", 1609, 1, 464, 1912), ("int8", i8, "128x128", 3590, 2, 432, 1016),
    ("int8", i8, "64x64", 799, 1, 496, 688), ("int8", i8, "64x64", 1343, 2, 400, 488),
    ("int8", i8, "32x64 thin", 2, 1, 752, 72), ("int8", i8, "32x64 thin", 10, 2, 592, 72),
    ("int8", i8, "16x64 thin", 2, 1, 432, 80), ("int8", i8, "16x64 thin", 21, 2, 400, 72),
]
NAMES = {bf: "bf16", f32: "fp32", i8: "int8"}
IDS = [f"{p}-{NAMES[t]}-{form.replace(' ', '-')}-{R}rows-{E}groups-{K}x{N}" for p, t, form, R, E, K, N in CASES]
each = pytest.mark.parametrize("product,dtype,form,R,E,K,N", CASES, ids=IDS)


def form_of(product, dtype, R, E, K, N, cus=CUS):
    return _lib.grouped_mm_form(product, R, E, K, N, _lib.MOE_F32 if dtype == f32 else _lib.MOE_BF16, cus)


@each
def test_the_case_takes_its_form(product, dtype, form, R, E, K, N):
    assert form_of(product, dtype, R, E, K, N) == form


def test_every_form_has_cases():
    tiles, thin = ["256x256", "128x128", "64x64"], ["32x64 thin", "16x64 thin"]
    want = {(p, t, f) for p, t in (("y", bf), ("dx", bf), ("int8", i8)) for f in tiles + thin}
    want |= {("dw", bf, f) for f in tiles + ["256x256 stream", "32x64 thin"]}
    want |= {(p, f32, f) for p in ("y", "dx") for f in ["64x64"] + thin} | {("dw", f32, "64x64"), ("dw", f32, "32x64 thin")}
    assert {c[:3] for c in CASES} == want


def test_form_query_refuses_what_the_product_refuses():
    for args, msg in ((("y", 8, 1, 12, 64), "multiples of 8"), (("int8", 8, 1, 24, 64), "multiple of 16"),
                      (("dw", -1, 1, 16, 64), "rows"), (("dx", 8, 300, 16, 64), "E = 300"),
                      (("y", (1 << 30) - 1, 256, 8, 1 << 20), "too many output tiles")):
        with pytest.raises(ValueError, match=msg):
            _lib.grouped_mm_form(*args, cus=CUS)
    lib = _lib.load()
    s = _lib.MmShape(8, 1, 16, 64, _lib.MOE_BF16, _lib.MOE_BF16, 0)
    assert lib.moe_grouped_mm_form(s, 4, CUS) is None and lib.moe_grouped_mm_form(s, -1, CUS) is None
    assert lib.moe_grouped_mm_form(s, 0, -1) is None and lib.moe_grouped_mm_form(None, 0, CUS) is None


# --------------------------------------------------------------------------- on the GPU
@pytest.fixture(scope="module")
def M():
    import mixture_experts_layer_46_amd as M
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M._lib.load()
    return M


def groups_of(R, E):
    """(offsets, rows of no group at either end): R rows in E ragged groups, where there are
    enough of them one without rows and one of a single row."""
    rest = 3 if R > 100 else 0
    n = R - 2 * rest
    if E == 1:
        counts = [n]
    else:
        share = np.random.RandomState(R + E).rand(E) + 0.2
        if E > 2:
            share[1], share[2] = 0.0, 0.0
        counts = np.floor(share / share.sum() * (n - 1)).astype(int)
        if E > 2:
            counts[2] = 1
        counts[-1] += n - counts.sum()
    off = np.concatenate([[0], np.cumsum(counts)]) + rest
    assert off[-1] == R - rest and (np.diff(off) >= 0).all()
    return torch.tensor(off, dtype=torch.int32), rest


def operands(product, dtype, R, E, K, N):
    """The product's two operands on the GPU (int8: with their scales)."""
    g = torch.Generator().manual_seed(R + E + K + N)
    if product == "int8":
        xq = torch.randint(-127, 128, (R, K), dtype=i8, generator=g).cuda()
        wq = torch.randint(-127, 128, (E, N, K), dtype=i8, generator=g).cuda()
        return xq, wq, (torch.rand(R, generator=g) + 0.01).cuda(), (torch.rand(E, N, generator=g) * 1e-3 + 1e-5).cuda()
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    if product == "dw":
        return r(R, K), r(R, N)
    return r(R, N if product == "dx" else K), (r(E, K, N) * K ** -0.5).to(dtype)


def run(M, product, ops, off, out=None, dtype=None):
    if product == "int8":
        xq, wq, xs, ws = ops
        return M.grouped_mm_int8(xq, xs, wq, ws, off, dtype=dtype or bf, out=out)
    if product == "dw":
        return M.grouped_mm_dw(*ops, off, out=out, dtype=dtype)
    return (M.grouped_mm_dx if product == "dx" else M.grouped_mm)(*ops, off, out=out)


def close(got, ref, acc, what):
    """The products' bound: the sum's error and one rounding to the output's type."""
    e = torch.finfo(got.dtype).eps / 2
    tol = acc + e * (ref.abs() + acc) + 1e-38
    bad = ~((got.to(f64) - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.numel())


def guarded(product, R, E, K, N, dtype, G=40):
    """An output between guards of sevens, and the whole buffer."""
    if product == "dw":
        buf = torch.full((E + 2, K, N), 7.0, dtype=dtype, device="cuda")
        return buf[1:-1], buf, 1
    buf = torch.full((R + 2 * G, K if product == "dx" else N), 7.0, dtype=dtype, device="cuda")
    return buf[G:G + R], buf, G


@gpu
@each
def test_values(M, product, dtype, form, R, E, K, N):
    """Against 64-bit products, for both output types where there are two; rows of no group hold
    NaN and keep out of everything.  A sum of n fp32 products is off by at most n 2^-23 of the
    magnitudes' sum; int8 sums are exact, with three fp32 roundings behind them."""
    print(f"form {form} {product} {dtype} R={R} E={E} K={K} N={N}", flush=True)
    assert form_of(product, dtype, R, E, K, N, 0) == form
    off, rest = groups_of(R, E)
    ops = operands(product, dtype, R, E, K, N)
    inner = slice(rest, R - rest)
    outside = torch.ones(R, dtype=torch.bool, device="cuda")
    outside[inner] = False
    for t in ((ops[2],) if product == "int8" else ops if product == "dw" else ops[:1]):
        t[outside] = float("nan")
    od = off.cuda()
    kinds = [bf, f32] if product == "int8" or (product == "dw" and dtype == bf) else [dtype]
    for to in kinds:
        out, buf, g = guarded(product, R, E, K, N, to)
        run(M, product, ops, od, out=out)
        assert bool((buf[:g] == 7).all()) and bool((buf[-g:] == 7).all())
        if product != "dw":
            assert bool((out[outside] == 7).all())
        again = run(M, product, ops, od, dtype=to)
        assert torch.equal(again if product == "dw" else again[inner], out if product == "dw" else out[inner])
        assert product == "dw" or not bool(again[outside].any())
        for e in range(E):
            a, b = int(off[e]), int(off[e + 1])
            if product == "dw":
                x, dy = ops[0][a:b].to(f64), ops[1][a:b].to(f64)
                close(out[e], x.T @ dy, (b - a) * 2.0 ** -23 * (x.T.abs() @ dy.abs()), f"group {e}")
            elif product == "int8":
                ref = (ops[0][a:b].to(f64) @ ops[1][e].to(f64).T) * ops[2][a:b, None].to(f64) * ops[3][e].to(f64)
                close(out[a:b], ref, 3.1 * 2.0 ** -24 * ref.abs(), f"group {e}")
            else:
                x, w = ops[0][a:b].to(f64), ops[1][e].to(f64)
                w = w.T if product == "dx" else w
                close(out[a:b], x @ w, x.shape[1] * 2.0 ** -23 * (x.abs() @ w.abs()), f"group {e}")


@gpu
@pytest.mark.parametrize("product,dtype,form,R,E,K,N", [c for c in CASES if c[4] > 1], ids=[i for i, c in zip(IDS, CASES) if c[4] > 1])
def test_a_group_keeps_its_values_to_itself(M, product, dtype, form, R, E, K, N):
    """NaN and infinities in one group's rows and matrix change no bit of another group's."""
    print(f"isolation {form} {product} {dtype} R={R} E={E} K={K} N={N}", flush=True)
    off, rest = groups_of(R, E)
    od = off.cuda()
    for bad in sorted({0, E // 2, E - 1}):
        a, b = int(off[bad]), int(off[bad + 1])
        ops = operands(product, dtype, R, E, K, N)
        clean = run(M, product, ops, od)
        if product == "int8":
            ops[2][a:b], ops[3][bad] = float("nan"), float("inf")
        else:
            ops[0][a:b] = float("nan")
            if product == "dw":
                ops[1][a:b] = float("inf")
            else:
                ops[1][bad] = float("inf")
        got = run(M, product, ops, od)
        if product == "dw":
            rest_e = [e for e in range(E) if e != bad]
            assert torch.equal(got[rest_e], clean[rest_e])
            assert bool(got[bad].isnan().all()) == (b > a)
        else:
            mine = torch.zeros(R, dtype=torch.bool, device="cuda")
            mine[a:b] = True
            assert torch.equal(got[~mine], clean[~mine])
            assert bool(got[mine].isnan().all())


@gpu
@each
def test_offsets_that_are_none(M, product, dtype, form, R, E, K, N):
    """Offsets that decrease or leave the rows name no groups: what is computed means nothing, and
    nothing outside the output is written."""
    print(f"bad offsets {form} {product} {dtype} R={R} E={E} K={K} N={N}", flush=True)
    ops = operands(product, dtype, R, E, K, N)
    saw = [R if i % 2 else 0 for i in range(E + 1)]
    for off in ([R - i * R // E for i in range(E + 1)], saw, saw[::-1], [-(1 << 31)] + [(1 << 31) - 1] * E,
                [R + 5] * (E + 1), [-1] * (E + 1)):
        out, buf, g = guarded(product, R, E, K, N, f32 if dtype == f32 else bf)
        run(M, product, ops, torch.tensor(off, dtype=torch.int32).cuda(), out=out)
        assert bool((buf[:g] == 7).all()) and bool((buf[-g:] == 7).all()), off[:4]
