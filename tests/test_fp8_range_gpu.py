"""The 8-bit floating-point products over long contractions, scales of every size, blocks of zeros and
products that cancel, in every form; the tolerances are those of test_fp8_gpu.py.

A form brings the exponents of a row's blocks in words of four, so that contractions from 512 on take
several of them, and from 1536 on each of the words' two places more than once.
"""
import pytest
import torch

from gpu_util import say
from test_fp8_gpu import E4, E8, FORMS, check, groups_of, open_rows, operands, product_ref

pytestmark = pytest.mark.gpu
bf, f32, f64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def M():
    import mixture_experts_layer_46_amd as M
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M._lib.load()
    return M


# form, type, rows, groups, K, N: K of several exponent words with a remainder
LONG = [("256x256", bf, 2655, 1, 1552, 3576), ("256x256", bf, 4543, 5, 2064, 1888),
        ("128x128", bf, 1975, 1, 1552, 1160), ("128x128", bf, 634, 5, 2064, 2976),
        ("64x64", bf, 1300, 1, 1552, 1400), ("64x64", bf, 600, 9, 1808, 1000),
        ("32x64 thin", bf, 700, 3, 1808, 520), ("32x64 thin", bf, 33, 2, 4112, 520),
        ("128x128", f32, 2600, 5, 1552, 1160), ("64x64", f32, 2150, 1, 1552, 1112), ("64x64", f32, 696, 5, 2064, 2832),
        ("32x64 thin", f32, 700, 3, 1808, 520), ("32x64 thin", f32, 2219, 5, 2064, 80), ("16x64 thin", f32, 33, 2, 4112, 520)]
names = lambda v: {bf: "bf16", f32: "fp32"}.get(v, str(v))


@pytest.mark.parametrize("form,dtype,R,E,K,N", LONG, ids=names)
def test_long_contractions(M, form, dtype, R, E, K, N):
    """Every block with a scale of its own (within 2^6 of each other, so that a wrong one shows), NaN in
    the scales' padding; the same call twice gives the same bits."""
    say("grouped_mm_fp8 long", form, R, E, K, N, dtype)
    code = M._lib.MOE_F32 if dtype == f32 else M._lib.MOE_BF16
    assert M._lib.grouped_mm_form("fp8", R, E, K, N, dtype=code, cus=256) == form
    xq, xs, wq, ws = operands(R, E, K, N)
    off, rest = groups_of(R, E)
    ref, tol = product_ref(xq, xs, wq, ws, off, dtype)
    args = [t.cuda() for t in (xq, xs, wq, ws, off)]
    y = M.grouped_mm_fp8(*args, dtype=dtype)
    check(y, ref, tol, form)
    assert torch.equal(M.grouped_mm_fp8(*args, dtype=dtype), y)


@pytest.mark.parametrize("form,dtype,R,E,K,N", [c for c in FORMS if c[1] == bf] + LONG, ids=names)
def test_scales_of_any_size(M, form, dtype, R, E, K, N):
    """Each row of xq and block of wq's columns with a scale from 2^-127 to 2^127, whose product lies in
    or out of fp32's range.  All products are positive and within a factor of 9 of each other, so
    that their sum has no cancellation: fp32 sums are off by K 2^-23 of it, what the instruction
    drops is at most 8 2^-13 of each group's largest product, 2^-10 of the sum, and where sums fall
    below fp32's least normal number every addition of a group of 8 may lose up to 2^-126.  Where
    they pass its largest they are infinite."""
    say("grouped_mm_fp8 scales", form, R, E, K, N, dtype)
    g = torch.Generator().manual_seed(R + K)
    xq, wq = ((torch.rand(*s, generator=g) + 0.5).to(E4) for s in ((R, K), (E, N, K)))
    S = 4 * ((K + 511) // 512)
    xs = torch.randint(0, 255, (R, 1), generator=g).expand(R, S).contiguous().to(torch.uint8).view(E8)
    ws = torch.randint(0, 255, (E, (N + 127) // 128, 1), generator=g).expand(-1, -1, S).contiguous().to(torch.uint8).view(E8)
    off, _ = groups_of(R, E)
    y = M.grouped_mm_fp8(*(t.cuda() for t in (xq, xs, wq, ws, off)), dtype=dtype).cpu()
    ref = torch.zeros(R, N, dtype=f64)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        w = open_rows(wq[e], ws[e].view(torch.uint8).repeat_interleave(128, 0)[:N].view(E8), K).cuda()
        ref[a:b] = (open_rows(xq[a:b], xs[a:b], K).cuda() @ w.T.contiguous()).cpu()
    acc = ref * (K * 2.0 ** -23 + (2.0 ** -10 if dtype == bf else 0)) + (K // 8 + 16) * 2.0 ** -126
    top, rest = ref > torch.finfo(f32).max * 1.02, ref < torch.finfo(f32).max * 0.98
    assert bool(top.any()) or R < 3
    assert bool(torch.isinf(y[top]).all()) and bool((y[top] > 0).all())
    bad = (y.to(f64) - ref).abs() > acc + torch.finfo(dtype).eps / 2 * (ref + acc)
    bad = (bad | ~torch.isfinite(y)) & rest
    if bool(bad.any()):
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at flat {i}: {y.flatten()[i].item()} for "
                             f"{ref.flatten()[i].item()}")


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,K,N", [([1], 1040, 72), ([20, 0, 13], 528, 264), ([200, 137], 1552, 520), ([1400], 528, 3000)])
def test_blocks_of_zeros(M, counts, K, N, dtype):
    """Rows, blocks and expert blocks of zeros have the least scale, 2^-127: they add nothing, and rows of
    nothing else are zeros."""
    R, E = sum(counts), len(counts)
    g = torch.Generator().manual_seed(R + N)
    x, w = torch.randn(R, K, generator=g), torch.randn(E, K, N, generator=g) * K ** -0.5
    x[::3, 128:256] = 0
    x[R // 2] = 0
    w[:, 256:384, :128] = 0
    q, s = M.quantize_rows_fp8(x.cuda())
    wq, ws = M.quantize_experts_fp8(w.cuda())
    assert int(s.view(torch.uint8)[R // 2, 0]) == 0 and int(ws.view(torch.uint8)[0, 0, 2]) == 0
    off = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32)
    y = M.grouped_mm_fp8(q, s, wq, ws, off.cuda(), dtype=dtype)
    check(y, *product_ref(q.cpu(), s.cpu(), wq.cpu(), ws.cpu(), off, dtype), "product")
    assert not bool(y[R // 2].any())


@pytest.mark.parametrize("R,E,K,N", [(1, 1, 880, 40), (352, 1, 1040, 784), (634, 5, 432, 2976), (2655, 1, 432, 3576),
                                     (1300, 1, 1552, 1400)])
def test_products_that_cancel(M, R, E, K, N):
    """In every block of 128 two large products cancel, beside small ones of 2^-14 or 1.5 2^-14 of them: with
    fp32 output those are summed in fp32, so that nothing of them is lost; bf16 output may lose what
    lies below 2^-13 of the largest product of a group of 8, 8 2^-13 of it for each group at most."""
    g = torch.Generator().manual_seed(K)
    x = torch.where(torch.rand(R, K, generator=g) < 0.5, 1.0, 1.5) * 2.0 ** -6
    x[:, ::128], x[:, 1::128] = 256.0, -256.0
    w = torch.ones(E, N, K) * 2.0 ** -1
    xq, wq = x.to(E4), w.to(E4)
    S = 4 * ((K + 511) // 512)
    xs, ws = torch.full((R, S), 127, dtype=torch.uint8).view(E8), torch.full((E, -(-N // 128), S), 127, dtype=torch.uint8).view(E8)
    off, rest = groups_of(R, E)
    args = [t.cuda() for t in (xq, xs, wq, ws, off)]
    ref, _ = product_ref(xq, xs, wq, ws, off, f32)
    # all products and sums are multiples of 2^-8 below 2^12, 20 bits, and exact in fp32 in any order
    assert torch.equal(M.grouped_mm_fp8(*args, dtype=f32).cpu().to(f64), ref)
    check(M.grouped_mm_fp8(*args, dtype=bf), *product_ref(xq, xs, wq, ws, off, bf), "bf16 output")
