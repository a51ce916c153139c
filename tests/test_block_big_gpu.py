"""The operators around the block on buffers past 2^32 bytes: what a call computes for the last rows
or experts is, bit by bit, what it computes for them alone."""
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
    yield M
    torch.cuda.empty_cache()


def rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def test_norms(M):
    T, H, n = 70000, 16384, 300                        # 4.6 GB a tensor
    say("norms", T, H)
    x, z, dy, du = (rand((T, H), f32, s) for s in range(4))
    w1, gate, w2 = (rand((H,), f32, s) for s in range(4, 7))
    args = lambda s: (x[s], z[s], w1, gate, 0.5, w2)
    last = slice(T - n, T)
    y, u = M.residual_norm(*args(slice(0, T)))
    ys, us = M.residual_norm(*args(last))
    assert torch.equal(y[last], ys) and torch.equal(u[last], us)
    del y, u
    dx, dz, *_ = M.residual_norm_grad(dy, du, *args(slice(0, T)))
    dxs, dzs, *_ = M.residual_norm_grad(dy[last], du[last], *args(last))
    assert torch.equal(dx[last], dxs) and torch.equal(dz[last], dzs)


def test_fp8(M):
    R, K = 70000, 32768                                # 2.3 G values, 4.6 GB of bf16
    say("quantize_rows_fp8", R, K)
    x = rand((R, K), bf, 1)
    q, s = M.quantize_rows_fp8(x)
    qs, ss = M.quantize_rows_fp8(x[-100:])
    assert torch.equal(q[-100:].view(torch.uint8), qs.view(torch.uint8)) and torch.equal(s[-100:].view(torch.uint8), ss.view(torch.uint8))
    del x
    E, N = 5, 32768                                    # 5.4 GB of experts, y past 2^32 bytes
    wq = torch.randint(0, 120, (E, N, K), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ws = torch.randint(110, 125, (E, N // 128, K // 128), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    cut = R - 40
    off = torch.tensor([0, 0, 0, cut, cut, R], dtype=torch.int32, device="cuda")
    for dtype in (bf, f32):
        y = M.grouped_mm_fp8(q, s, wq, ws, off, dtype=dtype)
        for e, r in ((2, slice(cut - 30, cut)), (4, slice(cut, R))):
            n = r.stop - r.start
            alone = M.grouped_mm_fp8(q[r].contiguous(), s[r].contiguous(), wq[e:e + 1], ws[e:e + 1],
                                     torch.tensor([0, n], dtype=torch.int32, device="cuda"), dtype=dtype)
            # other forms sum in another order: K 2^-23 of the magnitudes (all values here are positive
            # or of one sign a row), and a rounding to dtype on each side
            err = (y[r].double() - alone.double()).abs().max() / alone.double().abs().max()
            assert float(err) <= K * 2.0 ** -23 + 2.0 ** -10 + torch.finfo(dtype).eps, (dtype, e, float(err))
        del y


def test_gated(M):
    E, K, N = 5, 16384, 32768                          # 5.4 GB a matrix
    say("gated_mm", E, K, N)
    w_in, w_up = (rand((E, K, N), bf, s).mul_(K ** -0.5) for s in (1, 2))
    R = 40
    x = rand((R, K), bf, 3)
    off = torch.tensor([0, 10, 10, 20, 20, R], dtype=torch.int32, device="cuda")
    h = M.gated_mm(x, w_in, w_up, off)
    a, b, dh = (rand((R, N), bf, s) for s in (4, 5, 6))
    dx = M.gated_mm_grad(dh, x, w_in, w_up, a, b, off)[0]
    one = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    r = slice(20, R)
    # (another number of groups may take another form, whose sums run in another order)
    hs = M.gated_mm(x[r], w_in[4:], w_up[4:], one(20))
    dxs = M.gated_mm_grad(dh[r], x[r], w_in[4:], w_up[4:], a[r], b[r], one(20))[0]
    for got, want in ((h[r], hs), (dx[r], dxs)):
        err = (got.double() - want.double()).abs().max() / want.double().abs().max()
        assert float(err) <= 2 * N * 2.0 ** -23 + torch.finfo(bf).eps, float(err)
