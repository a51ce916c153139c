"""Tensors past the sizes at which an operator changes its way: combine_grad's rows past what the
memory-side cache holds, and byte offsets past 2^32 of it and of the gated activation."""
import numpy as np
import pytest
import torch

from gpu_util import say
from test_ops_forms import close
from test_ops_gpu import act_ref
from test_ops_layers_gpu import _philox_at

pytestmark = pytest.mark.gpu
bf, f32, f64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def M():
    import mixture_experts_layer_46_amd as M
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    M._lib.load()
    yield M
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,k,H,dtype", [
    (66500, 2, 1016, bf),           # 270 MB of rows, a wavefront per token
    (17000, 8, 504, f32),           # 274 MB, a wavefront per token
    (8201, 4, 4104, bf),            # 269 MB, a workgroup per token
    (5500, 3, 4104, f32),           # 271 MB, a workgroup per token
    (33750, 8, 8008, bf),           # 4.3 GB
])
def test_combine_grad_of_many_rows(M, T, k, H, dtype):
    """Past 256 MB the rows are read past the caches.  Every row's gradient is one product and one
    rounding; dtopk_w a sum of H fp32 products."""
    say(f"combine_grad T={T} k={k} H={H} {dtype}")
    P = T * k
    assert P * H * (2 if dtype == bf else 4) > (256 << 20)
    g = torch.Generator(device="cuda").manual_seed(T)
    rows = torch.randperm(P, device="cuda", generator=g)
    rows[::7] = -1                                       # dropped pairs, the first one among them
    rows[-3] = -1
    dout = torch.empty((T, H), dtype=dtype, device="cuda").normal_(generator=g)
    y = torch.empty((P, H), dtype=dtype, device="cuda").normal_(generator=g)
    w = torch.rand((T, k), device="cuda", generator=g)
    dy, dw = M.combine_grad(dout, y, rows.int(), w)
    assert not bool(dw.flatten()[rows < 0].any())
    tokens = torch.cat([torch.arange(64), torch.arange(T - 64, T), torch.randint(0, T, (200,), generator=torch.Generator().manual_seed(1))])
    high = torch.topk(rows, 40).indices.cpu() // k       # the tokens of the last rows
    for t in (tokens.cuda(), high.cuda()):
        pair = (t[:, None] * k + torch.arange(k, device="cuda")).flatten()
        pair = pair[rows[pair] >= 0]
        d = dout[pair // k].to(f64)
        ref = d * w.flatten()[pair].to(f64)[:, None]
        close(dy[rows[pair]], ref, 2.0 ** -24 * ref.abs(), "dy_perm")
        v = y[rows[pair]].to(f64)
        close(dw.flatten()[pair], (d * v).sum(1), H * 2.0 ** -24 * (d * v).abs().sum(1), "dtopk_w")


@pytest.mark.parametrize("packed", [False, True])
def test_gated_act_past_32_bits(M, packed):
    """4.3 GB a tensor (a packed pair 8.6): the last rows and their mask are right."""
    say(f"gated_act past 32 bits, packed={packed}")
    R, F, n, p, seed, step = 266000, 8088, 40, 0.1, 5, 6
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.empty(s, dtype=bf, device="cuda").normal_(generator=g)
    if packed:
        ab = new(R, 2 * F)
        a, b = ab[:, :F], ab[:, F:]
    else:
        a, b = new(R, F), new(R, F)
    assert R * F * 2 > 1 << 32
    dh = new(R, F)
    first = (R - n) * F
    assert first % 8 == 0
    keep = torch.from_numpy(_philox_at(np.arange(first // 8, R * F // 8, dtype=np.uint64), seed, step).reshape(-1) >= round(p * 65536))
    keep = keep.view(n, F)
    c = 65536.0 / (65536 - round(p * 65536))
    h, da, mag, db = act_ref(a[-n:].cpu(), b[-n:].cpu(), dh[-n:].cpu(), keep, c)
    u = (16 + 130) * 2.0 ** -24                          # as in the operator's own test, |a| below 90
    close(M.gated_act(a, b, p, seed, step)[-n:].cpu(), h, u * h.abs(), "h")
    if packed:
        out = torch.empty((R, 2 * F), dtype=bf, device="cuda")
        ga, gb = M.gated_act_grad(dh, a, b, p, seed, step, out=(out[:, :F], out[:, F:]))
    else:
        ga, gb = M.gated_act_grad(dh, a, b, p, seed, step)
    close(ga[-n:].cpu(), da, u * mag, "da")
    close(gb[-n:].cpu(), db, u * db.abs(), "db")
