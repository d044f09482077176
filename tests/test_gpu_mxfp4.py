"""MXFP4: quantisation bit for bit against its definition, every code and scale
decoded, and the products of MXFP4 experts with 16-bit and MXFP4 activations."""
import math

import pytest
import torch

import moe_ref as ref
import sharded_gemm_alltosharded_amd as sg
from test_gpu_moe import BF, F32, HF, chain_reference, gen, normal, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    sg.lib()


def same_codes(x):
    codes, scales = sg.quantize_mxfp4(x.cuda())
    wc, ws = ref.encode(x)
    assert torch.equal(scales.cpu(), ws)
    assert torch.equal(codes.cpu(), wc)
    return codes, scales


def same_values(got, want):
    """Equal values, NaN (an infinity in the input's block) where NaN is due."""
    got = got.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(torch.where(want.isnan(), 0.0, got), torch.where(want.isnan(), 0.0, want))


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (17, 14336), (5, 7, 64), (257, 160)])
def test_quantize(shape, dtype):
    g = gen(sum(shape))
    x = normal(g, shape) * torch.exp(3 * normal(g, (*shape[:-1], 1)))
    x[torch.rand(shape, generator=g) < 0.02] *= 30
    x[torch.rand(shape, generator=g) < 0.02] = 0
    codes, scales = same_codes(x.to(dtype))
    want = ref.decode(codes.cpu(), scales.cpu())
    for out in (F32, BF, HF):
        same_values(sg.dequantize_mxfp4(codes, scales, out), want.float().to(out))


def test_quantize_ties_and_edges():
    halves = torch.arange(-64, 64).float() / 8  # every tie of the grid among them
    x = torch.zeros((4, 128))
    x[0] = halves
    x[1] = halves * 2.0 ** -100
    x[2] = halves * 2.0 ** 100
    x[:3, ::32] = torch.tensor([4.0, 4.0 * 2.0 ** -100, 4.0 * 2.0 ** 100])[:, None]  # the block's largest: up to 8
    x[3, :32] = -0.0
    x[3, 32:64] = 2.0 ** -149  # the smallest number: scale 2^-127, all codes 0
    x[3, 64] = torch.finfo(F32).max
    x[3, 96] = 2.0 ** -126
    x[3, 97] = 2.0 ** -128
    same_codes(x)


def test_quantize_infinities_and_nans():
    x = torch.ones((1, 128))
    x[0, 3], x[0, 40], x[0, 100] = math.inf, -math.inf, math.nan
    codes, scales = same_codes(x)
    assert scales.tolist() == [[255, 255, 125, 255]]
    v = sg.dequantize_mxfp4(codes, scales)
    assert v.isnan().tolist()[0] == [True] * 64 + [False] * 32 + [True] * 32


def test_dequantize_every_code_and_scale():
    codes = torch.arange(256).to(torch.uint8).view(16, 16).repeat(256, 1)
    scales = torch.arange(256).to(torch.uint8).repeat_interleave(16).view(-1, 1)
    want = ref.decode(codes, scales)
    for dtype in (F32, BF):
        same_values(sg.dequantize_mxfp4(codes.cuda(), scales.cuda(), dtype), want.float().to(dtype))


def test_quantize_strided_and_empty():
    g = gen(1)
    for width, at in ((96, 0), (97, 1), (80, 8)):
        x = normal(g, (9, width), BF).cuda()[:, at:at + 64]
        a, b = sg.quantize_mxfp4(x), sg.quantize_mxfp4(x.contiguous())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c, s = sg.quantize_mxfp4(torch.empty((0, 64), device="cuda"))
    assert c.shape == (0, 32) and s.shape == (0, 2)


# ---- products ---------------------------------------------------------------

def mx_weights(g, E, n, K):
    codes = torch.randint(0, 256, (E, n, K // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    scales = torch.randint(118, 123, (E, n, K // 32), generator=g, dtype=torch.int32).to(torch.uint8)
    return codes, scales


COLUMNS = [  # E, R, in, out / P / S, P, S
    (1, 1, 32, 1, 1, 1), (1, 200, 96, 16, 2, 2), (3, 5, 160, 20, 1, 2), (4, 64, 256, 33, 2, 2), (8, 100, 64, 24, 4, 2),
    (5, 700, 1024, 48, 2, 1), (2, 300, 288, 130, 1, 2), (40, 90, 416, 16, 1, 2), (1, 700, 640, 272, 1, 2),
    (1, 3, 8192, 16, 1, 1), (2, 3, 8224, 144, 1, 2), (3, 3, 8320, 1400, 1, 1),
]


@pytest.mark.parametrize("acts", [16, 4])
@pytest.mark.parametrize("E,R,K,f,P,S", COLUMNS)
def test_mxfp4_column(E, R, K, f, P, S, acts):
    g = gen(R + K)
    n, T = f * P * S, max(1, R // 2)
    codes, scales = mx_weights(g, E, n, K)
    w = ref.decode(codes, scales)
    layer = sg.shard_mxfp4_experts(codes.cuda(), scales.cuda(), "all-to-sharded", segments=S, P=P)
    x = normal(g, (T, K), BF)
    off = offsets_of(g, E, R)
    rows = torch.randint(0, 2 * T, (R,), generator=g, dtype=torch.int32)
    rows[R // 2] = 2 * T  # no token: zeros
    if acts == 4:
        xc, xs = ref.encode(x)
        args, kw, xv = (xc.cuda(),), {"x_scales": xs.cuda()}, ref.decode(xc, xs)
    else:
        args, kw, xv = (x.cuda(),), {}, x.double()
    out, mag = (torch.zeros((R, n), dtype=torch.float64) for _ in range(2))
    ref.product(ref.gathered(xv, rows, 2), w, off, out, mag)
    order = ref.shard_rows(n, S, P)
    res, bound = torch.stack([out[:, o] for o in order]), torch.stack([mag[:, o] for o in order])
    for dt in (BF, F32):
        got = sg.experts_all_to_sharded(layer, *args, off.cuda(), rows.cuda(), 2, out_dtype=dt, **kw)
        ref.close(got, res, ref.sum_bound(bound, K), f"column {dt}")
        if S == 2:
            got = sg.experts_all_to_sharded(layer, *args, off.cuda(), rows.cuda(), 2, True, out_dtype=dt, **kw)
            (a, b), (ma, mb) = res.split(f, -1), bound.split(f, -1)
            ref.close(got, ref.silu(a) * b, ref.swiglu_bound(a, b, ma, mb, K), f"column swiglu {dt}")


@pytest.mark.parametrize("acts", [16, 4])
@pytest.mark.parametrize("E,R,K,f,P,S", [(1, 4200, 128, 8200, 2, 1), (3, 6000, 384, 3000, 1, 2), (1, 900, 640, 4100, 1, 2),
                                         (2, 300, 256, 9000, 1, 1)])
def test_mxfp4_wide_tiles(E, R, K, f, P, S, acts):
    """Sampled rows at sizes that take the widest tiles and their quarters."""
    g = gen(R)
    n = f * P * S
    codes, scales = mx_weights(g, E, n, K)
    w = ref.decode(codes, scales)
    layer = sg.shard_mxfp4_experts(codes.cuda(), scales.cuda(), "all-to-sharded", segments=S, P=P)
    x = normal(g, (R, K), BF)
    off = offsets_of(g, E, R, empty=False)
    pick = torch.unique(torch.cat([torch.randint(0, R, (30,), generator=g), off[1:].long() - 1,
                                   torch.tensor([0, 127, 128, 255, 256])]))
    expert = torch.searchsorted(off[1:].contiguous(), pick.int(), right=True)
    if acts == 4:
        xc, xs = sg.quantize_mxfp4(x.cuda())
        args, kw, xv = (xc,), {"x_scales": xs}, ref.decode(*ref.encode(x[pick]))
    else:
        args, kw, xv = (x.cuda(),), {}, x[pick].double()
    y = torch.stack([w[e] @ v for v, e in zip(xv, expert)])
    mag = torch.stack([w[e].abs() @ v.abs() for v, e in zip(xv, expert)])
    order = ref.shard_rows(n, S, P)
    res, bound = torch.stack([y[:, o] for o in order]), torch.stack([mag[:, o] for o in order])
    got = sg.experts_all_to_sharded(layer, *args, off.cuda(), out_dtype=F32, **kw)
    ref.close(got[:, pick.cuda()], res, ref.sum_bound(bound, K), "column")
    if S == 2:
        got = sg.experts_all_to_sharded(layer, *args, off.cuda(), swiglu=True, out_dtype=BF, **kw)
        (a, b), (ma, mb) = res.split(f, -1), bound.split(f, -1)
        ref.close(got[:, pick.cuda()], ref.silu(a) * b, ref.swiglu_bound(a, b, ma, mb, K), "swiglu")


ROWS = [  # E, R, out, in / P, P
    (1, 1, 1, 32, 1), (1, 150, 64, 96, 2), (3, 5, 20, 160, 1), (4, 64, 33, 64, 3), (8, 100, 250, 32, 4),
    (3, 900, 300, 288, 2), (40, 70, 64, 128, 1), (2, 2, 72, 2080, 4),
]


@pytest.mark.parametrize("acts", [16, 4])
@pytest.mark.parametrize("E,R,n,kr,P", ROWS)
def test_mxfp4_row(E, R, n, kr, P, acts):
    g = gen(R + n)
    codes, scales = mx_weights(g, E, n, kr * P)
    layer = sg.shard_mxfp4_experts(codes.cuda(), scales.cuda(), "sharded-to-all", P=P)
    h = normal(g, (P, R, kr), BF)
    off = offsets_of(g, E, R)
    if acts == 4:
        hc, hs = ref.encode(h)
        args, kw, hv = (hc.cuda(),), {"h_scales": hs.cuda()}, ref.decode(hc, hs)
    else:
        args, kw, hv = (h.cuda(),), {}, h.double()
    out, mag = (torch.zeros((R, n), dtype=torch.float64) for _ in range(2))
    ref.product(hv.transpose(0, 1).flatten(1), ref.decode(codes, scales), off, out, mag)
    for dt in (BF, F32):
        ref.close(sg.experts_sharded_to_all(layer, *args, off.cuda(), out_dtype=dt, **kw), out,
                  ref.sum_bound(mag, kr * P), f"row {dt}")


@pytest.mark.parametrize("acts", [16, 4])
def test_mxfp4_integers_exact(acts):
    """Codes and scales of whole numbers: the products are exact, bit for bit."""
    g = gen(3)
    E, R, K, n = 2, 60, 256, 32
    codes = torch.randint(0, 256, (E, n, K // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    scales = torch.randint(128, 131, (E, n, K // 32), generator=g, dtype=torch.int32).to(torch.uint8)
    layer = sg.shard_mxfp4_experts(codes.cuda(), scales.cuda(), "all-to-sharded")
    off = torch.tensor([0, 25, 60], dtype=torch.int32)
    x = torch.randint(-3, 4, (R, K), generator=g).to(BF)
    x[:, ::32] = 4  # every block's scale is 2^0: 4 = 2^2, so the codes hold the values
    w = ref.decode(codes, scales)
    want = torch.cat([x[:25].double() @ w[0].T, x[25:].double() @ w[1].T])[None]
    if acts == 4:
        c, s = sg.quantize_mxfp4(x.cuda())
        assert (s == 127).all()
        got = sg.experts_all_to_sharded(layer, c, off.cuda(), x_scales=s, out_dtype=F32)
    else:
        got = sg.experts_all_to_sharded(layer, x.cuda(), off.cuda(), out_dtype=F32)
    assert torch.equal(got.double().cpu(), want)


@pytest.mark.parametrize("R", [5, 100])
@pytest.mark.parametrize("acts", [16, 4])
def test_mxfp4_nan_scale(acts, R):
    g = gen(4)
    codes, scales = mx_weights(g, 1, 48, 128)
    codes[0, 7] = 0
    scales[0, 7, 2] = 255
    layer = sg.shard_mxfp4_experts(codes.cuda(), scales.cuda(), "all-to-sharded")
    x = normal(g, (R, 128), BF).cuda()
    if acts == 4:
        c, s = sg.quantize_mxfp4(x)
        s[3, 1] = 255
        got = sg.experts_all_to_sharded(layer, c, x_scales=s)
    else:
        got = sg.experts_all_to_sharded(layer, x)
    nan = torch.zeros((1, R, 48), dtype=torch.bool)
    nan[..., 7] = True
    if acts == 4:
        nan[0, 3] = True
    assert torch.equal(got.isnan().cpu(), nan)


@pytest.mark.parametrize("T,E,k,D,F,P", [(1, 4, 2, 256, 256, 8), (40, 6, 3, 160, 192, 2), (300, 2, 1, 96, 128, 1),
                                         (600, 3, 2, 256, 384, 4)])
def test_mxfp4_moe_mlp(T, E, k, D, F, P):
    g = gen(T)
    z = normal(g, (T, E), F32, 1.5)
    z[T - T // 9:] = -math.inf
    x = normal(g, (T, D), BF)
    gu, dn = mx_weights(g, E, 2 * F, D), mx_weights(g, E, D, F)
    lg = sg.shard_mxfp4_experts(gu[0].cuda(), gu[1].cuda(), "all-to-sharded", segments=2, P=P)
    ld = sg.shard_mxfp4_experts(dn[0].cuda(), dn[1].cuda(), "sharded-to-all", P=P)
    r = sg.moe_route(z.cuda(), k)
    out = sg.moe_mlp(lg, ld, x.cuda(), r)
    want, bound = chain_reference(z, x, ref.decode(*gu), ref.decode(*dn), k, BF)
    ref.close(out, want, bound, "moe_mlp")
    h = sg.experts_all_to_sharded(lg, x.cuda(), r.offsets, r.rows, k, swiglu=True)
    y = sg.experts_sharded_to_all(ld, h, r.offsets, out_dtype=F32)
    assert torch.equal(sg.moe_combine(y, r.slots, r.weights, out_dtype=BF), out)
