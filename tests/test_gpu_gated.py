"""MX FP8 activations and the gated block that keeps them, against their 64-bit
definitions: codes bit for bit, forward and backward of every size, type and
grouping, and the block's chain.

Tolerances: fp32 sums as in moe_ref; kept values are within half a step of E4M3 of
the fp32 ones (mx8_ref.check_kept); gradients through the derivatives of their
factors (mx8_ref.gated_bounds)."""
import math

import pytest
import torch

import moe_ref as ref
import mx8_ref as mx
import sharded_gemm_alltosharded_amd as sg

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    sg.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def offsets_of(g, E, R):
    w = torch.rand(E, generator=g)
    if E > 2:
        w[torch.randperm(E, generator=g)[: E // 3]] = 0
        w[0] += 0.1
    cuts = (torch.cumsum(w, 0) / w.sum() * R).round().int()
    return torch.cat([torch.zeros(1, dtype=torch.int32), cuts])


# ---- MX FP8 -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("shape", [(1, 1), (1, 32), (3, 31), (5, 33), (17, 4096), (4, 1003), (2, 3, 100), (64,), (0, 64),
                                   (300, 8), (7, 0)])
def test_quantize(shape, dtype):
    g = gen(sum(shape) + 1)
    x = normal(g, shape, F32) * torch.exp(2 * normal(g, (*shape[:-1], 1)))
    x = x.to(dtype)
    codes, scales = sg.quantize_mxfp8(x.cuda())
    wc, ws = mx.encode(x)
    assert torch.equal(scales.cpu(), ws) and torch.equal(codes.cpu(), wc)
    for out in (F32, BF, HF):
        got = sg.dequantize_mxfp8(codes, scales, out_dtype=out)
        assert torch.equal(got.cpu().double(), mx.decode(wc, ws).to(out).double())


def test_quantize_every_code_and_border():
    """All magnitudes, the middles between neighbours (ties go to the even code), and
    both sides of them, at scales from the smallest to the largest."""
    grid = mx.magnitudes()
    mid = (grid[1:] + grid[:-1]) / 2
    v = torch.cat([grid, mid, mid * (1 - 2.0 ** -20), mid * (1 + 2.0 ** -20)])
    v = torch.cat([v, -v])
    rows = []
    for e in (-127, -126, -100, -17, 0, 1, 60, 118, 119):
        for i in range(0, len(v), 31):
            r = torch.full((32,), 448.0, dtype=torch.float64)
            part = v[i:i + 31]
            r[1:1 + len(part)] = part
            rows.append(r * 2.0 ** e)
    x = torch.stack(rows).float()
    codes, scales = sg.quantize_mxfp8(x.cuda())
    wc, ws = mx.encode(x)
    assert torch.equal(scales.cpu(), ws) and torch.equal(codes.cpu(), wc)


def test_quantize_scale_borders():
    """A maximum of 448 2^e takes e, the next value above it e + 1; nothing saturates."""
    top = torch.tensor([448.0 * 2.0 ** k for k in (-130, -127, -126, -3, 0, 5, 119)], dtype=F32)
    x = torch.zeros((3, len(top), 32))
    x[0, :, 5], x[1, :, 5], x[2, :, 5] = top, torch.nextafter(top, torch.tensor(math.inf)), -torch.nextafter(top, torch.tensor(0.0))
    codes, scales = sg.quantize_mxfp8(x.cuda())
    wc, ws = mx.encode(x)
    assert torch.equal(scales.cpu(), ws) and torch.equal(codes.cpu(), wc)
    tiny = torch.tensor([0.0, -0.0, 2.0 ** -149, 2.0 ** -136, 2.0 ** -137, 3 * 2.0 ** -138, 2.0 ** -126] + [0.0] * 25)
    codes, scales = sg.quantize_mxfp8(tiny[None].cuda())
    wc, ws = mx.encode(tiny[None])
    assert torch.equal(scales.cpu(), ws) and torch.equal(codes.cpu(), wc)


@pytest.mark.parametrize("dtype", [F32, BF, HF])
def test_quantize_infinities_and_nans(dtype):
    x = torch.ones((3, 100), dtype=dtype)
    x[0, 40], x[1, 99], x[2, 0] = math.inf, math.nan, -math.inf
    codes, scales = sg.quantize_mxfp8(x.cuda())
    wc, ws = mx.encode(x)
    assert torch.equal(scales.cpu(), ws) and torch.equal(codes.cpu(), wc)
    assert (scales.cpu() == 255).sum() == 3
    back = sg.dequantize_mxfp8(codes, scales).cpu()
    want = torch.zeros((3, 4), dtype=torch.bool)
    want[0, 1] = want[1, 3] = want[2, 0] = True
    assert torch.equal(torch.isnan(back), want.repeat_interleave(32, 1)[:, :100])


def test_quantize_strided_and_unaligned():
    g = gen(4)
    wide = normal(g, (40, 131), HF).cuda()
    for at, n in ((0, 96), (3, 64), (1, 99)):
        a = sg.quantize_mxfp8(wide[:, at:at + n])
        b = sg.quantize_mxfp8(wide[:, at:at + n].contiguous())
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_quantize_past_2_31_values():
    n = (1 << 31) + 320
    x = torch.zeros((n // 320, 320), dtype=BF, device="cuda")
    x[-1, 300:] = torch.arange(20, device="cuda").to(BF)
    codes, scales = sg.quantize_mxfp8(x)
    wc, ws = mx.encode(x[-1:].cpu())
    assert torch.equal(codes[-1:].cpu(), wc) and torch.equal(scales[-1:].cpu(), ws)
    assert int(codes[:-1].max()) == 0 and int(scales[:-1].max()) == 0
    # (17 and 19 lie between two values of E4M3, whose step from 16 on is 2)
    assert torch.equal(sg.dequantize_mxfp8(codes, scales, out_dtype=BF)[-1:].cpu().double(), mx.decode(wc, ws))


# ---- the gated half ---------------------------------------------------------

# E, R, in, f, P, dtype: no tile, no scale block filled; odd blocks of 16 on several
# ranks; the widest tiles and their quarters
GATED = [
    (1, 1, 8, 1, 1, BF), (1, 3, 64, 32, 2, HF), (1, 200, 64, 16, 2, BF), (1, 777, 100, 363, 2, HF), (3, 50, 32, 20, 1, HF),
    (4, 130, 136, 33, 2, BF), (8, 100, 62, 48, 4, HF), (2, 300, 256, 130, 1, HF), (70, 90, 64, 16, 1, BF),
    (2, 1100, 192, 272, 1, BF), (1, 300, 35, 7, 3, BF), (1, 96, 512, 64, 8, BF), (5, 700, 200, 96, 2, BF),
]


def gated_case(E, R, K, f, P, dtype):
    g = gen(R + K + f)
    w = normal(g, (E, 2 * P * f, K), dtype, 1 / math.sqrt(K))
    off = offsets_of(g, E, R)
    T = max(1, R // 2)
    x = normal(g, (T, K), dtype, 2.0)
    rows = torch.randint(0, T * 2, (R,), generator=g, dtype=torch.int32)
    rows[R // 2] = -1  # reads zeros
    out, mag = torch.zeros((R, 2 * P * f), dtype=torch.float64), torch.zeros((R, 2 * P * f), dtype=torch.float64)
    ref.product(ref.gathered(x.double(), rows, 2), w.double(), off, out, mag)
    order = ref.shard_rows(2 * P * f, 2, P)
    pick = lambda v: torch.stack([v[:, o] for o in order]).unflatten(-1, (2, f))  # noqa: E731
    layer = sg.shard_experts(w.cuda(), "all-to-sharded", segments=2, P=P)
    return layer, x, off, rows, pick(out), pick(mag)


@pytest.mark.parametrize("case", GATED)
def test_gated_forward(case):
    E, R, K, f, P, dtype = case
    layer, x, off, rows, gu, mag = gated_case(*case)
    h, codes, scales = sg.experts_gated(layer, x.cuda(), off.cuda(), rows.cuda(), 2)
    end = int(off[-1])
    (g, u), (mg, mu) = (v[:, :end].unbind(2) for v in (gu, mag))
    ref.close(h[:, :end], ref.silu(g) * u, ref.swiglu_bound(g, u, mg, mu, K), "h")
    mx.check_kept(codes[:, :end], scales[:, :end], gu[:, :end], ref.sum_bound(mag[:, :end], K), "kept")
    # h is the one that the product without keeping gives, up to fp32's last steps
    plain = sg.experts_all_to_sharded(layer, x.cuda(), off.cuda(), rows.cuda(), 2, swiglu=True)
    ref.close(h[:, :end], plain[:, :end].double().cpu(), 2 * ref.HALF[dtype] * (ref.silu(g) * u).abs() +
              2 * ref.swiglu_bound(g, u, mg, mu, K), "h and the SwiGLU epilogue's")


def kept_case(g, P, R, f):
    gu = normal(g, (P, R, 2, f), F32, 2.0)
    gu[:, R // 3, 0] *= 50  # gates that saturate
    return mx.encode(gu)


@pytest.mark.parametrize("case", GATED)
def test_gated_backward(case):
    E, R, D, f, P, dtype = case  # D: the block's outputs
    g = gen(R + f)
    w = normal(g, (E, D, P * f), dtype, 1 / math.sqrt(P * f))
    off = offsets_of(g, E, R)
    codes, scales = kept_case(g, P, R, f)
    dy = normal(g, (R, D), dtype)
    down = sg.shard_experts(w.cuda(), "sharded-to-all", P=P)
    dgu, h = sg.experts_gated_backward(down, dy.cuda(), codes.cuda(), scales.cuda(), off.cuda())
    dh, mag = torch.zeros((R, P * f), dtype=torch.float64), torch.zeros((R, P * f), dtype=torch.float64)
    ref.product(dy.double(), w.double().transpose(1, 2), off, dh, mag)
    end = int(off[-1])
    dh, mag = (v.view(R, P, f).transpose(0, 1)[:, :end] for v in (dh, mag))
    gg, uu = mx.decode(codes, scales)[:, :end].unbind(2)
    wants, bounds = mx.gated_grad(gg, uu, dh), mx.gated_bounds(gg, uu, dh, ref.sum_bound(mag, D))
    got = (dgu[:, :end, :f].contiguous(), dgu[:, :end, f:].contiguous(), h[:, :end])
    for v, want, bound, name in zip(got, wants, bounds, ("dgate", "dup", "h")):
        ref.close(v, want, bound, name)
    only, none = sg.experts_gated_backward(down, dy.cuda(), codes.cuda(), scales.cuda(), off.cuda(), need_h=False)
    assert none is None and torch.equal(only[:, :end], dgu[:, :end])


# the wide tiles, their quarters and the narrow ones, on rows that end inside them:
# E, R, in, f, P, dtype
WIDE = [(1, 2600, 96, 2304, 1, BF), (1, 2600, 72, 752, 4, HF), (3, 2000, 64, 2104, 1, HF), (2, 4700, 136, 1024, 2, BF),
        (1, 700, 64, 8200, 1, BF), (1, 4100, 40, 2501, 1, BF)]


@pytest.mark.parametrize("E,R,K,f,P,dtype", WIDE)
def test_gated_wide_tiles(E, R, K, f, P, dtype):
    """Sampled rows, forward and backward, at sizes that take the widest tiles."""
    g = gen(R + f)
    w = normal(g, (E, 2 * P * f, K), dtype, 1 / math.sqrt(K))
    wd = normal(g, (E, K, P * f), dtype, 1 / math.sqrt(P * f))
    x = normal(g, (R, K), dtype)
    off = offsets_of(g, E, R)
    off[-1] = R
    pick = torch.unique(torch.cat([torch.randint(0, R, (60,), generator=g), off[1:].long() - 1,
                                   torch.tensor([0, 127, 128, 255, 256, R - 1])]))
    pick = pick[pick >= 0]
    expert = torch.searchsorted(off[1:].contiguous(), pick.int(), right=True)
    order = ref.shard_rows(2 * P * f, 2, P)
    shard = lambda v: torch.stack([v[:, o] for o in order]).unflatten(-1, (2, f))  # noqa: E731
    gu = shard(torch.stack([w[e].double() @ x[m].double() for m, e in zip(pick, expert)]))
    mag = shard(torch.stack([w[e].double().abs() @ x[m].double().abs() for m, e in zip(pick, expert)]))
    up = sg.shard_experts(w.cuda(), "all-to-sharded", segments=2, P=P)
    down = sg.shard_experts(wd.cuda(), "sharded-to-all", P=P)
    h, codes, scales = sg.experts_gated(up, x.cuda(), off.cuda())
    (a, b), (ma, mb) = gu.unbind(2), mag.unbind(2)
    at = pick.cuda()
    ref.close(h[:, at], ref.silu(a) * b, ref.swiglu_bound(a, b, ma, mb, K), "h")
    mx.check_kept(codes[:, at], scales[:, at], gu, ref.sum_bound(mag, K), "kept")
    dgu, h2 = sg.experts_gated_backward(down, x.cuda(), codes, scales, off.cuda())
    dh = torch.stack([x[m].double() @ wd[e].double() for m, e in zip(pick, expert)]).view(-1, P, f).transpose(0, 1)
    md = torch.stack([x[m].double().abs() @ wd[e].double().abs() for m, e in zip(pick, expert)]).view(-1, P, f).transpose(0, 1)
    gg, uu = mx.decode(codes[:, at].cpu(), scales[:, at].cpu()).unbind(2)
    wants, bounds = mx.gated_grad(gg, uu, dh), mx.gated_bounds(gg, uu, dh, ref.sum_bound(md, K))
    got = (dgu[:, at, :f].contiguous(), dgu[:, at, f:].contiguous(), h2[:, at])
    for v, want, bound, name in zip(got, wants, bounds, ("dgate", "dup", "h")):
        ref.close(v, want, bound, name)


def test_gated_rows_behind_the_last_stay():
    g = gen(2)
    E, R, K, f, P = 3, 40, 64, 48, 2
    layer = sg.shard_experts(normal(g, (E, 2 * P * f, K), BF, 0.1).cuda(), "all-to-sharded", segments=2, P=P)
    down = sg.shard_experts(normal(g, (E, K, P * f), BF, 0.1).cuda(), "sharded-to-all", P=P)
    off = torch.tensor([0, 9, 9, 23], dtype=torch.int32).cuda()
    x = normal(g, (R, K), BF)
    x[23:] = math.nan
    h = torch.full((P, R, f), 7.0, dtype=BF, device="cuda")
    codes = torch.full((P, R, 2, f), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((P, R, 2, 2), 9, dtype=torch.uint8, device="cuda")
    L, at = sg.lib(), lambda t: t.data_ptr()  # noqa: E731
    xc = x.cuda()
    ws = torch.empty(L.sg_experts_gated_workspace(layer.handle, R), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert L.sg_experts_gated(layer.handle, at(xc), R, K, at(off), None, 1, R, at(h), at(codes), at(scales), at(ws),
                              ws.numel(), s) == 0
    assert (h[:, 23:] == 7).all() and (codes[:, 23:] == 9).all() and (scales[:, 23:] == 9).all()
    assert torch.isfinite(h[:, :23]).all() and (scales[:, :23] != 255).all()
    dgu = torch.full((P, R, 2 * f), 7.0, dtype=BF, device="cuda")
    h2 = torch.full((P, R, f), 7.0, dtype=BF, device="cuda")
    assert L.sg_experts_gated_backward(down.handle, at(xc), at(codes), at(scales), at(off), R, at(dgu), at(h2), s) == 0
    assert (dgu[:, 23:] == 7).all() and (h2[:, 23:] == 7).all() and torch.isfinite(dgu[:, :23]).all()


def test_gated_infinities_are_kept_as_nan_blocks():
    """An infinite input spoils its own token's blocks only."""
    g = gen(3)
    layer = sg.shard_experts(normal(g, (1, 128, 64), BF, 0.1).cuda(), "all-to-sharded", segments=2)
    x = normal(g, (20, 64), BF)
    clean = sg.experts_gated(layer, x.cuda())
    x[7, 3] = math.inf
    h, codes, scales = sg.experts_gated(layer, x.cuda())
    keep = [i for i in range(20) if i != 7]
    assert (scales[0, 7] == 255).all() and (codes[0, 7] == 0).all()
    for a, b in zip((h, codes, scales), clean):
        assert torch.equal(a[:, keep], b[:, keep])


# ---- the block --------------------------------------------------------------

BLOCKS = [  # E, T, D, F, out, P, dtype; the last ones' sums are split
    (1, 1, 8, 8, 8, 1, BF), (1, 77, 100, 726, 60, 2, HF), (1, 300, 256, 512, 256, 4, BF), (3, 150, 72, 96, 40, 2, BF),
    (1, 1000, 136, 320, 136, 1, HF), (1, 33, 77, 1030, 50, 2, BF), (1, 100, 1024, 2048, 512, 4, HF),
    (1, 12, 200, 3000, 90, 3, BF),
]


@pytest.mark.parametrize("E,T,D,F,N,P,dtype", BLOCKS)
def test_block_is_the_chain_of_its_calls(E, T, D, F, N, P, dtype):
    g = gen(T + D)
    wg = normal(g, (E, 2 * F, D), dtype, 1 / math.sqrt(D))
    gu = sg.shard_experts(wg.cuda(), "all-to-sharded", segments=2, P=P)
    wd = normal(g, (E, N, F), dtype, 1 / math.sqrt(F))
    dn = sg.shard_experts(wd.cuda(), "sharded-to-all", P=P)
    x = normal(g, (T, D), dtype).cuda()
    kw = {}
    R = T
    if E > 1:  # every token through two of the experts
        route = sg.moe_route(normal(g, (T, E)).cuda(), 2)
        R = 2 * T
        kw = dict(offsets=route.offsets, rows=route.rows, k=2)
    off = dict(offsets=kw.get("offsets"))
    dy = normal(g, (R, N), dtype).cuda()
    y, kept = sg.gated_mlp(gu, dn, x, **kw)
    h, codes, scales = sg.experts_gated(gu, x, **kw)
    xc, xs = sg.quantize_mxfp8(x)
    for a, b in zip(kept, (xc, xs, codes, scales)):
        assert torch.equal(a, b)
    # y's and dx's sums may be split: fp32 sums of the same products, rounded alike
    yw, w = sg.experts_sharded_to_all(dn, h, out_dtype=F32, **off).double().cpu(), P * F // P
    mag = torch.zeros((R, N), dtype=torch.float64)
    ends = torch.tensor([0, R]) if E == 1 else kw["offsets"].cpu()
    full = h.double().cpu().transpose(0, 1).flatten(1).abs()
    ref.product(full, wd.double().abs(), ends, torch.zeros_like(mag), mag)
    ref.close(y, yw, 2 * ref.sum_bound(mag, w), "y")
    for dt in (dtype, F32):
        dx, dwg, dwd = sg.gated_mlp_backward(gu, dn, kept, dy, dx_dtype=dt, dw_dtype=dt, **kw)
        dgu, h2 = sg.experts_gated_backward(dn, dy, codes, scales, **off)
        x8 = sg.dequantize_mxfp8(xc, xs, out_dtype=dtype)
        _, ww = sg.experts_all_to_sharded_backward(gu, x8, dgu, dw_dtype=dt, **kw)
        wx, _ = sg.experts_all_to_sharded_backward(gu, None, dgu, need_dw=False, dx_dtype=F32, **kw)
        _, wn = sg.experts_sharded_to_all_backward(dn, h2, dy, need_dx=False, dw_dtype=dt, **off)
        assert torch.equal(dwg, ww) and torch.equal(dwd, wn)
        order = ref.shard_rows(2 * F, 2, P)
        full = torch.zeros((R, 2 * F), dtype=torch.float64)
        for r, o in enumerate(order):
            full[:, o] = dgu[r].double().cpu().abs()
        mx_ = torch.zeros((R, D), dtype=torch.float64)
        ref.product(full, wg.double().transpose(1, 2), ends, torch.zeros_like(mx_), mx_)
        ref.close(dx, wx.double().cpu(), 2 * ref.sum_bound(mx_, 2 * F), "dx")
    only, n1, n2 = sg.gated_mlp_backward(gu, dn, kept, dy, need_dw=False, dx_dtype=F32, **kw)
    assert n1 is None and n2 is None and torch.equal(only, dx)
    none, w1, w2 = sg.gated_mlp_backward(gu, dn, kept, dy, need_dx=False, **kw)
    assert none is None and torch.equal(w1, dwg) and torch.equal(w2, dwd)


def test_block_gradients_by_differences():
    """The gradients against the formulas, and those against differences of the block,
    on values that E4M3 holds exactly, so that what was kept is the block's own."""
    g = gen(9)
    T, D, F = 24, 32, 64
    pick = lambda shape, vals: torch.tensor(vals)[torch.randint(0, len(vals), shape, generator=g)]  # noqa: E731
    x = pick((T, D), [-1.0, -0.5, 0.0, 0.5, 1.0])
    # one +-1 weight a row: gate and up are inputs again, which E4M3 holds
    wg = torch.zeros((2 * F, D))
    wg[torch.arange(2 * F), torch.randint(0, D, (2 * F,), generator=g)] = pick((2 * F,), [-1.0, 1.0])
    wd = pick((D, F), [-0.5, -0.25, 0.25, 0.5])
    dy = pick((T, D), [-1.0, 1.0, 0.5])
    gu = sg.shard_experts(wg.to(BF).cuda()[None], "all-to-sharded", segments=2)
    dn = sg.shard_experts(wd.to(BF).cuda()[None], "sharded-to-all")
    _, kept = sg.gated_mlp(gu, dn, x.to(BF).cuda())
    z = x.double() @ wg.double().T
    assert torch.equal(mx.decode(kept.gu_codes.cpu(), kept.gu_scales.cpu())[0].flatten(1), z)
    assert torch.equal(mx.decode(kept.x_codes.cpu(), kept.x_scales.cpu()), x.double())
    dx, dwg, dwd = sg.gated_mlp_backward(gu, dn, kept, dy.to(BF).cuda(), dx_dtype=F32)

    # the formulas, and what the stored dgu and h (bf16: half a step, 2^-8, of every
    # term) and the fp32 sums may be off by
    a, b = z.split(F, 1)
    w, c, d = wg.double(), wd.double(), dy.double()
    dh = d @ c
    da, db, h = mx.gated_grad(a, b, dh)
    dgu = torch.cat([da, db], 1)
    ea, eb, eh = mx.gated_bounds(a, b, dh, ref.sum_bound(d.abs() @ c.abs(), D))
    e = torch.cat([ea, eb], 1) + 2.0 ** -8 * (dgu.abs() + torch.cat([ea, eb], 1))
    eh = eh + 2.0 ** -8 * (h.abs() + eh)
    fx, fg, fd = dgu @ w, dgu.T @ x.double(), d.T @ h
    ref.close(dx, fx, e @ w.abs() + ref.sum_bound((dgu.abs() + e) @ w.abs(), 2 * F), "dx")
    ref.close(dwg[0, 0], fg, e.T @ x.double().abs() + ref.sum_bound((dgu.abs() + e).T @ x.double().abs(), T), "dw gate_up")
    ref.close(dwd[0, 0], fd, d.abs().T @ eh + ref.sum_bound(d.abs().T @ (h.abs() + eh), T), "dw down")

    def loss(p, q, r):
        v = p @ q.T
        return ((ref.silu(v[:, :F]) * v[:, F:]) @ r.T * d).sum()

    args = [x.double(), w, c]
    for i, grad in enumerate((fx, fg, fd)):
        for _ in range(3):
            v = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
            step = 1e-5
            hi, lo = (loss(*(p + (sgn * step * v if j == i else 0) for j, p in enumerate(args))) for sgn in (1, -1))
            # differences: off by step^2 times third derivatives, and 2^-53 of the losses over the step
            assert abs((v * grad).sum() - (hi - lo) / (2 * step)) <= 1e-6 * (v.abs() * grad.abs()).sum()


def test_block_without_tokens():
    g = gen(1)
    gu = sg.shard_experts(normal(g, (1, 64, 32), BF).cuda(), "all-to-sharded", segments=2)
    dn = sg.shard_experts(normal(g, (1, 32, 32), BF).cuda(), "sharded-to-all")
    y, kept = sg.gated_mlp(gu, dn, torch.empty((0, 32), dtype=BF, device="cuda"))
    assert y.shape == (0, 32) and kept.gu_codes.shape == (1, 0, 2, 32)
    dx, a, b = sg.gated_mlp_backward(gu, dn, kept, y)
    assert dx.shape == (0, 32) and (a == 0).all() and (b == 0).all()


def test_block_on_another_stream_and_in_a_graph():
    g = gen(12)
    gu = sg.shard_experts(normal(g, (1, 256, 96), BF, 0.1).cuda(), "all-to-sharded", segments=2, P=2)
    dn = sg.shard_experts(normal(g, (1, 96, 128), BF, 0.1).cuda(), "sharded-to-all", P=2)
    xs = [normal(g, (150, 96), BF).cuda() for _ in range(4)]
    dys = [normal(g, (150, 96), BF).cuda() for _ in range(4)]

    def step(x, dy):
        y, kept = sg.gated_mlp(gu, dn, x)
        return (y, *kept, *sg.gated_mlp_backward(gu, dn, kept, dy))

    want = [step(a, b) for a, b in zip(xs, dys)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step(xs[0], dys[0])
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    x, dy = xs[0].clone(), dys[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, dy)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        dy.copy_(dys[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
        step(xs[i], dys[i])  # eager work between the replays
