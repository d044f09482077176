"""The mixture-of-experts operators against their 64-bit definitions: grouped
products of every direction and type, the router and its plan, the weighted
sum, SwiGLU, and their gradients; sizes that fill no tile, experts without
rows, masked tokens, strided inputs, other streams and graph capture.

Tolerances: an fp32 sum of n products is off by at most n half steps of its sum
of magnitudes, whatever its order; a stored result adds half a step of its type
(moe_ref.close)."""
import math

import pytest
import torch

import moe_ref as ref
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


def offsets_of(g, E, R, empty=True):
    """Ragged counts that add up to R, some of them zero."""
    w = torch.rand(E, generator=g)
    if empty and E > 2:
        w[torch.randperm(E, generator=g)[: E // 3]] = 0
        w[0] += 0.1
    cuts = (torch.cumsum(w, 0) / w.sum() * R).round().int()
    return torch.cat([torch.zeros(1, dtype=torch.int32), cuts])


# ---- router -----------------------------------------------------------------

ROUTES = [  # T, E, k, dtype
    (1, 1, 1, F32), (1, 64, 8, BF), (8, 64, 8, F32), (7, 3, 3, HF), (33, 65, 5, F32), (256, 8, 2, BF),
    (200, 200, 10, F32), (300, 128, 8, BF), (1500, 300, 16, HF), (3000, 40, 1, F32), (257, 1024, 4, F32),
    (1100, 600, 3, BF),
]


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", ROUTES)
def test_route(T, E, k, dtype, normalize):
    g = gen(T * 7 + E + k)
    z = normal(g, (T, E), dtype, 2.0)
    z[torch.rand((T, E), generator=g) < 0.15] = -math.inf
    z[T - T // 8:] = -math.inf  # padding
    w, e, off, rows, slots = ref.route(z, k, normalize)
    r = sg.moe_route(z.cuda(), k, normalize)
    assert torch.equal(r.experts.cpu(), e)
    assert torch.equal(r.offsets.cpu(), off)
    assert torch.equal(r.rows.cpu(), rows)
    assert torch.equal(r.slots.cpu(), slots)
    # weights: exp of a difference that is exact but for one fp32 rounding
    # (2^-24 |z - top|, at most 2^-24 * 40 where the weight counts), a sum of E
    # terms, a quotient
    ref.close(r.weights, w, (E + 64) * 2.0 ** -24 * w, "weights")


def test_route_ties_go_to_the_lowest_expert():
    z = torch.tensor([[1.0, 2.0, 2.0, 0.0, 2.0], [0.0, -0.0, 0.0, -0.0, -1.0], [3.0] * 5])
    r = sg.moe_route(z.cuda(), 3)
    assert r.experts.tolist() == [[1, 2, 4], [0, 1, 2], [0, 1, 2]]
    assert r.rows.tolist() == [3, 6, 0, 4, 7, 1, 5, 8, 2]


def test_route_closed_experts():
    inf, nan = math.inf, math.nan
    low = torch.finfo(F32).min
    z = torch.tensor([[-inf, -inf, -inf], [nan, 1.0, nan], [low, low, -inf], [nan, nan, -inf], [0.0, -inf, low]])
    for normalize in (True, False):
        r = sg.moe_route(z.cuda(), 2, normalize)
        assert r.experts.tolist() == [[-1, -1], [1, -1], [0, 1], [-1, -1], [0, 2]]
        assert r.weights.tolist() == [[0, 0], [1, 0], [0.5, 0.5], [0, 0], [1, 0]]
        assert r.offsets.tolist() == [0, 2, 4, 5]
        assert r.rows.tolist() == [4, 8, 2, 5, 9] + [-1] * 5
        assert r.slots.tolist() == [[-1, -1], [2, -1], [0, 3], [-1, -1], [1, 4]]


def test_route_strided_logits():
    g = gen(3)
    wide = normal(g, (50, 40), BF).cuda()
    z = wide[:, 3:19]
    a, b = sg.moe_route(z, 4), sg.moe_route(z.contiguous(), 4)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_route_no_tokens():
    r = sg.moe_route(torch.empty((0, 5), device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 6 and r.weights.shape == (0, 2)


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, F32), (9, 5, 3, F32), (130, 64, 8, F32), (70, 200, 6, BF),
                                         (40, 1000, 16, HF)])
def test_route_backward(T, E, k, dtype, normalize):
    g = gen(E + k)
    z = normal(g, (T, E), dtype, 1.5)
    z[torch.rand((T, E), generator=g) < 0.2] = -math.inf
    z[T - T // 8:] = -math.inf
    dw = normal(g, (T, k))
    r = sg.moe_route(z.cuda(), k, normalize)
    dz = sg.moe_route_backward(z.cuda(), r, dw.cuda(), normalize)
    e = r.experts.cpu()
    want = ref.route_backward(z, e, dw, normalize)
    # p (g - sum p g): p off by (E + 64) half steps, the sum by k more
    mag = dw.abs().amax(1, keepdim=True).double()
    ref.close(dz, want, 4 * (E + 80) * 2.0 ** -24 * mag.expand_as(want), "dlogits")
    assert (dz.cpu()[torch.isinf(z)] == 0).all()


def test_route_backward_by_differences():
    g = gen(11)
    T, E, k = 6, 12, 4
    z, dw = normal(g, (T, E)).double(), normal(g, (T, k)).double()
    for normalize in (True, False):
        _, e, *_ = ref.route(z, k, normalize)
        d = ref.route_backward(z, e, dw, normalize)
        step = 1e-6
        for t in range(T):
            for c in range(E):
                up, dn = z.clone(), z.clone()
                up[t, c] += step
                dn[t, c] -= step
                f = [(ref.route(v, k, normalize)[0] * dw).sum() for v in (up, dn)]
                assert abs((f[0] - f[1]) / (2 * step) - d[t, c]) < 1e-7
        r = sg.moe_route(z.float().cuda(), k, normalize)
        got = sg.moe_route_backward(z.float().cuda(), r, dw.float().cuda(), normalize)
        want = ref.route_backward(z.float(), e, dw.float(), normalize)
        ref.close(got, want, torch.full_like(want, 400 * 2.0 ** -24 * dw.abs().max().item()), "dlogits")


# ---- weighted sum -----------------------------------------------------------

@pytest.mark.parametrize("dtype,out_dtype", [(F32, BF), (BF, BF), (HF, F32), (F32, F32)])
@pytest.mark.parametrize("T,k,D", [(1, 1, 1), (5, 3, 8), (17, 2, 1000), (40, 8, 2056), (9, 16, 4096), (33, 4, 37)])
def test_combine(T, k, D, dtype, out_dtype):
    g = gen(T + D)
    R = T * k
    y = normal(g, (R, D), dtype)
    slots = torch.randperm(R, generator=g).int().view(T, k)
    slots[torch.rand((T, k), generator=g) < 0.2] = -1
    slots[0, 0] = R + 5  # outside: left out
    w = torch.rand((T, k), generator=g)
    ok = (slots >= 0) & (slots < R)
    pick = torch.where(ok[..., None], y.double()[slots.long().clamp(0, R - 1)], 0.0)
    for weights in (w, None):
        ww = (w if weights is not None else torch.ones_like(w)).double()[..., None]
        want, mag = (ww * pick).sum(1), (ww * pick.abs()).sum(1)
        got = sg.moe_combine(y.cuda(), slots.cuda(), None if weights is None else w.cuda(), out_dtype=out_dtype)
        ref.close(got, want, ref.sum_bound(mag, k), "combine")


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("T,k,D", [(1, 1, 1), (5, 3, 8), (17, 2, 1000), (12, 8, 2056), (9, 16, 37)])
def test_combine_backward(T, k, D, dtype):
    g = gen(T + D)
    R = T * k + 3
    y, dout = normal(g, (R, D), dtype), normal(g, (T, D), dtype)
    slots = torch.randperm(R, generator=g)[: T * k].int().view(T, k)
    slots[torch.rand((T, k), generator=g) < 0.2] = -1
    w = torch.rand((T, k), generator=g)
    mark = torch.full((R, D), 7.0, dtype=dtype)
    dy, dw = sg.moe_combine_backward(dout.cuda(), y.cuda(), slots.cuda(), w.cuda(), dy=mark.cuda())
    ok = slots >= 0
    want = mark.double()
    used = slots[ok].long()
    prod = (w.double()[..., None] * dout.double()[:, None])[ok]
    want[used] = prod
    ref.close(dy, want, 2.0 ** -24 * want.abs(), "dy")
    untouched = torch.ones(R, dtype=torch.bool)
    untouched[used] = False
    assert (dy.cpu()[untouched] == 7).all()
    pick = torch.where(ok[..., None], y.double()[slots.long().clamp(0)], 0.0)
    dots, mag = (pick * dout.double()[:, None]).sum(-1), (pick * dout.double()[:, None]).abs().sum(-1)
    ref.close(dw, dots, ref.sum_bound(mag, D), "dweights")
    only, none = sg.moe_combine_backward(dout.cuda(), y.cuda(), slots.cuda(), w.cuda(), need_dweights=False)
    assert none is None and (only.cpu()[untouched] == 0).all()
    assert torch.equal(only.cpu()[used], dy.cpu()[used])


# ---- SwiGLU -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("shape", [(1, 2), (3, 7, 16), (2, 5, 726), (4, 130)])
def test_swiglu(shape, dtype):
    g = gen(sum(shape))
    gu = normal(g, shape, dtype, 3.0)
    f = shape[-1] // 2
    dh = normal(g, (*shape[:-1], f), dtype)
    a, b = gu.double().split(f, -1)
    h = ref.silu(a) * b
    ref.close(sg.swiglu(gu.cuda()), h, 16 * 2.0 ** -24 * h.abs(), "h")
    a.requires_grad_(True), b.requires_grad_(True)
    da, db = torch.autograd.grad((ref.silu(a) * b * dh.double()).sum(), (a, b))
    d = sg.swiglu_backward(gu.cuda(), dh.cuda())
    # dg's factor s (1 + g (1 - s)) is a difference for negative g: its terms' magnitudes
    s = 1 / (1 + torch.exp(-a.detach()))
    mag = (dh.double() * b.detach() * s).abs() * (1 + a.detach().abs() * (1 - s))
    ref.close(d[..., :f].contiguous(), da, 16 * 2.0 ** -24 * mag, "dgate")
    ref.close(d[..., f:].contiguous(), db, 16 * 2.0 ** -24 * db.abs(), "dup")


def test_swiglu_far_values():
    big = [-1e30, -200.0, -90.0, 0.0, 90.0, 1e30]
    gu = torch.tensor([[a, 1.0] for a in big])
    h = sg.swiglu(gu.cuda()).cpu().flatten().tolist()
    assert h[3] == 0 and h[4] == 90 and h[5] == pytest.approx(1e30) and all(abs(v) < 1e-30 for v in h[:3])
    d = sg.swiglu_backward(gu.cuda(), torch.ones((6, 1)).cuda())
    assert torch.isfinite(d).all()


# ---- grouped products -------------------------------------------------------

# E, R, in, out / P / S, P, S, dtype
COLUMNS = [
    (1, 1, 8, 1, 1, 1, BF), (1, 200, 64, 16, 2, 2, BF), (3, 5, 32, 20, 1, 2, HF), (4, 64, 136, 33, 2, 2, BF),
    (8, 100, 62, 24, 4, 2, HF), (5, 700, 1000, 48, 2, 1, BF), (2, 300, 256, 130, 1, 2, HF), (6, 40, 520, 16, 8, 2, BF),
    (70, 90, 64, 16, 1, 2, BF), (4, 513, 320, 64, 3, 3, BF), (2, 1100, 192, 272, 1, 2, BF), (1, 300, 35, 7, 3, 2, BF),
    (100, 1300, 72, 24, 1, 2, HF), (130, 2000, 33, 5, 2, 2, BF),
    (2, 2, 2048, 256, 1, 2, BF), (1, 5, 2051, 40, 2, 2, HF), (3, 17, 2500, 24, 1, 1, BF),
]


def column_case(E, R, K, f, P, S, dtype, swiglu):
    g = gen(R + K + f)
    n = f * P * S
    w = normal(g, (E, n, K), dtype, 1 / math.sqrt(K))
    T = max(1, R // 2)
    x = normal(g, (T, K), dtype)
    off = offsets_of(g, E, R)
    rows = torch.randint(0, T * 2, (R,), generator=g, dtype=torch.int32)
    rows[R // 2] = -1  # reads zeros
    out, mag = torch.zeros((R, n), dtype=torch.float64), torch.zeros((R, n), dtype=torch.float64)
    ref.product(ref.gathered(x.double(), rows, 2), w.double(), off, out, mag)
    layer = sg.shard_experts(w.cuda(), "all-to-sharded", segments=S, P=P)
    order = ref.shard_rows(n, S, P)
    res, bound = torch.stack([out[:, o] for o in order]), torch.stack([mag[:, o] for o in order])
    if swiglu:
        (a, b), (ma, mb) = res.split(f, -1), bound.split(f, -1)
        return layer, x, off, rows, ref.silu(a) * b, ref.swiglu_bound(a, b, ma, mb, K)
    return layer, x, off, rows, res, ref.sum_bound(bound, K)


@pytest.mark.parametrize("case", COLUMNS)
def test_experts_column(case):
    S, dtype = case[5], case[6]
    for swiglu in ([False, True] if S == 2 else [False]):
        layer, x, off, rows, want, bound = column_case(*case, swiglu)
        for out_dtype in (dtype, F32):
            got = sg.experts_all_to_sharded(layer, x.cuda(), off.cuda(), rows.cuda(), 2, swiglu, out_dtype=out_dtype)
            ref.close(got, want, bound, f"column swiglu={swiglu} {out_dtype}")


ROWS = [  # E, R, out, in / P, P, S, dtype
    (1, 1, 1, 8, 1, 1, BF), (1, 150, 64, 64, 2, 1, BF), (3, 5, 20, 32, 1, 1, HF), (4, 64, 33, 96, 3, 1, BF),
    (8, 100, 250, 31, 4, 1, HF), (5, 700, 72, 363, 2, 1, BF), (2, 300, 1000, 128, 8, 1, HF), (6, 40, 16, 40, 8, 2, BF),
    (70, 90, 48, 64, 1, 1, BF), (3, 900, 300, 88, 4, 1, BF), (1, 2, 32, 523, 4, 1, BF), (3, 4, 700, 1100, 2, 2, HF),
    (2, 100, 24, 5, 3, 1, BF), (2, 1500, 1030, 1001, 1, 1, HF),
]


def row_case(E, R, n, kr, P, S, dtype):
    g = gen(R + n + kr)
    K = kr * P
    w = normal(g, (E, n, K), dtype, 1 / math.sqrt(K))
    h = normal(g, (P, R, kr), dtype)
    off = offsets_of(g, E, R)
    layer = sg.shard_experts(w.cuda(), "sharded-to-all", segments=S, P=P)
    order = ref.shard_rows(K, S, P)
    return w, h, off, layer, order


@pytest.mark.parametrize("case", ROWS)
def test_experts_row(case):
    E, R, n, kr, P, S, dtype = case
    w, h, off, layer, order = row_case(*case)
    out, mag = torch.zeros((R, n), dtype=torch.float64), torch.zeros((R, n), dtype=torch.float64)
    full = torch.zeros((R, kr * P), dtype=torch.float64)
    for r, o in enumerate(order):
        full[:, o] = h[r].double()
    ref.product(full, w.double(), off, out, mag)
    for out_dtype in (dtype, F32):
        got = sg.experts_sharded_to_all(layer, h.cuda(), off.cuda(), out_dtype=out_dtype)
        ref.close(got, out, ref.sum_bound(mag, kr * P), f"row {out_dtype}")


@pytest.mark.parametrize("case", COLUMNS)
def test_experts_column_backward(case):
    E, R, K, f, P, S, dtype = case
    layer, x, off, rows, _, _ = column_case(*case, False)
    g = gen(1)
    n = f * P * S
    w = normal(gen(R + K + f), (E, n, K), dtype, 1 / math.sqrt(K)).double()
    dy = normal(g, (P, R, f * S), dtype)
    order = ref.shard_rows(n, S, P)
    full = torch.zeros((R, n), dtype=torch.float64)
    for r, o in enumerate(order):
        full[:, o] = dy[r].double()
    dx, mx = torch.zeros((R, K), dtype=torch.float64), torch.zeros((R, K), dtype=torch.float64)
    ref.product(full, w.transpose(1, 2), off, dx, mx)
    xg = ref.gathered(x.double(), rows, 2)
    for dt in (dtype, F32):
        gx, gw = sg.experts_all_to_sharded_backward(layer, x.cuda(), dy.cuda(), off.cuda(), rows.cuda(), 2,
                                                    dx_dtype=dt, dw_dtype=dt)
        ref.close(gx, dx, ref.sum_bound(mx, n), f"dx {dt}")
        for e in range(E):
            a, b = int(off[e]), int(off[e + 1])
            for r, o in enumerate(order):
                d, m = full[a:b][:, o].T @ xg[a:b], full[a:b][:, o].abs().T @ xg[a:b].abs()
                ref.close(gw[e, r], d, ref.sum_bound(m, b - a), f"dw {dt} {e} {r}")
    only, none = sg.experts_all_to_sharded_backward(layer, None, dy.cuda(), off.cuda(), need_dw=False, dx_dtype=F32)
    assert none is None and torch.equal(only, gx)


@pytest.mark.parametrize("case", ROWS)
def test_experts_row_backward(case):
    E, R, n, kr, P, S, dtype = case
    w, h, off, layer, order = row_case(*case)
    dy = normal(gen(2), (R, n), dtype)
    dh, mh = torch.zeros((R, kr * P), dtype=torch.float64), torch.zeros((R, kr * P), dtype=torch.float64)
    ref.product(dy.double(), w.double().transpose(1, 2), off, dh, mh)
    want, bound = torch.stack([dh[:, o] for o in order]), torch.stack([mh[:, o] for o in order])
    for dt in (dtype, F32):
        gh, gw = sg.experts_sharded_to_all_backward(layer, h.cuda(), dy.cuda(), off.cuda(), dx_dtype=dt, dw_dtype=dt)
        ref.close(gh, want, ref.sum_bound(bound, n), f"dh {dt}")
        for e in range(E):
            a, b = int(off[e]), int(off[e + 1])
            for r in range(P):
                d, m = dy[a:b].double().T @ h[r, a:b].double(), dy[a:b].double().abs().T @ h[r, a:b].double().abs()
                ref.close(gw[e, r], d, ref.sum_bound(m, b - a), f"dw {dt} {e} {r}")


# the wide tiles, their quarters and the narrow ones, on rows that end inside
# them: E, R, in, out / P / S, P, S, dtype
WIDE = [
    (1, 2600, 96, 2304, 1, 2, BF), (1, 2600, 72, 1500, 3, 1, HF), (3, 2000, 64, 2104, 1, 2, HF),
    (2, 4700, 136, 1024, 2, 2, BF), (5, 3000, 200, 3000, 1, 1, BF), (1, 700, 64, 16392, 1, 1, HF),
]


@pytest.mark.parametrize("E,R,K,f,P,S,dtype", WIDE)
def test_experts_wide_tiles(E, R, K, f, P, S, dtype):
    """Sampled rows of the products, and of both gradients, at sizes that take the widest tiles."""
    g = gen(R + f)
    n = f * P * S
    w, x = normal(g, (E, n, K), dtype, 1 / math.sqrt(K)), normal(g, (R, K), dtype)
    off = offsets_of(g, E, R, empty=False)
    order = ref.shard_rows(n, S, P)
    col = sg.shard_experts(w.cuda(), "all-to-sharded", segments=S, P=P)
    pick = torch.unique(torch.cat([torch.randint(0, R, (40,), generator=g), off[1:-1].long(), off[1:].long() - 1,
                                   torch.tensor([0, 127, 128, 255, 256, R - 1])]))
    pick = pick[pick < R]
    expert = torch.searchsorted(off[1:].contiguous(), pick.int(), right=True)
    y = torch.stack([w[e].double() @ x[r].double() for r, e in zip(pick, expert)])
    mag = torch.stack([w[e].double().abs() @ x[r].double().abs() for r, e in zip(pick, expert)])
    res, bound = torch.stack([y[:, o] for o in order]), torch.stack([mag[:, o] for o in order])
    got = sg.experts_all_to_sharded(col, x.cuda(), off.cuda(), out_dtype=F32)
    ref.close(got[:, pick.cuda()], res, ref.sum_bound(bound, K), "column")
    if S == 2:
        h = sg.experts_all_to_sharded(col, x.cuda(), off.cuda(), swiglu=True)
        (a, b), (ma, mb) = res.split(f, -1), bound.split(f, -1)
        ref.close(h[:, pick.cuda()], ref.silu(a) * b, ref.swiglu_bound(a, b, ma, mb, K), "swiglu")
    # the same weights transposed: dx of a layer whose inputs are the wide side
    row = sg.shard_experts(w.transpose(1, 2).contiguous().cuda(), "sharded-to-all", segments=S, P=P)
    dh, dw = sg.experts_sharded_to_all_backward(row, got.to(dtype), x.cuda(), off.cuda(), dx_dtype=F32)
    ref.close(dh[:, pick.cuda()], res, ref.sum_bound(bound, K), "dh")
    o = torch.randint(0, K, (5,), generator=g)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        hs = got[:, a:b].to(dtype).double().cpu()
        for r in range(P):
            d = x[a:b, o].double().T @ hs[r]
            m = x[a:b, o].double().abs().T @ hs[r].abs()
            ref.close(dw[e, r][o.cuda()], d, ref.sum_bound(m, b - a), f"dw {e} {r}")
    # and back: the wide side summed over
    dy = normal(g, (P, R, f * S), dtype)
    full = torch.zeros((len(pick), n), dtype=torch.float64)
    for r, q in enumerate(order):
        full[:, q] = dy[r, pick].double()
    dx, _ = sg.experts_all_to_sharded_backward(col, None, dy.cuda(), off.cuda(), need_dw=False, dx_dtype=F32)
    want = torch.stack([full[i] @ w[e].double() for i, e in enumerate(expert)])
    mag = torch.stack([full[i].abs() @ w[e].double().abs() for i, e in enumerate(expert)])
    ref.close(dx[pick.cuda()], want, ref.sum_bound(mag, n), "dx")


@pytest.mark.parametrize("R", [0, 1, 16, 40, 129, 400])
def test_experts_rows_behind_the_last_stay(R):
    g = gen(R)
    E, K, f = 3, 128, 24
    w = normal(g, (E, f, K), BF, 0.1)
    layer = sg.shard_experts(w.cuda(), "all-to-sharded")
    x = normal(g, (R, K), BF)
    off = torch.tensor([0, R // 3, R // 3, R // 2], dtype=torch.int32)
    out = torch.full((1, R, f), 7.0, dtype=BF, device="cuda")
    sg.experts_all_to_sharded(layer, x.cuda(), off.cuda(), out=out)
    assert (out[:, R // 2:] == 7).all()
    ro = sg.shard_experts(w.cuda(), "sharded-to-all")
    out = torch.full((R, f), 7.0, dtype=BF, device="cuda")
    sg.experts_sharded_to_all(ro, x.cuda()[None], off.cuda(), out=out)
    assert (out[R // 2:] == 7).all()
    _, dw = sg.experts_all_to_sharded_backward(layer, x.cuda(), torch.ones((1, R, f), dtype=BF, device="cuda"),
                                               off.cuda())
    assert (dw[1] == 0).all() and torch.isfinite(dw).all()


def test_experts_row_contents_stay_apart():
    """NaN rows of one expert, and behind the last row, reach no other row."""
    g = gen(5)
    E, R, K, f = 3, 90, 200, 40
    w = normal(g, (E, f, K), BF, 0.1)
    x = normal(g, (R, K), BF)
    off = torch.tensor([0, 20, 50, 80], dtype=torch.int32)
    layer = sg.shard_experts(w.cuda(), "all-to-sharded")
    dy = normal(g, (1, R, f), BF)
    clean = sg.experts_all_to_sharded(layer, x.cuda(), off.cuda())[:, :80]
    cx, cw = sg.experts_all_to_sharded_backward(layer, x.cuda(), dy.cuda(), off.cuda())
    x[20:50], x[80:] = math.nan, math.inf
    dy[:, 20:50], dy[:, 80:] = math.inf, math.nan
    got = sg.experts_all_to_sharded(layer, x.cuda(), off.cuda())[:, :80]
    keep = [i for i in range(80) if not 20 <= i < 50]
    assert torch.equal(got[:, keep], clean[:, keep])
    gx, gw = sg.experts_all_to_sharded_backward(layer, x.cuda(), dy.cuda(), off.cuda())
    assert torch.equal(gx[keep], cx[keep])
    assert torch.equal(gw[0], cw[0]) and torch.equal(gw[2], cw[2])


def test_experts_bad_offsets_stay_inside():
    """Offsets beyond the rows or falling end inside the arrays (their rows' results are unspecified)."""
    g = gen(6)
    layer = sg.shard_experts(normal(g, (4, 32, 64), BF).cuda(), "all-to-sharded")
    x = normal(g, (50, 64), BF).cuda()
    for off in ([0, 10, 1 << 30, 1 << 30, 1 << 30], [0, 40, 10, 60, 20], [-5, -1, 7, 7, 50]):
        guard = torch.full((3, 50, 32), 7.0, dtype=BF, device="cuda")
        o = torch.tensor(off, dtype=torch.int32).cuda()
        sg.experts_all_to_sharded(layer, x, o, out=guard[1:2])
        sg.experts_all_to_sharded_backward(layer, x, guard[1:2], o)
        assert (guard[0] == 7).all() and (guard[2] == 7).all()


def test_experts_strided_x():
    g = gen(7)
    layer = sg.shard_experts(normal(g, (2, 48, 96), HF).cuda(), "all-to-sharded")
    off = torch.tensor([0, 11, 30], dtype=torch.int32).cuda()
    for width, at in ((128, 0), (128, 8), (99, 1), (97, 0)):
        x = normal(g, (30, width), HF).cuda()[:, at:at + 96]
        assert torch.equal(sg.experts_all_to_sharded(layer, x, off),
                           sg.experts_all_to_sharded(layer, x.contiguous(), off))
        dy = normal(g, (1, 30, 48), HF).cuda()
        for a, b in zip(sg.experts_all_to_sharded_backward(layer, x, dy, off),
                        sg.experts_all_to_sharded_backward(layer, x.contiguous(), dy, off)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("R", [6, 20, 150])
def test_rows_of_no_token_read_zeros(R):
    """Entries of the row map outside 0 .. T k - 1, and falling offsets, for few rows and for many."""
    g = gen(R)
    E, T, k, K, f = 3, 9, 2, 72, 40
    w = normal(g, (E, f, K), BF, 0.1)
    layer = sg.shard_experts(w.cuda(), "all-to-sharded")
    x, off = normal(g, (T, K), BF).cuda(), offsets_of(g, E, R).cuda()
    rows = torch.randint(0, T * k, (R,), generator=g, dtype=torch.int32)
    out = torch.rand(R, generator=g) < 0.4
    bad = torch.tensor([-1, T * k, 2**31 - 1, -2**31, -k], dtype=torch.int32)
    rows[out] = bad[torch.randint(0, 5, (int(out.sum()),), generator=g)]
    flat = torch.where(out[:, None], 0, x.cpu()[torch.where(out, 0, rows).long() // k])
    y = sg.experts_all_to_sharded(layer, x, off, rows=rows.cuda(), k=k)
    assert torch.equal(y, sg.experts_all_to_sharded(layer, flat.cuda(), off))
    assert (y[:, out.cuda()] == 0).all()
    dy = normal(g, (1, R, f), BF).cuda()
    _, dw = sg.experts_all_to_sharded_backward(layer, x, dy, off, rows=rows.cuda(), k=k, need_dx=False)
    assert torch.equal(dw, sg.experts_all_to_sharded_backward(layer, flat.cuda(), dy, off, need_dx=False)[1])
    guard = torch.full((3, R, f), 7.0, dtype=BF, device="cuda")
    sg.experts_all_to_sharded(layer, x, torch.tensor([0, R, 1, 2 * R], dtype=torch.int32).cuda(), rows=rows.cuda(), k=k,
                              out=guard[1:2])
    assert (guard[0] == 7).all() and (guard[2] == 7).all()


def test_results_past_2_to_the_32():
    """Arrays of more than 2^32 values: the last rows are where they belong."""
    g = gen(11)
    R, K, f = (1 << 17) + 40, 64, 1 << 15
    w = normal(g, (1, f, K), BF, 0.2)
    layer = sg.shard_experts(w.cuda(), "all-to-sharded", segments=2)
    tail = normal(g, (64, K), BF).cuda()
    x = torch.zeros((R, K), dtype=BF, device="cuda")
    x[-64:] = tail
    y = sg.experts_all_to_sharded(layer, x)
    assert torch.equal(y[:, -64:], sg.experts_all_to_sharded(layer, tail)) and not y[0, : R - 64].any()
    slots = torch.tensor([[R - 1, R - 64], [R - 5, -1]], dtype=torch.int32).cuda()
    near = (slots - torch.where(slots >= 0, R - 64, 0)).int()
    assert torch.equal(sg.moe_combine(y[0], slots), sg.moe_combine(y[0, -64:].contiguous(), near))
    assert torch.equal(sg.swiglu(y[0])[-64:], sg.swiglu(y[0, -64:].contiguous()))
    for a, b in zip(sg.quantize_mxfp4(y[0]), sg.quantize_mxfp4(y[0, -64:].contiguous())):
        assert torch.equal(a[-64:], b)
    down = sg.shard_experts(w.transpose(1, 2).contiguous().cuda(), "sharded-to-all")
    dh, _ = sg.experts_sharded_to_all_backward(down, None, x, need_dw=False)
    t, v = tail.cpu().double(), w[0].double()
    for got in (y, dh):
        ref.close(got[0, -64:], t @ v.T, ref.sum_bound(t.abs() @ v.abs().T, K), "last rows")


def test_a_layer_given_up_in_a_capture_outlives_it():
    g = gen(12)
    w, x = normal(g, (1, 64, 128), BF), normal(g, (5, 128), BF).cuda()
    keep, gone = (sg.shard_experts(w.cuda(), "all-to-sharded") for _ in range(2))
    want = sg.experts_all_to_sharded(keep, x)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        del gone
        sg.experts_all_to_sharded(keep, x, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert len(sg._freed) == 1
    keep.free()
    assert not sg._freed


def test_row_map_needs_its_k():
    layer = sg.shard_experts(normal(gen(1), (1, 16, 64), BF).cuda(), "all-to-sharded")
    x, rows = normal(gen(2), (4, 64), BF).cuda(), torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(sg.ShardGemmError, match="k is None"):
        sg.experts_all_to_sharded(layer, x, rows=rows)
    with pytest.raises(sg.ShardGemmError, match="k is None"):
        sg.experts_all_to_sharded_backward(layer, x, torch.zeros((1, 8, 16), dtype=BF, device="cuda"), rows=rows)


def test_experts_refuse_what_does_not_fit():
    """Refusals that need a layer: wrong mode, widths, dtypes, devices, scales and pairs."""
    g = gen(3)
    col = sg.shard_experts(normal(g, (2, 32, 64), BF).cuda(), "all-to-sharded", segments=2)
    row = sg.shard_experts(normal(g, (2, 64, 16), BF).cuda(), "sharded-to-all")
    one = sg.shard_experts(normal(g, (2, 32, 64), BF).cuda(), "all-to-sharded")
    off = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    x = normal(g, (4, 64), BF).cuda()
    bad = lambda code, f, *a, **k: pytest.raises(sg.ShardGemmError, f, *a, **k).value.code == code
    assert bad(sg.ERR_BAD_MODE, sg.experts_all_to_sharded, row, x[:, :16].contiguous(), off)
    assert bad(sg.ERR_INVALID_ARG, sg.experts_all_to_sharded, col, x[:, :32], off)
    assert bad(sg.ERR_INVALID_ARG, sg.experts_all_to_sharded, col, x.float(), off)
    assert bad(sg.ERR_INVALID_ARG, sg.experts_all_to_sharded, col, x.cpu(), off)
    assert bad(sg.ERR_INVALID_ARG, sg.experts_all_to_sharded, col, x)  # no offsets for two experts
    assert bad(sg.ERR_INVALID_ARG, sg.experts_all_to_sharded, col, x, off.long())
    assert bad(sg.ERR_INVALID_ARG, sg.experts_all_to_sharded, col, x.t().contiguous().t(), off)
    assert bad(sg.ERR_INVALID_ARG, sg.experts_all_to_sharded, one, x, off, swiglu=True)
    codes, scales = sg.quantize_mxfp4(x)
    assert bad(sg.ERR_INVALID_ARG, sg.experts_all_to_sharded, col, codes, off, x_scales=scales)
    assert bad(sg.ERR_INVALID_ARG, sg.experts_sharded_to_all, row, x[None], off)
    z = normal(g, (4, 2), F32).cuda()
    r = sg.moe_route(z, 1)
    assert bad(sg.ERR_INVALID_ARG, sg.moe_mlp, one, row, x, r)  # segments = 1
    assert bad(sg.ERR_INVALID_ARG, sg.moe_mlp, row, col, x[:, :16].contiguous(), r)
    assert bad(sg.ERR_NOT_DIVISIBLE, sg.quantize_mxfp4, x[:, :40])
    mx = sg.shard_mxfp4_experts(*sg.quantize_mxfp4(normal(g, (2, 32, 64)).cuda()), "all-to-sharded", segments=2)
    assert bad(sg.ERR_UNSUPPORTED, sg.experts_all_to_sharded_backward, mx, x, torch.zeros((1, 4, 32), dtype=BF,
                                                                                       device="cuda"), off)
    assert bad(sg.ERR_UNSUPPORTED, mx.update, normal(g, (2, 32, 64), BF).cuda())
    col.free()
    assert bad(sg.ERR_INVALID_ARG, sg.experts_all_to_sharded, col, x, off)


def test_experts_update():
    g = gen(8)
    a, b = normal(g, (3, 40, 72), BF), normal(g, (3, 40, 72), BF)
    x = normal(g, (20, 72), BF).cuda()
    off = torch.tensor([0, 5, 9, 20], dtype=torch.int32).cuda()
    for host in (a, a.cuda()):
        layer = sg.shard_experts(host, "all-to-sharded", segments=2, P=4)
        layer.update(b.cuda())
        want = sg.experts_all_to_sharded(sg.shard_experts(b.cuda(), "all-to-sharded", segments=2, P=4), x, off)
        assert torch.equal(sg.experts_all_to_sharded(layer, x, off), want)


# ---- the chain --------------------------------------------------------------

CHAIN = [  # T, E, k, D, F, P, dtype
    (1, 8, 2, 256, 512, 8, BF), (3, 4, 4, 64, 96, 1, HF), (33, 64, 4, 128, 64, 4, BF), (300, 5, 3, 200, 366, 2, BF),
    (1000, 4, 2, 128, 256, 4, HF), (77, 3, 1, 70, 54, 2, BF), (20, 64, 2, 512, 74, 2, BF),
    (2, 4, 2, 2056, 2100, 1, BF),
]


def chain_case(T, E, k, D, F, P, dtype, seed=0):
    g = gen(T + D + seed)
    z = normal(g, (T, E), F32, 1.5)
    z[T - T // 9:] = -math.inf
    x = normal(g, (T, D), dtype)
    gu, dn = normal(g, (E, 2 * F, D), dtype, 1 / math.sqrt(D)), normal(g, (E, D, F), dtype, 1 / math.sqrt(F))
    return z, x, gu, dn


def chain_reference(z, x, gu, dn, k, h_dtype):
    w, e, off, rows, slots = ref.route(z, k, True)
    R, F = int(off[-1]), gu.shape[1] // 2
    T, D = x.shape
    a, m = (torch.zeros((R, 2 * F), dtype=torch.float64) for _ in range(2))
    xg = ref.gathered(x.double(), rows[:R], k)
    ref.product(xg, gu.double(), off, a, m)
    h = ref.silu(a[:, :F]) * a[:, F:]
    bh = ref.swiglu_bound(a[:, :F], a[:, F:], m[:, :F], m[:, F:], D)
    bh = bh + ref.HALF[h_dtype] * (h.abs() + bh) + ref.TINY[h_dtype]  # h is stored in h_dtype
    y, my = (torch.zeros((R, D), dtype=torch.float64) for _ in range(2))
    ref.product(h, dn.double(), off, y, my)
    by, _ = (torch.zeros((R, D), dtype=torch.float64) for _ in range(2))
    ref.product(bh, dn.double().abs(), off, by, _)
    by += ref.sum_bound(my + by, F)
    ok = slots >= 0
    pick = lambda v: torch.where(ok[..., None], v[slots.long().clamp(0)], 0.0) if R else torch.zeros((T, k, D)).double()
    out = (w[..., None] * pick(y)).sum(1)
    bound = (w[..., None] * pick(by)).sum(1) + (z.shape[1] + 80) * 2.0 ** -24 * (w[..., None] * pick(my)).sum(1)
    return out, bound


@pytest.mark.parametrize("case", CHAIN)
def test_moe_mlp(case):
    T, E, k, D, F, P, dtype = case
    z, x, gu, dn = chain_case(*case)
    lg = sg.shard_experts(gu.cuda(), "all-to-sharded", segments=2, P=P)
    ld = sg.shard_experts(dn.cuda(), "sharded-to-all", P=P)
    r = sg.moe_route(z.cuda(), k)
    out = sg.moe_mlp(lg, ld, x.cuda(), r)
    want, bound = chain_reference(z, x, gu, dn, k, dtype)
    ref.close(out, want, bound, "moe_mlp")
    assert (out[T - T // 9:] == 0).all() if T // 9 else True
    # bitwise the three calls
    h = sg.experts_all_to_sharded(lg, x.cuda(), r.offsets, r.rows, k, swiglu=True)
    y = sg.experts_sharded_to_all(ld, h, r.offsets, out_dtype=F32)
    assert torch.equal(sg.moe_combine(y, r.slots, r.weights, out_dtype=dtype), out)


def test_training_step_gradients():
    """Router, layers, SwiGLU and weighted sum forward and backward, against autograd in 64 bits."""
    T, E, k, D, F, P = 60, 4, 2, 64, 48, 2
    z, x, gu, dn = chain_case(T, E, k, D, F, P, BF)
    dout = normal(gen(9), (T, D), BF)
    lg = sg.shard_experts(gu.cuda(), "all-to-sharded", segments=2, P=P)
    ld = sg.shard_experts(dn.cuda(), "sharded-to-all", P=P)
    r = sg.moe_route(z.cuda(), k)
    pre = sg.experts_all_to_sharded(lg, x.cuda(), r.offsets, r.rows, k)
    h = sg.swiglu(pre)
    y = sg.experts_sharded_to_all(ld, h, r.offsets)
    dy, dw = sg.moe_combine_backward(dout.cuda(), y, r.slots, r.weights)
    dz = sg.moe_route_backward(z.cuda(), r, dw)
    dh, ddn = sg.experts_sharded_to_all_backward(ld, h, dy, r.offsets)
    dx, dgu = sg.experts_all_to_sharded_backward(lg, x.cuda(), sg.swiglu_backward(pre, dh), r.offsets, r.rows, k)
    dx = sg.moe_combine(dx, r.slots, out_dtype=F32)
    leaves = [v.double().requires_grad_(True) for v in (z, x, gu, dn)]
    zz, xx, gg, dd = leaves
    _, e, *_ = ref.route(z, k, True)
    total = 0
    for t in range(T):
        ids = [int(i) for i in e[t] if i >= 0]
        if not ids:
            continue
        w = torch.softmax(zz[t, ids], 0)
        for j, i in enumerate(ids):
            a = gg[i] @ xx[t]
            total = total + w[j] * (dd[i] @ (ref.silu(a[:F]) * a[F:]) * dout[t].double()).sum()
    gz, gx, ggu, gdn = torch.autograd.grad(total, leaves)
    order = ref.shard_rows(2 * F, 2, P)
    ggu = torch.stack([torch.stack([ggu[i][o] for o in order]) for i in range(E)])
    gdn = torch.stack([torch.stack(list(gdn[i].split(F // P, 1))) for i in range(E)])
    # five bf16 roundings stand in the way at most, half a step of 2^-8 each, on
    # intermediate values whose errors add up like their rms: 5 * 2^-8 in norm
    for name, got, want in (("dz", dz, gz), ("dx", dx, gx), ("dgate_up", dgu, ggu), ("ddown", ddn, gdn)):
        rel = ((got.double().cpu() - want).norm() / want.norm()).item()
        assert rel <= 5 * 2.0 ** -8, (name, rel)


@pytest.mark.parametrize("T", [4, 400])
def test_capture_and_replay(T):
    E, k, D, F, P = 6, 2, 128, 96, 2
    z, x, gu, dn = chain_case(T, E, k, D, F, P, BF)
    lg = sg.shard_experts(gu.cuda(), "all-to-sharded", segments=2, P=P)
    ld = sg.shard_experts(dn.cuda(), "sharded-to-all", P=P)
    zs, xs, ds = z.cuda(), x.cuda(), normal(gen(4), (T, D), BF).cuda()

    def step(z, x, d):
        r = sg.moe_route(z, k)
        out = sg.moe_mlp(lg, ld, x, r)
        pre = sg.experts_all_to_sharded(lg, x, r.offsets, r.rows, k, out=torch.zeros((P, T * k, 2 * F // P), dtype=BF,
                                                                                    device="cuda"))
        h = sg.swiglu(pre)
        y = sg.experts_sharded_to_all(ld, h, r.offsets, out=torch.zeros((T * k, D), dtype=BF, device="cuda"))
        dy, dw = sg.moe_combine_backward(d, y, r.slots, r.weights)
        dz = sg.moe_route_backward(z, r, dw)
        _, ddn = sg.experts_sharded_to_all_backward(ld, h, dy, r.offsets, need_dx=False)
        return out, dz, ddn

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(zs, xs, ds)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(zs, xs, ds)
    for seed in range(4):
        z2, x2, *_ = chain_case(T, E, k, D, F, P, BF, seed)
        zs.copy_(z2), xs.copy_(x2)
        want = step(z2.cuda(), x2.cuda(), ds)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_other_stream_and_repeats():
    T, E, k, D, F, P = 200, 6, 2, 128, 96, 2
    z, x, gu, dn = chain_case(T, E, k, D, F, P, BF)
    lg = sg.shard_experts(gu.cuda(), "all-to-sharded", segments=2, P=P)
    ld = sg.shard_experts(dn.cuda(), "sharded-to-all", P=P)
    r = sg.moe_route(z.cuda(), k)
    want = sg.moe_mlp(lg, ld, x.cuda(), r)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                outs.append(sg.moe_mlp(lg, ld, x.cuda(), sg.moe_route(z.cuda(), k)))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
