"""Low-rank adapters where calls meet: captures of other threads, the widest tiles."""
import math
import threading

import pytest
import torch

import adapters_ref as aref
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


@pytest.mark.parametrize("i,o", [(72, 104), (96, 80)])  # stored row-major; in fragments that are not the tiles'
def test_first_adapted_call_while_another_thread_captures(i, o):
    g = gen(i)
    T, n, r = 40, 2, 8
    w = normal(g, (o, i), BF, 0.1).cuda()
    keep, first, same = (sg.shard_linear(w, "all-to-sharded", P=2) for _ in range(3))
    ad = sg.Adapters(normal(g, (n, r, i), BF, 0.1).cuda(), normal(g, (n, o, r), BF, 0.1).cuda())
    x, dy = normal(g, (T, i), BF).cuda(), normal(g, (2, T, o // 2), BF).cuda()
    plan = sg.adapter_plan(torch.randint(-1, n, (T,), generator=g, dtype=torch.int32).cuda(), n)

    def both(layer):
        return (sg.adapted_all_to_sharded(layer, x, ad, plan),
                *sg.adapted_all_to_sharded_backward(layer, x, dy, ad, plan))

    want, plain = both(same), sg.all_to_sharded(keep, x)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(plain)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hold = torch.empty(8, device="cuda")  # keeps 2 MiB of torch's, whose own allocation would end the capture
    torch.cuda.synchronize()
    capturing, errors, got = threading.Event(), [], []

    def call():
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(side):  # (a wait of torch's own would end it, too)
                if capturing.wait(60):
                    got.extend(both(first))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    other = threading.Thread(target=call)
    other.start()
    with torch.cuda.graph(graph):
        capturing.set()
        other.join()
        sg.all_to_sharded(keep, x, out=out)
    side.synchronize()
    assert not errors, errors
    assert len(got) == 4 and all(torch.equal(a, b) for a, b in zip(got, want))
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plain)
    del hold


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("mode,i,o", [(0, 64, 96), (0, 80, 64), (1, 64, 96), (1, 96, 64)])
def test_first_backward_call_captured(mode, i, o, dtype):
    """A backward call captured before the layer has its transposed copy: the vector units' sums."""
    g = gen(i + o + mode)
    B, P = 20, 2
    w = normal(g, (o, i), dtype, 1 / math.sqrt(o))
    layer = sg.shard_linear(w.cuda(), mode, P=P)
    dys = [normal(g, (P, B, o // P) if mode == 0 else (B, o), dtype).cuda() for _ in range(3)]
    dy, graph = dys[0].clone(), torch.cuda.CUDAGraph()
    back = sg.all_to_sharded_backward if mode == 0 else sg.sharded_to_all_backward
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, _ = back(layer, None, dy, need_dw=False, dx_dtype=F32)
    for k in (1, 2, 0):
        dy.copy_(dys[k])
        graph.replay()
        eager, _ = back(layer, None, dys[k], need_dw=False, dx_dtype=F32)
        torch.cuda.synchronize()
        full = dys[k].double().cpu()
        if mode == 0:
            full = full.transpose(0, 1).flatten(1)
        want, mag = full @ w.double(), full.abs() @ w.double().abs()
        if mode == 1:
            want, mag = (v.view(B, P, i // P).transpose(0, 1) for v in (want, mag))
        for got, name in ((out, "captured"), (eager, "eager")):
            ref.close(got, want, ref.sum_bound(mag, o), name)


# ---- layers given up ----------------------------------------------------------

def test_a_layer_given_up_in_a_capture_outlives_it():
    g = gen(12)
    w, x = normal(g, (64, 128), BF).cuda(), normal(g, (5, 128), BF).cuda()
    keep, gone = (sg.shard_linear(w, "all-to-sharded") for _ in range(2))
    want = sg.all_to_sharded(keep, x)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        del gone
        sg.all_to_sharded(keep, x, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert len(sg._freed_layers) == 1
    again = sg.shard_linear(w, "all-to-sharded")
    assert not sg._freed_layers and torch.equal(sg.all_to_sharded(again, x), want)


def test_a_layer_given_up_while_another_thread_captures():
    g = gen(15)
    w, x = normal(g, (80, 96), BF).cuda(), normal(g, (20, 96), BF).cuda()
    keep, gone = (sg.shard_linear(w, "all-to-sharded") for _ in range(2))
    codes, scales = sg.quantize_mxfp8(w)
    mx8 = sg.shard_mxfp8_linear(codes, scales, "all-to-sharded")
    ad = sg.Adapters(normal(g, (1, 8, 96), BF).cuda(), normal(g, (1, 80, 8), BF).cuda())
    plan = sg.adapter_plan(torch.zeros(20, dtype=torch.int32, device="cuda"), 1)
    sg.adapted_all_to_sharded(gone, x, ad, plan)  # (it then holds a copy, too)
    want = sg.all_to_sharded(keep, x)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    torch.cuda.synchronize()
    capturing, errors = threading.Event(), []

    def drop():
        try:
            torch.cuda.set_device(0)
            if capturing.wait(60):
                gone.free()
                mx8.free()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    other = threading.Thread(target=drop)
    other.start()
    with torch.cuda.graph(graph):
        capturing.set()
        other.join()
        sg.all_to_sharded(keep, x, out=out)
    assert not errors and not sg._freed_layers
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_giving_up_a_layer_waits_for_the_device():
    g = gen(16)
    layers = [sg.shard_linear(normal(g, (1024, 1024), BF).cuda(), "all-to-sharded") for _ in range(2)]
    x = normal(g, (4096, 1024), BF).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty((1, 4096, 1024), dtype=BF, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(1000):
            sg.all_to_sharded(layers[0], x, out=out)
        done = torch.cuda.Event()
        done.record()
    busy = not done.query()
    layers[1].free()
    assert busy and done.query()
    layers[0].free()


# ---- the widest tiles ---------------------------------------------------------
# 4100 tokens beside outputs (backward: inputs) of some 4400 columns take tiles of 256 x 256,
# those behind the last time round 256 compute units their quarters; the last tile has four
# rows.  T, in, out, mode, P, S, adapters, rank, type
FORWARD = [(4100, 72, 4416, 0, 2, 3, 5, 40, BF), (4100, 64, 4413, 0, 3, 1, 200, 20, HF), (4100, 128, 4400, 1, 2, 1, 3, 12, BF),
           (4100, 64, 4400, 1, 1, 1, 70, 100, HF), (5300, 40, 4608, 0, 1, 2, 1, 8, HF)]
SWIGLU = [(4100, 72, 4400, 0, 2, 2, 3, 24, BF), (4100, 64, 4404, 0, 1, 2, 150, 100, HF), (4100, 64, 4416, 0, 3, 2, 900, 16, BF)]
BACKWARD = [(4100, 4408, 96, 0, 2, 1, 3, 17, BF), (4100, 4400, 64, 0, 1, 2, 150, 40, HF), (4100, 4416, 64, 1, 2, 1, 4, 48, HF),
            (4100, 4480, 72, 1, 2, 2, 90, 16, BF), (4100, 4401, 64, 0, 1, 1, 2, 9, BF)]


def wide_case(T, i, o, mode, P, S, n, r, dtype):
    g = gen(T + i + o + r)
    w = normal(g, (o, i), dtype, 1 / math.sqrt(i))
    ad = sg.Adapters(normal(g, (n, r, i), dtype, 1 / math.sqrt(i)).cuda(), normal(g, (n, o, r), dtype, 1 / math.sqrt(r)).cuda(),
                     (torch.rand(n, generator=g) + 0.5).cuda())
    which = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32)
    x, dy = normal(g, (T, i), dtype), normal(g, (T, o), dtype)
    # tokens at the borders of tiles and quarters in the plan's order, and others
    _, rows = aref.plan(which, n)
    at = [m for k in range(0, T, 128) for m in (k - 1, k, k + 15, k + 16) if 0 <= m < T] + [T - 1]
    pick = torch.tensor(sorted({rows[m] for m in at} | set(torch.randint(0, T, (60,), generator=g).tolist())))
    order = ref.shard_rows(o if mode == 0 else i, S, P)
    shard = lambda v: torch.stack([v[:, q] for q in order])  # noqa: E731
    return w, ad, which, x, dy, pick, shard, sg.adapter_plan(which.cuda(), n)


def adapted_rows(w, ad, which, x, pick, r, dtype):
    """x W^T and the adapters' part for the picked tokens, and the sum's bound."""
    v = x[pick].double()
    d, e = aref.delta(v, which[pick], ad.A.cpu(), ad.B.cpu(), ad.scale.cpu(), dtype)
    base, eb = v @ w.double().T, ref.sum_bound(v.abs() @ w.double().abs().T, v.shape[1])
    return base + d, e + eb + (2 * r + 4) * 2.0 ** -24 * (base.abs() + d.abs() + e)


@pytest.mark.parametrize("case", FORWARD)
def test_wide_tiles_forward(case):
    T, i, o, mode, P, S, n, r, dtype = case
    w, ad, which, x, _, pick, shard, plan = wide_case(*case)
    layer = sg.shard_linear(w.cuda(), mode, segments=S, P=P)
    want, bound = adapted_rows(w, ad, which, x, pick, r, dtype)
    if mode == 0:
        want, bound = shard(want), shard(bound)
    for out in (dtype, F32):
        if mode == 0:
            y = sg.adapted_all_to_sharded(layer, x.cuda(), ad, plan, out_dtype=out)
            z = sg.adapted_all_to_sharded(layer, x.cuda(), ad, plan, out_dtype=out, gather=True)
            assert torch.equal(z.view(T, P, -1).transpose(0, 1), y)
            ref.close(y[:, pick.cuda()], want, bound, f"y {out}")
        else:
            y = sg.adapted_sharded_to_all(layer, shard(x).cuda(), ad, plan, out_dtype=out)
            ref.close(y[pick.cuda()], want, bound, f"y {out}")
        assert torch.isfinite(y).all()


@pytest.mark.parametrize("case", SWIGLU)
def test_wide_tiles_swiglu(case):
    T, i, o, mode, P, S, n, r, dtype = case
    w, ad, which, x, _, pick, shard, plan = wide_case(*case)
    layer = sg.shard_linear(w.cuda(), mode, segments=S, P=P)
    z, e = adapted_rows(w, ad, which, x, pick, r, dtype)
    (a, b), (ea, eb) = shard(z).chunk(2, -1), shard(e).chunk(2, -1)
    want = ref.silu(a) * b
    bound = 1.1 * (b.abs() + eb) * ea + (ref.silu(a).abs() + 1.1 * ea) * eb + 16 * 2.0 ** -24 * want.abs()
    for out in (dtype, F32):
        h = sg.adapted_all_to_sharded(layer, x.cuda(), ad, plan, swiglu=True, out_dtype=out)
        ref.close(h[:, pick.cuda()], want, bound, f"h {out}")
        assert torch.isfinite(h).all()


@pytest.mark.parametrize("case", BACKWARD)
def test_wide_tiles_backward(case):
    T, i, o, mode, P, S, n, r, dtype = case
    w, ad, which, x, dy, pick, shard, plan = wide_case(*case)
    layer = sg.shard_linear(w.cuda(), mode, segments=S, P=P)
    v = dy[pick].double()
    (dx, ex), _, _ = aref.gradients(x[pick].double(), v, which[pick], ad.A.cpu(), ad.B.cpu(), ad.scale.cpu(), dtype)
    base, eb = v @ w.double(), ref.sum_bound(v.abs() @ w.double().abs(), o)
    want, bound = base + dx, ex + eb + (2 * r + 4) * 2.0 ** -24 * (base.abs() + dx.abs() + ex)
    for out in (dtype, F32):
        if mode == 0:
            got, _, _ = sg.adapted_all_to_sharded_backward(layer, None, shard(dy).cuda(), ad, plan, need_d=False, dx_dtype=out)
            ref.close(got[pick.cuda()], want, bound, f"dx {out}")
        else:
            got, _, _ = sg.adapted_sharded_to_all_backward(layer, None, dy.cuda(), ad, plan, need_d=False, dx_dtype=out)
            ref.close(got[:, pick.cuda()], shard(want), shard(bound), f"dx {out}")
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("mode,i,o,P,S,swiglu", [(0, 576, 4416, 2, 1, False), (0, 448, 4416, 1, 2, True), (1, 640, 4400, 2, 1, False)])
def test_wide_tiles_of_odd_4_bit_layers(mode, i, o, P, S, swiglu, dtype):
    """Weights in two halves: the inputs twice through the tiles."""
    T, n, r = 4100, 6, 24
    _, ad, which, x, _, pick, shard, plan = wide_case(T, i, o, mode, P, S, n, r, dtype)
    g = gen(i + o)
    words = torch.randint(-2 ** 31, 2 ** 31, (o, i // 8), generator=g, dtype=torch.int64).to(torch.int32)
    sc = ((0.5 + torch.rand((o, i // 64), generator=g)) / (8 * math.sqrt(i))).half()
    qb = (-7.5 * sc).half()
    layer = sg.shard_quantized_linear(words.cuda(), sc.view(torch.int16).cuda(), qb.view(torch.int16).cuda(), i, mode,
                                      segments=S, P=P, act_dtype=dtype)
    q = ((words.long() & 0xffffffff)[..., None] >> (4 * torch.arange(8)) & 15).flatten(1).double()
    sq, b = sc.double().repeat_interleave(64, 1) * q, qb.double().repeat_interleave(64, 1)
    z, e = adapted_rows(sq + b, ad, which, x, pick, r, dtype)
    # the weights in two halves, and twice as many products
    e = e + (aref.SPLIT[dtype] + (i + 4) * 2.0 ** -24) * (x[pick].double().abs() @ (sq.abs() + b.abs()).T)
    if swiglu:
        (a, c), (ea, ec) = shard(z).chunk(2, -1), shard(e).chunk(2, -1)
        z = ref.silu(a) * c
        e = 1.1 * (c.abs() + ec) * ea + (ref.silu(a).abs() + 1.1 * ea) * ec + 16 * 2.0 ** -24 * z.abs()
    elif mode == 0:
        z, e = shard(z), shard(e)
    for out in (dtype, F32):
        if mode == 0:
            y = sg.adapted_all_to_sharded(layer, x.cuda(), ad, plan, swiglu=swiglu, out_dtype=out)
            ref.close(y[:, pick.cuda()], z, e, f"y {out}")
        else:
            y = sg.adapted_sharded_to_all(layer, shard(x).cuda(), ad, plan, out_dtype=out)
            ref.close(y[pick.cuda()], z, e, f"y {out}")
        assert torch.isfinite(y).all()


# ---- arguments of any alignment, gathered SwiGLU ------------------------------

def shifted(t, by=1):
    """The same values, packed, `by` elements behind a 16-byte border."""
    flat = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
    v = flat[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,i,o,mode,P,S,n,r", [(5, 64, 96, 0, 2, 1, 3, 16), (40, 256, 192, 0, 2, 3, 3, 8), (40, 256, 96, 1, 2, 1, 2, 24),
                                                (300, 64, 4096, 0, 2, 2, 3, 16), (300, 4096, 64, 0, 1, 1, 70, 8),
                                                (300, 4096, 64, 1, 2, 1, 3, 16), (300, 64, 4096, 1, 1, 1, 3, 40)])
def test_arguments_of_any_alignment(T, i, o, mode, P, S, n, r, dtype):
    w, ad, which, x, dy, _, shard, plan = wide_case(T, i, o, mode, P, S, n, r, dtype)
    layer = sg.shard_linear(w.cuda(), mode, segments=S, P=P)
    every = torch.arange(T)
    want, bound = adapted_rows(w, ad, which, x, every, r, dtype)
    (dx, ex), (dA, eA), (dB, eB) = aref.gradients(x.double(), dy.double(), which, ad.A.cpu(), ad.B.cpu(), ad.scale.cpu(), dtype)
    base, eb = dy.double() @ w.double(), ref.sum_bound(dy.double().abs() @ w.double().abs(), o)
    dx, ex = base + dx, ex + eb + (2 * r + 4) * 2.0 ** -24 * (base.abs() + dx.abs() + ex)
    if mode == 0:
        want, bound, xs, dys = shard(want), shard(bound), x, shard(dy)
        call, back = sg.adapted_all_to_sharded, sg.adapted_all_to_sharded_backward
    else:
        dx, ex, xs, dys = shard(dx), shard(ex), shard(x), dy
        call, back = sg.adapted_sharded_to_all, sg.adapted_sharded_to_all_backward
    odd = sg.Adapters(shifted(ad.A), shifted(ad.B, 3), shifted(ad.scale))
    for out in (dtype, F32):
        y = shifted(torch.zeros(want.shape, dtype=out, device="cuda"))
        ref.close(call(layer, shifted(xs), odd, plan, out=y), want, bound, f"y {out}")
        assert y.data_ptr() % 16
        gx, gA, gB = back(layer, shifted(xs, 5), shifted(dys), odd, plan, dx_dtype=out, d_dtype=out)
        ref.close(gx, dx, ex, f"dx {out}")
        ref.close(gA, dA, eA, f"dA {out}")
        ref.close(gB, dB, eB, f"dB {out}")


@pytest.mark.parametrize("kind", ["dense", "bias", "q4"])
@pytest.mark.parametrize("T,i,o,P", [(3, 64, 96, 2), (20, 128, 256, 4), (300, 64, 4128, 3)])
def test_gathered_swiglu(T, i, o, P, kind):
    """The gathered layout holds what the sharded one does."""
    g = gen(T + o)
    if kind == "q4":
        words = torch.randint(-2 ** 31, 2 ** 31, (o, i // 8), generator=g, dtype=torch.int64).to(torch.int32)
        sc = (torch.rand((o, i // 64), generator=g) * 0.01).half()
        layer = sg.shard_quantized_linear(words.cuda(), sc.view(torch.int16).cuda(), (-7 * sc).half().view(torch.int16).cuda(), i,
                                          0, segments=2, P=P, act_dtype=BF)
    else:
        layer = sg.shard_linear(normal(g, (o, i), BF, 0.1).cuda(), 0, segments=2, P=P,
                                bias=normal(g, (o,), BF).cuda() if kind == "bias" else None)
    ad = sg.Adapters(normal(g, (3, 12, i), BF, 0.1).cuda(), normal(g, (3, o, 12), BF, 0.1).cuda())
    plan = sg.adapter_plan(torch.randint(-1, 3, (T,), generator=g, dtype=torch.int32).cuda(), 3)
    x = normal(g, (T, i), BF).cuda()
    for out in (BF, F32):
        h = sg.adapted_all_to_sharded(layer, x, ad, plan, swiglu=True, out_dtype=out)
        z = sg.adapted_all_to_sharded(layer, x, ad, plan, swiglu=True, gather=True, out_dtype=out)
        assert torch.equal(z.view(T, P, -1).transpose(0, 1), h) and h.any() and torch.isfinite(h).all()


@pytest.mark.parametrize("T,i,o,mode,P,S,n,r,dtype", [(5, 96, 64, 0, 2, 1, 2, 8, BF), (40, 72, 104, 0, 2, 2, 3, 12, HF), (300, 4100, 96, 0, 2, 1, 3, 40, BF),
                                                      (40, 96, 64, 1, 1, 1, 2, 8, HF), (300, 2900, 48, 1, 2, 1, 3, 16, BF), (4100, 4408, 96, 0, 1, 3, 5, 8, HF)])
def test_gradients_beside_a_bias(T, i, o, mode, P, S, n, r, dtype):
    w, ad, which, x, dy, pick, shard, plan = wide_case(T, i, o, mode, P, S, n, r, dtype)
    layer = sg.shard_linear(w.cuda(), mode, segments=S, P=P, bias=normal(gen(1), (o,), dtype, 100.0).cuda())
    v = dy[pick].double()
    (dx, ex), _, _ = aref.gradients(x[pick].double(), v, which[pick], ad.A.cpu(), ad.B.cpu(), ad.scale.cpu(), dtype)
    base, eb = v @ w.double(), ref.sum_bound(v.abs() @ w.double().abs(), o)
    want, bound = base + dx, ex + eb + (2 * r + 4) * 2.0 ** -24 * (base.abs() + dx.abs() + ex)
    for out in (dtype, F32):
        if mode == 0:
            got, _, _ = sg.adapted_all_to_sharded_backward(layer, None, shard(dy).cuda(), ad, plan, need_d=False, dx_dtype=out)
            ref.close(got[pick.cuda()], want, bound, f"dx {out}")
        else:
            got, _, _ = sg.adapted_sharded_to_all_backward(layer, None, dy.cuda(), ad, plan, need_d=False, dx_dtype=out)
            ref.close(got[:, pick.cuda()], shard(want), shard(bound), f"dx {out}")
