"""The mixture-of-experts and MXFP4 operators where values, sizes and callers are
unusual: gates far from zero, no tokens, rows of any alignment, infinities,
pairs of different weights, layers given up by several threads, and activation
slices that fill their 32-bit offsets.

Tolerances as in test_gpu_moe.py."""
import math
import threading

import pytest
import torch

import moe_ref as ref
import sharded_gemm_alltosharded_amd as sg
from test_gpu_moe import BF, F32, HF, gen, normal, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    sg.lib()


# gates c * a for the columns' c and the rows' a, one product each, so exact
FAR_COLUMNS = [1.0, -1.0, 0.0, 64.0, -64.0, 0.5, -0.5]
FAR_ROWS = [1.0, 16.0, 69.0, 70.0, 87.0, 88.0, 89.0, 96.0, 100.0, 104.0, 126.0, 128.0, 200.0]


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "mxfp4", "mxfp4 x mxfp4"])
def test_swiglu_epilogue_far_gates(kind, tiles):
    """silu of gates down to where e^-z is no fp32 number, in the streaming kernel and in the tiles.

    Where e^-z is beyond 2^126 its reciprocal is below the smallest normal fp32
    number and may be 0: |silu(z)| = |z| / (1 + e^-z) < 90 * 2^-126 for those z
    (z < -87.3, and |z| e^z falls from there on) may be lost, times |up|."""
    dtype = HF if kind == "fp16" else BF
    a = FAR_ROWS + ([] if kind == "fp16" else [2.0 ** 100])
    P, K, f, up = 2, 96, len(FAR_COLUMNS) * 2, 1.5
    E, R = (1, len(a) * 12) if tiles else (4, len(a))
    x = torch.zeros((R, K), dtype=dtype)
    x[:, 0] = torch.tensor(a).repeat(R // len(a)).to(dtype)
    x[:, 40] = up  # (another scale block)
    w = torch.zeros((E, 2, f, K))
    w[:, 0, :, 0] = torch.tensor(FAR_COLUMNS * 2)
    w[:, 1, :, 40] = 1.0
    w = w.view(E, 2 * f, K)
    off = offsets_of(gen(1), E, R)
    kw, xv, call = {}, x, x.cuda()
    if kind.startswith("mxfp4"):
        codes, scales = ref.encode(w)
        assert torch.equal(ref.decode(codes, scales), w.double())
        layer = sg.shard_mxfp4_experts(codes.cuda(), scales.cuda(), "all-to-sharded", segments=2, P=P)
        if kind != "mxfp4":
            call, xs = sg.quantize_mxfp4(x.cuda())
            kw, xv = {"x_scales": xs}, ref.decode(call.cpu(), xs.cpu())
    else:
        layer = sg.shard_experts(w.to(dtype).cuda(), "all-to-sharded", segments=2, P=P)
    gate = xv[:, 0].double()[:, None] * torch.tensor(FAR_COLUMNS * 2, dtype=torch.float64)
    u = xv[:, 40].double()[:, None].expand_as(gate)
    zero = torch.zeros_like(gate)
    bound = ref.swiglu_bound(gate, u, zero, zero, K)
    # (e^-z of a rounded exponent: log2 e in fp32 is 1.93e-8 off, an e of relative error
    # 1.93e-8 ln 2 |z| < 1.2e-6 where it is finite, 20 half steps; a few more of the
    # hardware's exponential and reciprocal)
    bound = bound + 32 * 2.0 ** -24 * (ref.silu(gate) * u).abs() + 90 * 2.0 ** -126 * u.abs()
    want, bound = (v.view(R, P, f // P).transpose(0, 1) for v in (ref.silu(gate) * u, bound))
    for out_dtype in (dtype, F32):
        got = sg.experts_all_to_sharded(layer, call, off.cuda(), swiglu=True, out_dtype=out_dtype, **kw)
        ref.close(got, want, bound, f"{kind} {out_dtype}")


@pytest.mark.parametrize("T", [3, 200])
def test_moe_mlp_of_far_gates(T):
    """A token one of whose gates is -100 keeps its output."""
    g = gen(T)
    D, F = 64, 32
    x, gu, dn = normal(g, (T, D), BF), normal(g, (1, 2 * F, D), BF, 0.1), normal(g, (1, D, F), BF, 0.1)
    x[:, 0] = 1.0
    gu[0, 5, :] = 0
    gu[0, 5, 0] = -100.0
    route = sg.moe_route(torch.zeros((T, 1), device="cuda"), 1)
    lg = sg.shard_experts(gu.cuda(), "all-to-sharded", segments=2)
    out = sg.moe_mlp(lg, sg.shard_experts(dn.cuda(), "sharded-to-all"), x.cuda(), route)
    dn[0, :, 5] = 0  # silu(-100) is below 2^-137: no output of that column's counts
    assert torch.equal(out, sg.moe_mlp(lg, sg.shard_experts(dn.cuda(), "sharded-to-all"), x.cuda(), route))


@pytest.mark.parametrize("E", [5, 256, 257, 300, 1024])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_of_no_tokens(E, normalize):
    z = torch.empty((0, E), device="cuda")
    r = sg.moe_route(z, 2, normalize)
    assert r.offsets.tolist() == [0] * (E + 1)
    assert r.weights.shape == r.experts.shape == r.slots.shape == (0, 2) and r.rows.shape == (0,)
    assert sg.moe_route_backward(z, r, torch.empty((0, 2), device="cuda"), normalize).shape == (0, E)


# E, R, in, out, segments: as many output blocks as take one, two, four, eight
# and sixteen waves for a block's inputs, and tiles
@pytest.mark.parametrize("E,R,K,n,S", [(4, 6, 2048, 28672, 1), (2, 5, 2048, 28672, 1), (1, 3, 2048, 28672, 1),
                                       (1, 2, 2048, 14336, 1), (4, 7, 4096, 28672, 2), (1, 2, 8192, 4096, 1),
                                       (1, 3, 8192, 2048, 2), (1, 40, 2048, 4096, 2)])
def test_mxfp4_results_do_not_depend_on_alignment(E, R, K, n, S):
    g = torch.Generator("cuda").manual_seed(n + E)
    codes = torch.randint(0, 256, (E, n, K // 2), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    scales = torch.randint(118, 123, (E, n, K // 32), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    layer = sg.shard_mxfp4_experts(codes, scales, "all-to-sharded", segments=S)
    off = offsets_of(gen(E), E, R, empty=False).cuda()
    for width, at in ((K + 3, 1), (K + 8, 8), (K + 4, 4)):
        x = torch.randn((R, width), generator=g, device="cuda").to(BF)[:, at:at + K]
        for swiglu in ([False, True] if S == 2 else [False]):
            got = sg.experts_all_to_sharded(layer, x, off, swiglu=swiglu, out_dtype=F32)
            assert torch.equal(got, sg.experts_all_to_sharded(layer, x.contiguous(), off, swiglu=swiglu, out_dtype=F32))


@pytest.mark.parametrize("T", [3, 200])
def test_moe_mlp_of_infinities(T):
    """Infinities go through the chain as through its three calls, where the hidden
    width is no multiple of the stored rows' eight columns."""
    g = gen(T)
    D, F, P = 64, 26, 2
    x = normal(g, (T, D), BF).abs()
    x[0, 3] = math.inf
    w = lambda *s: normal(g, s, BF, 0.1).abs() + 0.01
    lg = sg.shard_experts(w(1, 2 * F, D).cuda(), "all-to-sharded", segments=2, P=P)
    ld = sg.shard_experts(w(1, D, F).cuda(), "sharded-to-all", P=P)
    r = sg.moe_route(torch.zeros((T, 1), device="cuda"), 1)
    h = sg.experts_all_to_sharded(lg, x.cuda(), r.offsets, r.rows, 1, swiglu=True)
    want = sg.moe_combine(sg.experts_sharded_to_all(ld, h, r.offsets, out_dtype=F32), r.slots, r.weights, out_dtype=BF)
    got = sg.moe_mlp(lg, ld, x.cuda(), r)
    assert torch.isinf(want[0]).all() and torch.isfinite(want[1:]).all()
    assert torch.equal(got, want)


@pytest.mark.parametrize("T,E,k,D,F,P", [(1, 4, 2, 64, 64, 2), (40, 6, 3, 96, 192, 2), (300, 2, 1, 96, 54, 2)])
def test_moe_mlp_of_one_mxfp4_layer(T, E, k, D, F, P):
    """MXFP4 gate|up with bf16 down, and the reverse: bitwise the three calls."""
    g = gen(T)
    x, r = normal(g, (T, D), BF).cuda(), sg.moe_route(normal(g, (T, E)).cuda(), k)
    gu, dn = normal(g, (E, 2 * F, D), BF, 0.1).cuda(), normal(g, (E, D, F), BF, 0.1).cuda()
    pairs = [(sg.shard_mxfp4_experts(*sg.quantize_mxfp4(gu), "all-to-sharded", segments=2, P=P),
              sg.shard_experts(dn, "sharded-to-all", P=P))]
    if F // P % 32 == 0:
        pairs.append((sg.shard_experts(gu, "all-to-sharded", segments=2, P=P),
                      sg.shard_mxfp4_experts(*sg.quantize_mxfp4(dn), "sharded-to-all", P=P)))
    for lg, ld in pairs:
        h = sg.experts_all_to_sharded(lg, x, r.offsets, r.rows, k, swiglu=True)
        y = sg.experts_sharded_to_all(ld, h, r.offsets, out_dtype=F32)
        assert torch.equal(sg.moe_mlp(lg, ld, x, r), sg.moe_combine(y, r.slots, r.weights, out_dtype=BF))


def test_layers_given_up_by_several_threads():
    w = normal(gen(14), (1, 32, 64), BF).cuda()
    layers = [sg.shard_experts(w, "all-to-sharded") for _ in range(48)]
    errors = []

    def drop(some):
        try:
            torch.cuda.set_device(0)
            for layer in some:
                layer.free()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=drop, args=(layers[i::8],)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and not sg._freed


def test_a_layer_given_up_while_another_thread_captures():
    g = gen(15)
    w, x = normal(g, (1, 64, 128), BF).cuda(), normal(g, (5, 128), BF).cuda()
    keep, gone = (sg.shard_experts(w, "all-to-sharded") for _ in range(2))
    mx = sg.shard_mxfp4_experts(*sg.quantize_mxfp4(w), "all-to-sharded")
    want = sg.experts_all_to_sharded(keep, x)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    capturing, errors = threading.Event(), []

    def drop():
        try:
            torch.cuda.set_device(0)
            if capturing.wait(60):
                gone.free()
                mx.free()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    other = threading.Thread(target=drop)
    other.start()
    with torch.cuda.graph(graph):
        capturing.set()
        other.join()
        sg.experts_all_to_sharded(keep, x, out=out)
    assert not errors and not sg._freed
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_giving_up_a_layer_waits_for_the_device():
    g = gen(16)
    layers = [sg.shard_experts(normal(g, (2, 512, 1024), BF).cuda(), "all-to-sharded") for _ in range(2)]
    x = normal(g, (4096, 1024), BF).cuda()
    off = torch.tensor([0, 2000, 4096], dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty((1, 4096, 512), dtype=BF, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(400):
            sg.experts_all_to_sharded(layers[0], x, off, out=out)
        done = torch.cuda.Event()
        done.record()
    busy = not done.query()
    layers[1].free()
    assert busy and done.query()
    layers[0].free()


@pytest.mark.parametrize("R", [40, 5])
def test_offsets_near_4_gib_of_tokens(R):
    """Rows at the end of the largest slice of activations: forward, dW and MXFP4 weights, in tiles and streams."""
    g = gen(R)
    T, K, n, E = 1000, 200, 48, 2
    ld = 2147450880 // T // 8 * 8  # T rows of ld fill the 4 GiB less 64 KiB that an offset reaches
    x = normal(g, (T, K), BF)
    wide = torch.zeros((T, ld), dtype=BF, device="cuda")
    wide[:, ld - K:] = x.cuda()
    for off8 in (0, 3):  # (rows of any alignment too)
        big = wide[:, ld - K - off8:ld - off8] if off8 else wide[:, ld - K:]
        small = big.contiguous()
        off = offsets_of(g, E, R, empty=False).cuda()
        rows = (T - 1 - torch.arange(R, dtype=torch.int32)).cuda()
        layer = sg.shard_experts(normal(g, (E, n, K), BF, 0.1).cuda(), "all-to-sharded")
        want = sg.experts_all_to_sharded(layer, small, off, rows, 1)
        assert torch.equal(sg.experts_all_to_sharded(layer, big, off, rows, 1), want)
        assert torch.isfinite(want).all() and want.any()
        dy = normal(g, (1, R, n), BF).cuda()
        for a, b in zip(sg.experts_all_to_sharded_backward(layer, big, dy, off, rows, 1),
                        sg.experts_all_to_sharded_backward(layer, small, dy, off, rows, 1)):
            assert torch.equal(a, b)
        mx = sg.shard_mxfp4_experts(*sg.quantize_mxfp4(normal(g, (E, n, 192), BF, 0.1).cuda()), "all-to-sharded")
        assert torch.equal(sg.experts_all_to_sharded(mx, big[:, :192], off, rows, 1),
                           sg.experts_all_to_sharded(mx, small[:, :192].contiguous(), off, rows, 1))
    with pytest.raises(sg.ShardGemmError) as e:  # a row's bytes more
        sg.experts_all_to_sharded(layer, torch.as_strided(wide, (T, K), (ld + 40, 1)), off, rows, 1)
    assert e.value.code == sg.ERR_UNSUPPORTED


def test_offsets_near_4_gib_of_rows():
    """The last rows of the largest packed slice: down product, both gradients of it, and the plain rows of dW."""
    g = gen(13)
    K, n = 2056, 16
    R = 2147450880 // K
    w = normal(g, (1, n, K), BF, 0.1)
    down = sg.shard_experts(w.cuda(), "sharded-to-all")
    h = torch.zeros((1, R, K), dtype=BF, device="cuda")
    h[:, -300:] = normal(g, (1, 300, K), BF).cuda()
    tail = h[:, -300:].contiguous()
    y = sg.experts_sharded_to_all(down, h)
    assert torch.equal(y[-300:], sg.experts_sharded_to_all(down, tail)) and not y[:-300].any()
    dy = torch.zeros((R, n), dtype=BF, device="cuda")
    dy[-300:] = normal(g, (300, n), BF).cuda()
    _, dw = sg.experts_sharded_to_all_backward(down, h, dy, need_dx=False)
    a, b = dy[-300:].cpu().double(), tail[0].cpu().double()
    ref.close(dw[0, 0], a.T @ b, ref.sum_bound(a.abs().T @ b.abs(), 300), "dw")
    col = sg.shard_experts(w.transpose(1, 2).contiguous().cuda(), "all-to-sharded")  # its dy is h
    dx, dw = sg.experts_all_to_sharded_backward(col, dy, h)
    assert torch.equal(dx[-300:], sg.experts_all_to_sharded_backward(col, dy[-300:], tail, need_dw=False)[0])
    assert not dx[:-300].any()
    ref.close(dw[0, 0], b.T @ a, ref.sum_bound(b.abs().T @ a.abs(), 300), "dw of columns")


@pytest.mark.parametrize("k", [0, -2])
def test_row_map_of_no_choices_is_refused(k):
    layer = sg.shard_experts(normal(gen(1), (1, 16, 64), BF).cuda(), "all-to-sharded")
    x, rows = normal(gen(2), (4, 64), BF).cuda(), torch.zeros(8, dtype=torch.int32, device="cuda")
    dy = torch.zeros((1, 8, 16), dtype=BF, device="cuda")
    for call in (lambda: sg.experts_all_to_sharded(layer, x, rows=rows, k=k),
                 lambda: sg.experts_all_to_sharded_backward(layer, x, dy, rows=rows, k=k),
                 lambda: sg.experts_all_to_sharded_backward(layer, None, dy, rows=rows, k=k, need_dw=False)):
        with pytest.raises(sg.ShardGemmError) as e:
            call()
        assert e.value.code == sg.ERR_INVALID_ARG
