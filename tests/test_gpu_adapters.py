"""Low-rank adapters beside a shared projection against their 64-bit definitions:
the plan, forward and backward beside layers of every kind and mode, ranks and
sizes that fill nothing, tokens without an adapter.

Tolerances (adapters_ref): x A^T is an fp32 sum; as an operand it is split into two
16-bit halves, off by 2^-16 (bf16) or 2^-22 (fp16) of itself; then an fp32 sum of
2 rank products more beside the projection's own, and one rounding.  Quantized
weights: as their codes, or in two such halves."""
import math

import pytest
import torch

import adapters_ref as aref
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


def draw_which(g, T, n):
    w = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32)
    if T > 4:
        w[T // 2], w[T // 3] = n + 3, -9  # no adapters either
    if n > 2:
        w[w == 1] = 0  # one without tokens
    return w


# ---- plan -------------------------------------------------------------------

@pytest.mark.parametrize("T,n", [(0, 3), (1, 1), (16, 32), (63, 2), (64, 1), (65, 1), (700, 5), (1025, 1024), (5000, 64),
                                 (20000, 3)])
def test_plan(T, n):
    which = draw_which(gen(T + n), T, n)
    p = sg.adapter_plan(which.cuda(), n)
    data = p.data.cpu().tolist()
    offsets, rows = aref.plan(which, n)
    assert data[:n + 2] == offsets and data[n + 2:n + 2 + T] == rows
    group = [int(w) if 0 <= int(w) < n else n for w in which]
    assert data[n + 2 + T:n + 2 + 2 * T] == [group[t] for t in rows]
    height = 64 if T >= 32 * (n + 1) else 16
    at = (n + 2 + 2 * T + 3) // 4 * 4
    tiles = [tuple(data[i:i + 3]) for i in range(at, len(data) // 4 * 4, 4)]
    want = [(a, r, min(height, offsets[a + 1] - r)) for a in range(n + 1)
            for r in range(offsets[a], offsets[a + 1], height)]
    assert tiles[:len(want)] == want and all(t[0] == -1 for t in tiles[len(want):len(data) // 4])


# ---- forward ----------------------------------------------------------------

# T, in, out, mode, P, S, n, rank, dtype
CASES = [
    (1, 8, 1, 0, 1, 1, 1, 1, BF), (1, 64, 32, 1, 2, 1, 3, 8, HF), (5, 35, 21, 0, 3, 1, 2, 5, BF),
    (16, 256, 192, 0, 4, 3, 20, 16, BF), (17, 96, 50, 1, 3, 1, 4, 17, HF), (33, 1000, 726, 0, 2, 1, 3, 12, HF),
    (70, 512, 96, 1, 4, 2, 2, 64, BF), (130, 72, 130, 0, 1, 2, 1, 100, HF), (300, 264, 520, 0, 2, 2, 3, 32, BF),
    (300, 264, 200, 1, 2, 1, 3, 4, HF), (700, 130, 77, 0, 7, 1, 6, 24, BF), (640, 2048, 64, 1, 8, 1, 2, 16, BF),
    (200, 4096, 48, 0, 2, 1, 1, 40, HF), (90, 64, 64, 0, 1, 1, 60, 200, BF), (1100, 40, 3000, 0, 1, 1, 2, 8, HF),
    # enough tiles for the products with the adapters in their epilogue: forward, backward
    (300, 100, 3003, 0, 3, 1, 3, 12, BF), (300, 36, 2820, 0, 2, 2, 2, 20, HF), (300, 45, 2900, 1, 3, 1, 2, 9, BF),
    (300, 2900, 45, 0, 3, 1, 3, 16, HF), (300, 2904, 50, 1, 2, 1, 3, 8, BF), (300, 2816, 64, 1, 2, 2, 2, 16, BF),
    (300, 2900, 64, 1, 2, 2, 2, 7, HF), (12, 64, 20480, 0, 4, 2, 30, 16, BF), (60, 20480, 72, 0, 1, 1, 9, 36, HF),
    (1500, 128, 4100, 0, 2, 2, 3, 16, HF), (1500, 4100, 96, 0, 2, 1, 3, 40, BF), (1500, 64, 4224, 0, 1, 2, 90, 8, BF),
]


def case_of(T, i, o, mode, P, S, n, r, dtype, which=None):
    g = gen(T + i + o + r)
    w = normal(g, (o, i), dtype, 1 / math.sqrt(i))
    layer = sg.shard_linear(w.cuda(), mode, segments=S, P=P)
    A, B = normal(g, (n, r, i), dtype, 1 / math.sqrt(i)), normal(g, (n, o, r), dtype, 1 / math.sqrt(r))
    scale = torch.rand(n, generator=g) + 0.5
    which = draw_which(g, T, n) if which is None else which
    x, dy = normal(g, (T, i), dtype), normal(g, (T, o), dtype)
    order = ref.shard_rows(o if mode == 0 else i, S, P)
    shard = lambda v: torch.stack([v[:, q] for q in order])  # noqa: E731
    xs, dys = (x, shard(dy)) if mode == 0 else (shard(x), dy)
    layer.weight = w.double()  # for the tests
    return layer, sg.Adapters(A.cuda(), B.cuda(), scale.cuda()), which, xs, dys, x.double(), dy.double(), order, shard


def exact_base(layer, x, shard=None):
    """x W^T and its bound as an fp32 sum."""
    v, e = x @ layer.weight.T, ref.sum_bound(x.abs() @ layer.weight.abs().T, x.shape[1])
    return (shard(v), shard(e)) if shard else (v, e)


def base_of(layer, x, mode):
    return (sg.all_to_sharded(layer, x.cuda(), out_dtype=F32) if mode == 0 else
            sg.sharded_to_all(layer, x.cuda(), out_dtype=F32)).double().cpu()


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    T, i, o, mode, P, S, n, r, dtype = case
    layer, ad, which, xs, _, x, _, order, shard = case_of(*case)
    plan = sg.adapter_plan(which.cuda(), n)
    d, e = aref.delta(x, which, ad.A.cpu(), ad.B.cpu(), ad.scale.cpu(), dtype)
    d, e = (shard(d), shard(e)) if mode == 0 else (d, e)
    base, eb = exact_base(layer, x, shard if mode == 0 else None)
    call = sg.adapted_all_to_sharded if mode == 0 else sg.adapted_sharded_to_all
    # (the sums of both parts in one: the adapters' 2 rank + 1 steps act on the base, too)
    eb = eb + (2 * r + 4) * 2.0 ** -24 * (base.abs() + d.abs() + e)
    for out in (dtype, F32):
        y = call(layer, xs.cuda(), ad, plan, out_dtype=out)
        ref.close(y, base + d, e + eb, f"y {out}")
    assert torch.equal(y, call(layer, xs.cuda(), ad, plan, out_dtype=F32))  # the same run to run
    one = sg.Adapters(ad.A, ad.B)  # scale 1
    y1 = call(layer, xs.cuda(), one, plan, out_dtype=F32)
    d1, e1 = aref.delta(x, which, ad.A.cpu(), ad.B.cpu(), torch.ones(n), dtype)
    d1, e1 = (shard(d1), shard(e1)) if mode == 0 else (d1, e1)
    ref.close(y1, base + d1, e1 + eb + (2 * r + 4) * 2.0 ** -24 * d1.abs(), "scale 1")
    if mode == 0:
        z = sg.adapted_all_to_sharded(layer, xs.cuda(), ad, plan, gather=True, out_dtype=F32)
        assert torch.equal(z.view(T, P, -1).transpose(0, 1), y)
        z = sg.adapted_all_to_sharded(layer, xs.cuda(), ad, plan, gather=True)
        assert torch.equal(z.view(T, P, -1).transpose(0, 1), call(layer, xs.cuda(), ad, plan))


@pytest.mark.parametrize("case", [c for c in CASES if c[3] == 0 and c[5] == 2])
def test_forward_swiglu(case):
    T, i, o, mode, P, S, n, r, dtype = case
    layer, ad, which, xs, _, x, _, order, shard = case_of(*case)
    plan = sg.adapter_plan(which.cuda(), n)
    d, e = aref.delta(x, which, ad.A.cpu(), ad.B.cpu(), ad.scale.cpu(), dtype)
    base, eb = exact_base(layer, x, shard)
    z, e = base + shard(d), shard(e) + eb
    e = e + (2 * r + 4) * 2.0 ** -24 * (base.abs() + shard(d).abs() + e)
    f = z.shape[-1] // 2
    (a, b), (ea, eb) = z.split(f, -1), e.split(f, -1)
    want = ref.silu(a) * b
    # through the derivatives (|silu'| < 1.1), and fp32's steps of silu
    bound = 1.1 * (b.abs() + eb) * ea + (ref.silu(a).abs() + 1.1 * ea) * eb + 16 * 2.0 ** -24 * want.abs()
    for out in (dtype, F32):
        h = sg.adapted_all_to_sharded(layer, xs.cuda(), ad, plan, swiglu=True, out_dtype=out)
        ref.close(h, want, bound, f"h {out}")


@pytest.mark.parametrize("T", [1, 8, 40, 200])
@pytest.mark.parametrize("kind", ["q4", "q4 f16", "mx8"])
@pytest.mark.parametrize("mode,i,o", [(0, 512, 256), (1, 512, 256), (0, 576, 6020), (1, 640, 6016)])
def test_beside_quantized_layers(mode, i, o, kind, T):
    """4-bit layers whose codes come in whole runs of 256 inputs, and others."""
    g = gen(T + mode)
    P, n, r = 2, 3, 16
    dtype = HF if kind == "q4 f16" else BF
    if kind != "mx8":
        w = torch.randint(-2 ** 31, 2 ** 31, (o, i // 8), generator=g, dtype=torch.int64).to(torch.int32)
        sc = (torch.rand((o, i // 64), generator=g) * 0.01).half()
        qb = (-7 * sc).half()
        layer = sg.shard_quantized_linear(w.cuda(), sc.view(torch.int16).cuda(), qb.view(torch.int16).cuda(), i, mode, P=P,
                                          act_dtype=dtype)
        q = ((w.long() & 0xffffffff)[..., None] >> (4 * torch.arange(8)) & 15).flatten(1).double()
        sq, b = sc.double().repeat_interleave(64, 1) * q, qb.double().repeat_interleave(64, 1)
        W, size = sq + b, sq.abs() + b.abs()
    else:
        codes, scales = mx.encode(normal(g, (o, i), F32, 0.05))
        layer = sg.shard_mxfp8_linear(codes.cuda(), scales.cuda(), mode, P=P)
        W = mx.decode(codes, scales)
        size = W.abs()
    A, B = normal(g, (n, r, i), dtype, 0.05), normal(g, (n, o, r), dtype, 0.2)
    scale, which = torch.rand(n, generator=g), draw_which(g, T, n)
    x, dy = normal(g, (T, i), dtype), normal(g, (T, o), dtype)
    order = ref.shard_rows(o if mode == 0 else i, 1, P)
    shard = lambda v: torch.stack([v[:, q] for q in order])  # noqa: E731
    xs, dys = (x, shard(dy)) if mode == 0 else (shard(x), dy)
    ad, plan = sg.Adapters(A.cuda(), B.cuda(), scale.cuda()), sg.adapter_plan(which.cuda(), n)
    d, e = aref.delta(x.double(), which, A, B, scale, dtype)
    # the projection: fp32 sums of the codes' and the biases' products, or of the weights
    # in two halves (2^-16 or 2^-22 of them)
    base = x.double() @ W.T
    e = e + (aref.SPLIT[dtype] + (2 * i + 2 * r + 8) * 2.0 ** -24) * (x.double().abs() @ size.T + d.abs())
    d, e, base = (shard(d), shard(e), shard(base)) if mode == 0 else (d, e, base)
    call = sg.adapted_all_to_sharded if mode == 0 else sg.adapted_sharded_to_all
    for out in (dtype, F32):
        ref.close(call(layer, xs.cuda(), ad, plan, out_dtype=out), base + d, e, "y")
    back = sg.adapted_all_to_sharded_backward if mode == 0 else sg.adapted_sharded_to_all_backward
    none, dA, dB = back(layer, xs.cuda(), dys.cuda(), ad, plan, need_dx=False)
    _, (wA, eA), (wB, eB) = aref.gradients(x.double(), dy.double(), which, A, B, scale, dtype)
    assert none is None
    ref.close(dA, wA, eA, "dA")
    ref.close(dB, wB, eB, "dB")
    with pytest.raises(sg.ShardGemmError, match="dense layers only"):
        back(layer, xs.cuda(), dys.cuda(), ad, plan)


# (4-bit groups of 64 lie in one rank; the epilogue is the all-to-sharded layer's)
ODD = [(mode, i, o, P, kind, swiglu, bias)
       for mode, i, o, P in [(0, 1344, 512, 4), (1, 1408, 176, 2), (0, 832, 488, 1), (1, 768, 40, 8)]
       for kind in ("q4", "mx8") if not (mode and kind == "q4" and i // P % 64)
       for swiglu, bias in ((False, False), (False, True), (True, False)) if not (mode and swiglu)]


@pytest.mark.parametrize("T", [3, 22, 33])
@pytest.mark.parametrize("mode,i,o,P,kind,swiglu,bias", ODD)
def test_quantized_layers_of_odd_sizes(mode, i, o, P, kind, T, swiglu, bias):
    """Layers whose codes no matrix-core kernel takes, up to 32 tokens and behind; with biases."""
    g = gen(T + o)
    n, r = 3, 12
    be = normal(g, (o,), BF) if bias else None
    b = be.cuda() if bias else None
    if kind == "q4":
        w = torch.randint(-2 ** 31, 2 ** 31, (o, i // 8), generator=g, dtype=torch.int64).to(torch.int32)
        sc = (torch.rand((o, i // 64), generator=g) * 0.01).half()
        qb = (-7 * sc).half()
        layer = sg.shard_quantized_linear(w.cuda(), sc.view(torch.int16).cuda(), qb.view(torch.int16).cuda(), i, mode, P=P,
                                          act_dtype=BF, bias=b, segments=2 if swiglu else 1)
        q = ((w.long() & 0xffffffff)[..., None] >> (4 * torch.arange(8)) & 15).flatten(1).double()
        sq, qb = sc.double().repeat_interleave(64, 1) * q, qb.double().repeat_interleave(64, 1)
        W, size = sq + qb, sq.abs() + qb.abs()
    else:
        codes, scales = mx.encode(normal(g, (o, i), F32, 0.05))
        layer = sg.shard_mxfp8_linear(codes.cuda(), scales.cuda(), mode, P=P, bias=b, segments=2 if swiglu else 1)
        W = mx.decode(codes, scales)
        size = W.abs()
    A, B = normal(g, (n, r, i), BF, 0.05), normal(g, (n, o, r), BF, 0.2)
    scale, which = torch.rand(n, generator=g), draw_which(g, T, n)
    x = normal(g, (T, i), BF)
    order = ref.shard_rows(o if mode == 0 else i, 1, P)
    ad, plan = sg.Adapters(A.cuda(), B.cuda(), scale.cuda()), sg.adapter_plan(which.cuda(), n)
    d, e = aref.delta(x.double(), which, A, B, scale, BF)
    base = x.double() @ W.T + (be.double() if bias else 0)
    # fp32 sums of the codes' and the biases' products, or of the weights in two halves (2^-16)
    e = e + (aref.SPLIT[BF] + (2 * i + 2 * r + 8) * 2.0 ** -24) * (x.double().abs() @ size.T + d.abs())
    e = e + 4 * 2.0 ** -24 * base.abs()
    want, bound = base + d, e
    if swiglu:  # through the derivatives (|silu'| < 1.1), and fp32's steps of silu
        (a, b), (ea, eb) = want.chunk(2, 1), e.chunk(2, 1)
        want = ref.silu(a) * b
        bound = 1.1 * (b.abs() + eb) * ea + (ref.silu(a).abs() + 1.1 * ea) * eb + 16 * 2.0 ** -24 * want.abs()
        order = ref.shard_rows(o // 2, 1, P)
    shard = lambda v: torch.stack([v[:, q] for q in order])  # noqa: E731
    xs = (shard(x) if mode else x).cuda()
    want, bound = (want, bound) if mode else (shard(want), shard(bound))
    for out in (BF, F32):
        y = (sg.adapted_sharded_to_all(layer, xs, ad, plan, out_dtype=out) if mode
             else sg.adapted_all_to_sharded(layer, xs, ad, plan, swiglu=swiglu, out_dtype=out))
        ref.close(y, want, bound, "y")


# ---- backward ---------------------------------------------------------------

@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    T, i, o, mode, P, S, n, r, dtype = case
    layer, ad, which, xs, dys, x, dy, order, shard = case_of(*case)
    plan = sg.adapter_plan(which.cuda(), n)
    (dx, ex), (dA, eA), (dB, eB) = aref.gradients(x, dy, which, ad.A.cpu(), ad.B.cpu(), ad.scale.cpu(), dtype)
    base, eb = dy @ layer.weight, ref.sum_bound(dy.abs() @ layer.weight.abs(), o)
    ex = ex + eb + (2 * r + 4) * 2.0 ** -24 * (base.abs() + dx.abs() + ex)
    if mode == 0:
        back = sg.adapted_all_to_sharded_backward
    else:
        base, dx, ex = shard(base), shard(dx), shard(ex)
        back = sg.adapted_sharded_to_all_backward
    for dt in (dtype, F32):
        gx, gA, gB = back(layer, xs.cuda(), dys.cuda(), ad, plan, dx_dtype=dt, d_dtype=dt)
        ref.close(gx, base + dx, ex, f"dx {dt}")
        ref.close(gA, dA, eA, f"dA {dt}")
        ref.close(gB, dB, eB, f"dB {dt}")
    only, n1, n2 = back(layer, None, dys.cuda(), ad, plan, need_d=False, dx_dtype=F32)
    assert n1 is None and n2 is None and torch.equal(only, gx)
    none, a, b = back(layer, xs.cuda(), dys.cuda(), ad, plan, need_dx=False)
    assert none is None and torch.equal(a, gA) and torch.equal(b, gB)


def test_gradients_by_differences():
    """The formulas the kernels are held to, against differences of the projection."""
    g = gen(3)
    T, i, o, n, r = 9, 12, 10, 3, 4
    x, dy, w = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((T, i), (T, o), (o, i)))
    A, B = torch.randn((n, r, i), generator=g, dtype=torch.float64), torch.randn((n, o, r), generator=g, dtype=torch.float64)
    scale, which = torch.rand(n, generator=g), draw_which(g, T, n)
    (dx, _), (dA, _), (dB, _) = aref.gradients(x, dy, which, A, B, scale, BF)

    def loss(x, A, B):
        return ((x @ w.T + aref.delta(x, which, A, B, scale, BF)[0]) * dy).sum()

    args = [x, A, B]
    for k, grad in enumerate((dx + dy @ w, dA, dB)):
        for _ in range(4):
            v = torch.randn(args[k].shape, generator=g, dtype=torch.float64)
            hi, lo = (loss(*(p + (s * 1e-5 * v if j == k else 0) for j, p in enumerate(args))) for s in (1, -1))
            assert abs((v * grad).sum() - (hi - lo) / 2e-5) <= 1e-7 * (v * grad).abs().sum()


@pytest.mark.parametrize("size", [1e-7, 3e4])
def test_fp16_far_from_one(size):
    """Gradients of 1e-7 and products beyond 65504 keep their digits in fp16 layers."""
    g = gen(8)
    T, i, o, n, r = 70, 64, 96, 2, 16
    layer = sg.shard_linear(normal(g, (o, i), HF, 0.1).cuda(), 0)
    A, B = normal(g, (n, r, i), HF, 1.0), normal(g, (n, o, r), HF, 1e-3 if size > 1 else 1.0)
    which, scale = draw_which(g, T, n), torch.ones(n)
    x = (normal(g, (T, i)) * (size if size > 1 else 1.0)).clamp(-60000, 60000).to(HF)
    dy = (normal(g, (T, o)) * size).clamp(-60000, 60000).to(HF)
    ad, plan = sg.Adapters(A.cuda(), B.cuda()), sg.adapter_plan(which.cuda(), n)
    d, e = aref.delta(x.double(), which, A, B, scale, HF)
    base = base_of(layer, x, 0)
    y = sg.adapted_all_to_sharded(layer, x.cuda(), ad, plan, out_dtype=F32)
    ref.close(y, base + d[None], e + 2.0 ** -24 * (base.abs() + d.abs() + e), "y")
    _, gA, gB = sg.adapted_all_to_sharded_backward(layer, x.cuda(), dy.cuda()[None], ad, plan, need_dx=False)
    _, (dA, eA), (dB, eB) = aref.gradients(x.double(), dy.double(), which, A, B, scale, HF)
    ref.close(gA, dA, eA, "dA")
    ref.close(gB, dB, eB, "dB")


@pytest.mark.parametrize("T,i,o", [(20, 72, 104), (300, 72, 104), (300, 72, 3000), (300, 2904, 40), (40, 64, 17000)])
def test_tokens_stay_apart(T, i, o):
    """An infinite or NaN token reaches no other one, nor other adapters' gradients;
    an infinite adapter reaches its own tokens only."""
    g = gen(T)
    n, r = 3, 12
    layer = sg.shard_linear(normal(g, (o, i), BF, 0.1).cuda(), 0)
    A, B = normal(g, (n, r, i), BF, 0.1), normal(g, (n, o, r), BF, 0.1)
    which = torch.randint(0, n, (T,), generator=g, dtype=torch.int32)
    which[3], which[4], which[5] = 2, 2, 0
    x, dy = normal(g, (T, i), BF), normal(g, (1, T, o), BF)
    plan = sg.adapter_plan(which.cuda(), n)

    def both(x, dy, B):
        ad = sg.Adapters(A.cuda(), B.cuda())
        return (sg.adapted_all_to_sharded(layer, x.cuda(), ad, plan)[0],
                *sg.adapted_all_to_sharded_backward(layer, x.cuda(), dy.cuda(), ad, plan))

    clean = both(x, dy, B)
    x[3, 7], x[4, 9], dy[0, 3, 2] = math.inf, math.nan, -math.inf
    got = both(x, dy, B)
    keep = [t for t in range(T) if t not in (3, 4)]
    assert torch.equal(got[0][keep], clean[0][keep])
    assert torch.equal(got[1][[t for t in range(T) if t != 3]], clean[1][[t for t in range(T) if t != 3]])
    for a, b in zip(got[2:], clean[2:]):
        assert torch.equal(a[:2], b[:2])
    x[3, 7] = x[4, 9] = dy[0, 3, 2] = 0
    clean = both(x, dy, B)
    B[1] = math.inf
    got = both(x, dy, B)
    other = (which != 1).cuda()
    assert torch.equal(got[0][other], clean[0][other]) and torch.equal(got[1][other], clean[1][other])
    assert torch.equal(got[2][[0, 2]], clean[2][[0, 2]]) and torch.equal(got[3], clean[3])


def test_no_tokens_and_no_adapters():
    g = gen(1)
    layer = sg.shard_linear(normal(g, (32, 16), BF).cuda(), 0, P=2)
    ad = sg.Adapters(normal(g, (2, 8, 16), BF).cuda(), normal(g, (2, 32, 8), BF).cuda())
    plan = sg.adapter_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 2)
    x, dy = torch.empty((0, 16), dtype=BF, device="cuda"), torch.empty((2, 0, 16), dtype=BF, device="cuda")
    assert sg.adapted_all_to_sharded(layer, x, ad, plan).shape == (2, 0, 16)
    dx, dA, dB = sg.adapted_all_to_sharded_backward(layer, x, dy, ad, plan)
    assert dx.shape == (0, 16) and (dA == 0).all() and (dB == 0).all()
    x = normal(g, (50, 16), BF).cuda()
    plan = sg.adapter_plan(torch.full((50,), -1, dtype=torch.int32, device="cuda"), 2)
    assert torch.equal(sg.adapted_all_to_sharded(layer, x, ad, plan), sg.all_to_sharded(layer, x))


@pytest.mark.parametrize("T,i,o", [(24, 64, 96), (400, 64, 96), (400, 64, 3000), (400, 3000, 64), (24, 64, 17000)])
def test_bad_plans_stay_inside(T, i, o):
    """A plan of any contents leads out of no array (its results are unspecified)."""
    g = gen(2)
    n, r = 2, 16
    layer = sg.shard_linear(normal(g, (o, i), BF).cuda(), 0)
    ad = sg.Adapters(normal(g, (n, r, i), BF).cuda(), normal(g, (n, o, r), BF).cuda())
    x, dy = normal(g, (T, i), BF).cuda(), normal(g, (1, T, o), BF).cuda()
    good = sg.adapter_plan(torch.zeros(T, dtype=torch.int32, device="cuda"), n)
    guard = torch.full((3, T, o), 7.0, dtype=BF, device="cuda")
    for fill in (-1, 1 << 30, -(1 << 30), 1, T - 1):
        bad = sg.AdapterPlan(torch.full_like(good.data, fill), T, n)
        sg.adapted_all_to_sharded(layer, x, ad, bad, out=guard[1:2])
        sg.adapted_all_to_sharded_backward(layer, x, dy, ad, bad)
        torch.cuda.synchronize()
        assert (guard[0] == 7).all() and (guard[2] == 7).all()


@pytest.mark.parametrize("i,o,n,r,T", [(256, 384, 4, 16, 30), (200, 6000, 4, 12, 300)])
def test_on_another_stream_and_in_graphs(i, o, n, r, T):
    g = gen(5)
    layer = sg.shard_linear(normal(g, (o, i), BF, 0.1).cuda(), 0, segments=2, P=2)
    down = sg.shard_linear(normal(g, (i, o // 2), BF, 0.1).cuda(), 1, P=2)
    ad = sg.Adapters(normal(g, (n, r, i), BF, 0.1).cuda(), normal(g, (n, o, r), BF, 0.1).cuda())
    ad2 = sg.Adapters(normal(g, (n, r, o // 2), BF, 0.1).cuda(), normal(g, (n, i, r), BF, 0.1).cuda())
    xs = [normal(g, (T, i), BF).cuda() for _ in range(4)]
    ws = [draw_which(g, T, n).cuda() for _ in range(4)]

    def step(x, which):  # the adapted MLP of a step, and the gradients of its down layer
        plan = sg.adapter_plan(which, n)
        h = sg.adapted_all_to_sharded(layer, x, ad, plan, swiglu=True)
        y = sg.adapted_sharded_to_all(down, h, ad2, plan)
        return (h, y, *sg.adapted_sharded_to_all_backward(down, h, y, ad2, plan))

    want = [step(a, b) for a, b in zip(xs, ws)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step(xs[1], ws[1])
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    pairs = []
    for k in range(2):  # two graphs, replayed in turn
        x, w = xs[k].clone(), ws[k].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(x, w)
        pairs.append((graph, x, w, out))
    for k in (1, 2, 3, 0):
        for graph, x, w, out in pairs:
            x.copy_(xs[k])
            w.copy_(ws[k])
            graph.replay()
            step(xs[0], ws[0])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[k])), k


@pytest.mark.parametrize("T", [5, 30])
@pytest.mark.parametrize("kind", ["q4", "mx8"])
def test_quantized_layers_of_odd_sizes_in_graphs(kind, T):
    g = gen(T)
    i, o, n, r = 448, 240, 3, 16
    if kind == "q4":
        w = torch.randint(-2 ** 31, 2 ** 31, (o, i // 8), generator=g, dtype=torch.int64).to(torch.int32)
        sc = (torch.rand((o, i // 64), generator=g) * 0.01).half()
        layer = sg.shard_quantized_linear(w.cuda(), sc.view(torch.int16).cuda(), (-7 * sc).half().view(torch.int16).cuda(), i,
                                          0, P=2, act_dtype=BF)
    else:
        codes, scales = mx.encode(normal(g, (o, i), F32, 0.05))
        layer = sg.shard_mxfp8_linear(codes.cuda(), scales.cuda(), 0, P=2)
    ad = sg.Adapters(normal(g, (n, r, i), BF, 0.1).cuda(), normal(g, (n, o, r), BF, 0.1).cuda())
    xs, ws = [normal(g, (T, i), BF).cuda() for _ in range(3)], [draw_which(g, T, n).cuda() for _ in range(3)]
    x, which = xs[0].clone(), ws[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # the layer's first adapted call: nothing of it is built before
        out = sg.adapted_all_to_sharded(layer, x, ad, sg.adapter_plan(which, n))
    want = [sg.adapted_all_to_sharded(layer, a, ad, sg.adapter_plan(b, n)) for a, b in zip(xs, ws)]
    for k in (1, 2, 0, 1):
        x.copy_(xs[k])
        which.copy_(ws[k])
        graph.replay()
        sg.adapted_all_to_sharded(layer, xs[0], ad, sg.adapter_plan(ws[0], n))
        torch.cuda.synchronize()
        assert torch.equal(out, want[k]), k


def test_adapters_trained_on_a_kept_input():
    """One layer's adapters from an input kept in 8 bits: the gradients of the values
    that were kept, and how a step down the gradient lowers the loss's linear part."""
    g = gen(6)
    T, i, o, n, r = 200, 128, 160, 2, 8
    layer = sg.shard_linear(normal(g, (o, i), BF, 0.1).cuda(), 0, P=2)
    ad = sg.Adapters(normal(g, (n, r, i), BF, 0.1).cuda(), normal(g, (n, o, r), BF, 0.1).cuda())
    which = draw_which(g, T, n)
    plan = sg.adapter_plan(which.cuda(), n)
    x, dy = normal(g, (T, i), BF).cuda(), normal(g, (2, T, o // 2), BF).cuda()
    kept = sg.quantize_mxfp8(x)
    back = sg.dequantize_mxfp8(*kept, out_dtype=BF)
    dx, dA, dB = sg.adapted_all_to_sharded_backward(layer, back, dy, ad, plan)
    x8 = mx.decode(*(v.cpu() for v in kept))
    order = ref.shard_rows(o, 1, 2)
    _, (wA, eA), (wB, eB) = aref.gradients(x8, aref.full(dy.cpu(), order), which, ad.A.cpu(), ad.B.cpu(), torch.ones(n), BF)
    ref.close(dA, wA, eA, "dA")
    ref.close(dB, wB, eB, "dB")
    assert torch.isfinite(dx).all()
