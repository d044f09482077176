"""Plain 64-bit forms of the mixture-of-experts and MXFP4 operators on the CPU,
and the error bounds that go with them.  Every function takes CPU tensors and
computes in float64 from the definitions."""
import math

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half a step relative to the value: bf16 keeps 8 bits, fp16 11, fp32 24
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def route(z, k, normalize):
    """weights (T, k), experts, offsets, rows, slots by the definition."""
    T, E = z.shape
    w = torch.zeros((T, k), dtype=torch.float64)
    ex = torch.full((T, k), -1, dtype=torch.int32)
    for t in range(T):
        v = [float(a) for a in z[t].double()]
        open_ = [e for e in range(E) if v[e] > -math.inf]  # NaN compares false
        if not open_:
            continue
        order = sorted(open_, key=lambda e: (-v[e], e))[:k]
        top = v[order[0]]
        p = {e: math.exp(v[e] - top) for e in open_}
        total = sum(p[e] for e in (order if normalize else open_))
        for j, e in enumerate(order):
            ex[t, j] = e
            w[t, j] = p[e] / total
    return w, ex, *plan(ex, E)


def plan(ex, E):
    flat = ex.flatten().tolist()
    rows = [s for e in range(E) for s in range(len(flat)) if flat[s] == e] if len(flat) < 3000 else \
        [s for _, s in sorted((e, s) for s, e in enumerate(flat) if e >= 0)]
    count = [0] * E
    for e in flat:
        if e >= 0:
            count[e] += 1
    offsets = [0]
    for c in count:
        offsets.append(offsets[-1] + c)
    slots = [-1] * len(flat)
    for r, s in enumerate(rows):
        slots[s] = r
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(rows + [-1] * (len(flat) - len(rows)), dtype=i32),
            torch.tensor(slots, dtype=i32).view(ex.shape))


def route_backward(z, ex, dw, normalize):
    """dz of sum_j dw_j w_j, w the weights of the fixed choice ex."""
    z = z.double()
    dz = torch.zeros_like(z)
    for t in range(z.shape[0]):
        chosen = [int(e) for e in ex[t] if e >= 0]
        if not chosen:
            continue
        pool = chosen if normalize else [e for e in range(z.shape[1]) if z[t, e] > -math.inf]
        p = torch.softmax(z[t, pool], 0)
        g = torch.zeros(len(pool), dtype=torch.float64)
        for j, e in enumerate(int(e) for e in ex[t]):
            if e >= 0:
                g[pool.index(e)] += dw[t, j].double()
        dz[t, pool] = p * (g - (p * g).sum())
    return dz


def silu(z):
    return z / (1 + torch.exp(-z))


def shard_rows(n, S, P):
    """The unsharded rows of rank r's, in rank order: rank r's part of every segment."""
    seg, part = n // S, n // S // P
    return [[s * seg + r * part + i for s in range(S) for i in range(part)] for r in range(P)]


def product(x, w, offsets, out, bound):
    """out[m] = x[m] W_e^T for the rows of every expert; bound: the sums of magnitudes."""
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        out[a:b] = x[a:b] @ w[e].T
        bound[a:b] = x[a:b].abs() @ w[e].abs().T


def gathered(x, rows, k):
    t = torch.div(rows, k, rounding_mode="floor").long()
    ok = (rows >= 0) & (t < x.shape[0])
    return torch.where(ok[:, None], x[t.clamp(0, x.shape[0] - 1)], 0.0)


def swiglu_bound(g, u, bg, bu, n):
    """What fp32 sums of n products leave of silu(g) u: the sums' own errors
    through the derivatives (|silu'| < 1.1), and the fp32 steps of silu itself
    (expf, the sum, the quotient and the product: a few ulp, 16 half steps)."""
    eg, eu = sum_bound(bg, n), sum_bound(bu, n)
    h = silu(g) * u
    return 1.1 * (u.abs() + eu) * eg + (silu(g).abs() + 1.1 * eg) * eu + 16 * 2.0 ** -24 * h.abs()


def sum_bound(mag, n):
    """An fp32 sum of n exact products, in any order: n half steps of the sum of magnitudes."""
    return (n + 2) * 2.0 ** -24 * mag


def close(got, want, bound, what=""):
    """got (a stored dtype) within `bound` of want plus its own rounding."""
    half, tiny = HALF[got.dtype], TINY[got.dtype]
    g = got.double().cpu()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    assert torch.isfinite(g).all(), what
    off = (g - want).abs()
    allowed = bound + half * (want.abs() + bound) + tiny
    worst = (off / allowed.clamp(min=1e-300)).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the allowed error, at most {off.max().item():.3g} off"


def power(n):
    return torch.ldexp(torch.ones_like(n, dtype=torch.float64), n)


def encode(x):
    """MXFP4 codes and scales of (..., n) by the definition."""
    b = x.double().unflatten(-1, (-1, 32))
    m = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    ms = torch.where(bad | (m == 0), 1.0, m)
    ex = torch.frexp(ms)[1] - 1  # floor(log2)
    ex = torch.where(m == 0, -127, (ex - 2).clamp(-127, 127))
    q = torch.where(bad[..., None], 0.0, b) / power(ex)[..., None]
    a = q.abs().clamp(max=6.0)
    grid = torch.tensor(E2M1, dtype=torch.float64)
    d = (a[..., None] - grid).abs()
    best = d.amin(-1, keepdim=True)
    near = d == best
    # ties lie between neighbours: the even one
    even = near & (torch.arange(8) % 2 == 0)
    code = torch.where(even.any(-1), even.int().argmax(-1), near.int().argmax(-1))
    code = (code + 8 * torch.signbit(q)).to(torch.uint8)
    code = torch.where(bad[..., None], torch.zeros_like(code), code).flatten(-2)
    scales = torch.where(bad, 255, ex + 127).to(torch.uint8)
    return code[..., ::2] | (code[..., 1::2] << 4), scales


def decode(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = torch.tensor(E2M1 + [-a for a in E2M1], dtype=torch.float64)[c]
    s = torch.where(scales == 255, math.nan, power(scales.long() - 127))
    return v * s.repeat_interleave(32, -1)
