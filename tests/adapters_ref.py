"""Plain 64-bit forms of the low-rank adapters on the CPU, and their error bounds."""
import torch

import moe_ref as ref

# what hi + lo in the operand's type leave of a value: half a step of a half step
SPLIT = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22}


def plan(which, n):
    """offsets (n + 2), rows: tokens in order (adapter, token), those without one last."""
    g = [int(a) if 0 <= int(a) < n else n for a in which]
    rows = sorted(range(len(g)), key=lambda t: (g[t], t))
    offsets = [sum(1 for a in g if a < b) for b in range(n + 2)]
    return offsets, rows


def tokens(which, a):
    return torch.nonzero(which == a).flatten()


def full(v, order):
    """(P, T, w / P) -> (T, w), `order` the unsharded columns of each rank."""
    w = sum(len(o) for o in order)
    z = torch.zeros((v.shape[1], w), dtype=torch.float64)
    for r, o in enumerate(order):
        z[:, o] = v[r].double()
    return z


def half(x, A, scale):
    """scale x A^T and its bound as an fp32 sum, split in two."""
    u, mag = x @ A.T, x.abs() @ A.abs().T
    e = ref.sum_bound(mag, x.shape[1]) + 2.0 ** -23 * u.abs()
    return scale * u, abs(scale) * e


def split_bound(u, e, dtype):
    """The error of an operand hi + lo of u, itself off by e (fp16: of its row's largest
    magnitude, 2^-36 at most)."""
    low = 2.0 ** -36 * (u.abs() + e).amax(-1, keepdim=True) if dtype == torch.float16 else 0.0
    return e + SPLIT[dtype] * (u.abs() + e) + low


def delta(x, which, A, B, scale, dtype):
    """scale_a (x A_a^T) B_a^T of every token, and its bound."""
    n, r = A.shape[0], A.shape[1]
    out = torch.zeros((x.shape[0], B.shape[1]), dtype=torch.float64)
    bound = torch.zeros_like(out)
    for a in range(n):
        t = tokens(which, a)
        if not len(t):
            continue
        u, e = half(x[t], A[a].double(), float(scale[a]))
        e = split_bound(u, e, dtype)
        out[t] = u @ B[a].double().T
        bound[t] = e @ B[a].double().abs().T + ref.sum_bound((u.abs() + e) @ B[a].double().abs().T, 2 * r)
    return out, bound


def gradients(x, dy, which, A, B, scale, dtype):
    """(dx through the adapters, dA, dB), each with its bound."""
    n = A.shape[0]
    dx, bx = torch.zeros_like(x), torch.zeros_like(x)
    dA, bA = torch.zeros(A.shape, dtype=torch.float64), torch.zeros(A.shape, dtype=torch.float64)
    dB, bB = torch.zeros(B.shape, dtype=torch.float64), torch.zeros(B.shape, dtype=torch.float64)
    for a in range(n):
        t = tokens(which, a)
        if not len(t):
            continue
        k, Ad, Bd = float(scale[a]), A[a].double(), B[a].double()
        v, ev = half(dy[t], Bd.T, k)
        u, eu = half(x[t], Ad, k)
        e = split_bound(v, ev, dtype)
        dx[t], bx[t] = v @ Ad, e @ Ad.abs() + ref.sum_bound((v.abs() + e) @ Ad.abs(), 2 * A.shape[1])
        for got, b, m, em, z in ((dA, bA, v, ev, x[t]), (dB, bB, u, eu, dy[t])):
            # (fp16: 32 rows share a power of two, so the small ones are off by their largest)
            s = split_bound(m, em, dtype) + (2.0 ** -36 * (m.abs() + em).max() if dtype == torch.float16 else 0.0)
            val = m.T @ z
            err = s.T @ z.abs() + ref.sum_bound((m.abs() + s).T @ z.abs(), 2 * len(t))
            got[a], b[a] = (val, err) if got is dA else (val.T, err.T)
    return (dx, bx), (dA, bA), (dB, bB)
