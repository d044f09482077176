"""Plain 64-bit forms of MX FP8 and of the gated block's gradients on the CPU."""
import math

import torch

import moe_ref as ref


def magnitudes():
    """What E4M3 can hold, by its code 0 .. 126."""
    return torch.tensor([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64)


def blocks(x):
    """(..., n) -> (..., ceil(n / 32), 32), zeros behind the row's end."""
    return torch.nn.functional.pad(x.double(), (0, -x.shape[-1] % 32)).unflatten(-1, (-1, 32))


def exponents(m):
    """The smallest integer e, -127 at least, with m <= 448 2^e."""
    e = torch.full_like(m, -127)
    for k in range(-127, 200):
        e = torch.where(m > 448.0 * 2.0 ** k, k + 1.0, e)
    return e.long()


def encode(x):
    """Codes and scales by the definition."""
    n, b = x.shape[-1], blocks(x)
    bad = ~torch.isfinite(b).all(-1)
    e = exponents(torch.where(bad, 0.0, b.abs().amax(-1)))
    a = torch.where(bad[..., None], 0.0, b.abs()) / ref.power(e)[..., None]
    grid = magnitudes()
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = torch.where(bad[..., None], 0, code + 128 * torch.signbit(b))
    return code.to(torch.uint8).flatten(-2)[..., :n].contiguous(), torch.where(bad, 255, e + 127).to(torch.uint8)


def decode(codes, scales):
    n = codes.shape[-1]
    c = codes.long()
    v = torch.where((c & 127) == 127, math.nan, magnitudes()[(c & 127).clamp(max=126)])
    v = torch.where(c >= 128, -v, v)
    s = torch.where(scales == 255, math.nan, ref.power(scales.long() - 127))
    return v * s.repeat_interleave(32, -1)[..., :n]


def check_kept(codes, scales, want, err, what=""):
    """Codes of values within `err` of `want`: the scale is that of a maximum within
    err, each value within half a step (2^-4 of it, or of the subnormals 2^-10)."""
    codes, scales = codes.cpu(), scales.cpu()
    got, n = decode(codes, scales), want.shape[-1]
    e = scales.double() - 127
    hi = blocks(want.abs() + err).amax(-1)
    lo = blocks((want.abs() - err).clamp(min=0)).amax(-1)
    top = 448 * ref.power(e.long())
    assert (lo <= top).all() and ((hi > top / 2) | (e == -127)).all(), f"{what}: scales"
    step = ref.power(e.long()).repeat_interleave(32, -1)[..., :n]
    off = (got - want).abs()
    allowed = err + torch.maximum(2.0 ** -4 * (want.abs() + err), 2.0 ** -10 * step)
    worst = (off / allowed).max().item()
    assert worst <= 1, f"{what}: {worst:.3g} times the allowed error"


def gated_grad(g, u, dh):
    """dg, du, h of h = silu(g) u."""
    s = 1 / (1 + torch.exp(-g))
    return dh * u * s * (1 + g * (1 - s)), dh * g * s, g * s * u


def gated_bounds(g, u, dh, e_dh):
    """Errors of dg, du, h for a dh that is off by e_dh: through the factors, and 16
    half steps of fp32 of each product (dg's sum: of its terms' magnitudes)."""
    s = 1 / (1 + torch.exp(-g))
    ulp = 16 * 2.0 ** -24
    big = (u * s).abs() * (1 + g.abs() * (1 - s))
    dg = (u * s * (1 + g * (1 - s))).abs() * e_dh + ulp * big * (dh.abs() + e_dh)
    du = (g * s).abs() * (e_dh + ulp * (dh.abs() + e_dh))
    return dg, du, ulp * (g * s * u).abs()
