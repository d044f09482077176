"""The gated block and MX FP8 activations without a GPU: what the entry points
refuse on the host, and the reference forms the GPU tests go by."""
import ctypes as C
import math
import os

import pytest
import torch

import moe_ref as ref
import mx8_ref as mx
import sharded_gemm_alltosharded_amd as sg

PTR = C.c_void_p(0x1000)  # never dereferenced: the calls below fail before


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sg.LIB_PATH):
        pytest.skip("library not built")
    return sg.lib()


def err(L):
    return L.sg_last_error().decode()


def test_quantize_refuses(L):
    q = lambda x=PTR, dt=sg.BF16, r=2, c=40, ld=40, co=PTR, sc=PTR: L.sg_quantize_mxfp8(x, dt, r, c, ld, co, sc, None)  # noqa: E731
    assert q(dt=7) == sg.ERR_INVALID_ARG and "dtype" in err(L)
    assert q(r=-1) == sg.ERR_INVALID_ARG and q(c=-1) == sg.ERR_INVALID_ARG
    assert q(ld=39) == sg.ERR_INVALID_ARG and "stride" in err(L)
    assert q(x=None) == sg.ERR_INVALID_ARG and q(co=None) == sg.ERR_INVALID_ARG and q(sc=None) == sg.ERR_INVALID_ARG
    assert q(r=1 << 40) == sg.ERR_UNSUPPORTED
    assert q(r=0) == sg.OK and q(c=0) == sg.OK
    d = lambda co=PTR, sc=PTR, r=2, c=40, x=PTR, dt=sg.BF16: L.sg_dequantize_mxfp8(co, sc, r, c, x, dt, None)  # noqa: E731
    assert d(dt=7) == sg.ERR_INVALID_ARG and d(co=None) == sg.ERR_INVALID_ARG and d(sc=None) == sg.ERR_INVALID_ARG
    assert d(x=None) == sg.ERR_INVALID_ARG and d(r=-1) == sg.ERR_INVALID_ARG and d(r=1 << 40) == sg.ERR_UNSUPPORTED
    assert d(r=0) == sg.OK


def test_missing_layers_are_refused(L):
    assert L.sg_experts_gated(None, PTR, 1, 8, None, None, 1, 1, PTR, PTR, PTR, PTR, 0, None) == sg.ERR_INVALID_ARG
    assert "layer is NULL" in err(L)
    assert L.sg_experts_gated_backward(None, PTR, PTR, PTR, None, 1, PTR, PTR, None) == sg.ERR_INVALID_ARG
    assert L.sg_gated_mlp(None, None, PTR, 1, 8, None, None, 1, 1, PTR, 1, PTR, PTR, PTR, PTR, PTR, 0,
                          None) == sg.ERR_INVALID_ARG
    assert L.sg_gated_mlp_backward(None, None, PTR, PTR, 1, PTR, PTR, PTR, None, None, 1, 1, PTR, 1, PTR, PTR, 1, PTR, 0,
                                   None) == sg.ERR_INVALID_ARG
    assert L.sg_experts_gated_workspace(None, 4) == 0
    assert L.sg_gated_mlp_workspace(None, None, 4) == 0 and L.sg_gated_mlp_backward_workspace(None, None, 4, 4) == 0


def test_binding_refuses():
    with pytest.raises(sg.ShardGemmError, match="x is None"):
        sg.quantize_mxfp8(None)
    with pytest.raises(sg.ShardGemmError, match="no columns"):
        sg.quantize_mxfp8(torch.tensor(1.0))
    with pytest.raises(sg.ShardGemmError, match="not on a GPU|on cpu"):
        sg.quantize_mxfp8(torch.zeros((2, 32)))
    with pytest.raises(sg.ShardGemmError, match="dtype"):
        sg.dequantize_mxfp8(torch.zeros((2, 32)), torch.zeros((2, 1)))


def test_reference_codes():
    grid = mx.magnitudes()
    assert grid[126] == 448 and grid[1] == 2.0 ** -9 and len(grid) == 127 and (grid[1:] > grid[:-1]).all()
    f8 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(f8, grid)
    x = torch.randn((50, 70), generator=torch.Generator().manual_seed(1)) * 3
    codes, scales = mx.encode(x)
    v = mx.decode(codes, scales)
    step = ref.power(scales.long() - 127).repeat_interleave(32, -1)[:, :70]
    assert ((v - x.double()).abs() <= torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * step)).all()
    again = mx.encode(v)  # the values of a checkpoint are kept exactly
    assert torch.equal(mx.decode(*again), v)
    # torch's own rounding to E4M3 of the scaled values
    b = mx.blocks(x) / ref.power(scales.long() - 127)[..., None]
    assert torch.equal(b.float().to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)[:, :70], codes)


def test_reference_scales():
    for k in (-20, 0, 9):
        m = torch.tensor([448.0 * 2.0 ** k, 448.0 * 2.0 ** k * (1 + 2.0 ** -50), 2.0 ** k], dtype=torch.float64)
        assert mx.exponents(m).tolist() == [k, k + 1, k - 8]
    assert mx.exponents(torch.zeros(1, dtype=torch.float64)).tolist() == [-127]


def test_reference_gradient_is_the_derivative():
    g = torch.Generator().manual_seed(2)
    a, b, d = (torch.randn(200, generator=g, dtype=torch.float64) * 3 for _ in range(3))
    a.requires_grad_(True), b.requires_grad_(True)
    h = ref.silu(a) * b
    da, db = torch.autograd.grad((h * d).sum(), (a, b))
    ga, gb, hh = mx.gated_grad(a.detach(), b.detach(), d)
    assert torch.allclose(ga, da, rtol=1e-12, atol=1e-13) and torch.allclose(gb, db, rtol=1e-12, atol=1e-13)
    assert torch.allclose(hh, h.detach(), rtol=1e-12, atol=0)
    assert math.isclose(float(ref.silu(torch.tensor(0.0))), 0.0)
