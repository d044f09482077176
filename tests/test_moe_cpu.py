"""The mixture-of-experts and MXFP4 entry points without a GPU: what they refuse
on the host, the binding's checks of its arguments, and the reference forms the
GPU tests go by (pinned by closed forms and differences)."""
import ctypes as C
import math
import os

import pytest
import torch

import moe_ref as ref
import sharded_gemm_alltosharded_amd as sg


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sg.LIB_PATH):
        pytest.skip("library not built")
    return sg.lib()


def err(L):
    return L.sg_last_error().decode()


PTR = C.c_void_p(0x1000)  # never dereferenced: the calls below fail before


def shard(L, E=2, out=64, inn=64, mode=0, segments=1, P=1, weight=PTR, dtype=sg.BF16):
    h = C.c_void_p()
    return L.sg_shard_experts(weight, dtype, E, out, inn, mode, segments, P, None, C.byref(h)), h


@pytest.mark.parametrize("kw,code,text", [
    (dict(mode=2), sg.ERR_BAD_MODE, "not supported"),
    (dict(E=0), sg.ERR_INVALID_ARG, ">= 1"),
    (dict(out=0), sg.ERR_INVALID_ARG, ">= 1"),
    (dict(P=0), sg.ERR_INVALID_ARG, ">= 1"),
    (dict(segments=0), sg.ERR_INVALID_ARG, ">= 1"),
    (dict(out=3, P=2), sg.ERR_NOT_DIVISIBLE, "Cannot shard the output of size 3 across 2 devices."),
    (dict(out=9, segments=2), sg.ERR_NOT_DIVISIBLE, "into 2 segments"),
    (dict(inn=6, mode=1, P=4), sg.ERR_NOT_DIVISIBLE, "input of size 6 across 4"),
    (dict(E=1025), sg.ERR_UNSUPPORTED, "1024 experts"),
    (dict(out=(1 << 24) + 1), sg.ERR_UNSUPPORTED, "2^24"),
    (dict(E=1024, out=1 << 20, inn=1 << 20), sg.ERR_UNSUPPORTED, "64 GiB"),
    (dict(weight=None), sg.ERR_INVALID_ARG, "weight is NULL"),
    (dict(dtype=sg.F32), sg.ERR_UNSUPPORTED, "bf16 or fp16"),
    (dict(dtype=9), sg.ERR_INVALID_ARG, "unknown dtype"),
])
def test_shard_experts_refuses(L, kw, code, text):
    rc, h = shard(L, **kw)
    assert rc == code and text in err(L) and h.value is None


def test_shard_mxfp4_refuses(L):
    h = C.c_void_p()

    def call(E, out, inn, mode, S, P, codes=PTR, scales=PTR):
        return L.sg_shard_mxfp4_experts(codes, scales, E, out, inn, mode, S, P, None, C.byref(h))

    assert call(1, 32, 48, 0, 1, 1) == sg.ERR_NOT_DIVISIBLE and "scale block of 32" in err(L)
    assert call(1, 32, 64, 1, 1, 4) == sg.ERR_NOT_DIVISIBLE and "straddle" in err(L)
    assert call(1, 32, 64, 0, 1, 1, codes=None) == sg.ERR_INVALID_ARG
    assert call(1, 32, 64, 0, 1, 1, scales=None) == sg.ERR_INVALID_ARG
    assert L.sg_shard_mxfp4_experts(PTR, PTR, 1, 32, 64, 0, 1, 1, None, None) == sg.ERR_INVALID_ARG


def test_null_layers_are_refused(L):
    assert L.sg_experts_update(None, PTR, None) == sg.ERR_INVALID_ARG
    assert L.sg_experts_info(None, *[None] * 8) == sg.ERR_INVALID_ARG
    assert L.sg_experts_all_to_sharded(None, PTR, None, 1, 64, PTR, None, 1, 1, PTR, 0, 1, None) == sg.ERR_INVALID_ARG
    assert L.sg_experts_sharded_to_all(None, PTR, None, PTR, 1, PTR, 1, None) == sg.ERR_INVALID_ARG
    assert L.sg_experts_all_to_sharded_backward(None, PTR, 1, 64, PTR, PTR, None, 1, 1, PTR, 1, PTR, 1,
                                                None) == sg.ERR_INVALID_ARG
    assert L.sg_experts_sharded_to_all_backward(None, PTR, PTR, PTR, 1, PTR, 1, PTR, 1, None) == sg.ERR_INVALID_ARG
    assert L.sg_moe_mlp(None, None, PTR, 1, 64, PTR, PTR, PTR, PTR, 1, PTR, 1, PTR, 0, None) == sg.ERR_INVALID_ARG
    assert L.sg_moe_mlp_workspace(None, None, 4, 2) == 0
    L.sg_experts_free(None)


def route(L, T=4, E=8, k=2, ld=None, dtype=sg.F32, logits=PTR, out=PTR, ws=PTR, bytes_=None):
    need = L.sg_moe_route_workspace(T, E, k)
    return L.sg_moe_route(logits, E if ld is None else ld, dtype, T, E, k, 1, out, out, out, out, out, ws,
                          need if bytes_ is None else bytes_, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), sg.ERR_INVALID_ARG), (dict(k=0), sg.ERR_INVALID_ARG), (dict(k=9), sg.ERR_INVALID_ARG),
    (dict(E=0, k=1), sg.ERR_INVALID_ARG), (dict(ld=7), sg.ERR_INVALID_ARG), (dict(dtype=5), sg.ERR_INVALID_ARG),
    (dict(E=1025), sg.ERR_UNSUPPORTED), (dict(E=64, k=17), sg.ERR_UNSUPPORTED), (dict(T=1 << 62), sg.ERR_UNSUPPORTED),
    (dict(T=1 << 30), sg.ERR_UNSUPPORTED), (dict(T=(1 << 25) + 1, k=1), sg.ERR_UNSUPPORTED),
    (dict(logits=None), sg.ERR_INVALID_ARG), (dict(out=None), sg.ERR_INVALID_ARG),
    (dict(T=5000, ws=None), sg.ERR_WORKSPACE), (dict(T=5000, bytes_=4), sg.ERR_WORKSPACE),
])
def test_route_refuses(L, kw, code):
    assert route(L, **kw) == code and err(L)


def test_route_backward_refuses(L):
    def call(T=4, E=8, k=2, ld=8, dtype=sg.F32, normalize=0, logits=PTR, w=PTR, d=PTR):
        return L.sg_moe_route_backward(logits, ld, dtype, T, E, k, normalize, w, PTR, PTR, d, None)

    assert call(k=9) == sg.ERR_INVALID_ARG
    assert call(ld=3) == sg.ERR_INVALID_ARG
    assert call(logits=None) == sg.ERR_INVALID_ARG
    assert call(w=None) == sg.ERR_INVALID_ARG
    assert call(d=None) == sg.ERR_INVALID_ARG
    assert call(T=0) == sg.OK


def test_combine_refuses(L):
    def call(R=8, T=4, k=2, D=16, yt=sg.F32, ot=sg.F32, y=PTR, slots=PTR, out=PTR):
        return L.sg_moe_combine(y, yt, R, slots, None, T, k, D, out, ot, None)

    for kw in (dict(R=-1), dict(T=-1), dict(k=0), dict(D=0), dict(yt=7), dict(ot=7), dict(y=None), dict(slots=None),
               dict(out=None)):
        assert call(**kw) == sg.ERR_INVALID_ARG, kw
    for kw in (dict(k=17), dict(T=1 << 62), dict(T=1 << 25), dict(R=1 << 40),
               dict(D=1 << 62), dict(T=1 << 10, D=1 << 62)):
        assert call(**kw) == sg.ERR_UNSUPPORTED, kw
    assert call(T=0) == sg.OK
    back = lambda dy, dw, y=PTR: L.sg_moe_combine_backward(PTR, y, sg.F32, 8, PTR, None, 4, 2, 16, dy, dw, None)
    assert back(None, None) == sg.ERR_INVALID_ARG
    assert back(None, PTR, y=None) == sg.ERR_INVALID_ARG


def test_swiglu_and_mxfp4_refuse(L):
    assert L.sg_swiglu(PTR, 7, 4, 8, PTR, None) == sg.ERR_INVALID_ARG
    assert L.sg_swiglu(PTR, sg.BF16, -1, 8, PTR, None) == sg.ERR_INVALID_ARG
    assert L.sg_swiglu(PTR, sg.BF16, 4, 0, PTR, None) == sg.ERR_INVALID_ARG
    assert L.sg_swiglu(None, sg.BF16, 4, 8, PTR, None) == sg.ERR_INVALID_ARG
    assert L.sg_swiglu(PTR, sg.BF16, 1 << 40, 1 << 20, PTR, None) == sg.ERR_UNSUPPORTED
    assert L.sg_swiglu_backward(PTR, None, sg.BF16, 4, 8, PTR, None) == sg.ERR_INVALID_ARG
    q = lambda rows=4, cols=64, ld=64, dt=sg.BF16, x=PTR, c=PTR, s=PTR: L.sg_quantize_mxfp4(x, dt, rows, cols, ld, c, s,
                                                                                          None)
    assert q(cols=48) == sg.ERR_NOT_DIVISIBLE
    assert q(ld=32) == sg.ERR_INVALID_ARG
    assert q(dt=3) == sg.ERR_INVALID_ARG
    assert q(rows=-1) == sg.ERR_INVALID_ARG
    assert q(x=None) == sg.ERR_INVALID_ARG and q(c=None) == sg.ERR_INVALID_ARG and q(s=None) == sg.ERR_INVALID_ARG
    assert q(c=C.c_void_p(0x1001)) == sg.ERR_INVALID_ARG
    assert q(rows=1 << 40) == sg.ERR_UNSUPPORTED
    assert q(rows=0) == sg.OK
    d = lambda **k: L.sg_dequantize_mxfp4(k.get("c", PTR), PTR, 4, k.get("cols", 64), k.get("x", PTR), sg.F32, None)
    assert d(cols=40) == sg.ERR_NOT_DIVISIBLE
    assert d(x=C.c_void_p(0x1004)) == sg.ERR_INVALID_ARG
    assert d(x=None) == sg.ERR_INVALID_ARG


def test_binding_refuses_tensors_it_cannot_take():
    with pytest.raises(sg.ShardGemmError, match="not on a GPU"):
        sg.moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(sg.ShardGemmError, match="not on a GPU"):
        sg.quantize_mxfp4(torch.zeros(2, 2, 32))
    with pytest.raises(sg.ShardGemmError, match="not on"):
        sg.quantize_mxfp4(torch.zeros(4, 32))
    with pytest.raises(sg.ShardGemmError, match="dtype"):
        sg.moe_route(torch.zeros(4, 8, dtype=torch.float64), 2)
    with pytest.raises(sg.ShardGemmError, match="shape"):
        sg.moe_route(torch.zeros(8), 2)
    with pytest.raises(sg.ShardGemmError, match="shape"):
        sg.shard_experts(torch.zeros(4, 4), "all-to-sharded")
    with pytest.raises(sg.ShardGemmError, match="uint8"):
        sg.shard_mxfp4_experts(torch.zeros(1, 4, 16), torch.zeros(1, 4, 1), "all-to-sharded")
    with pytest.raises(sg.ShardGemmError, match="GPU"):
        sg.swiglu(torch.zeros(4, 8))
    with pytest.raises(sg.ShardGemmError, match="GPU"):
        sg.moe_combine(torch.zeros(4, 8), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(sg.ShardGemmError, match="dtype"):
        sg.dequantize_mxfp4(torch.zeros(2, 16), torch.zeros(2, 1))


# ---- the reference forms ----------------------------------------------------

def test_reference_route_by_hand():
    z = torch.tensor([[0.0, math.log(3.0), -math.inf], [1.0, 1.0, 1.0], [math.nan, -math.inf, -math.inf]])
    w, e, off, rows, slots = ref.route(z, 2, True)
    assert e.tolist() == [[1, 0], [0, 1], [-1, -1]]
    # (the logits are stored in 32 bits)
    assert torch.allclose(w, torch.tensor([[0.75, 0.25], [0.5, 0.5], [0, 0]]).double(), atol=1e-7)
    assert off.tolist() == [0, 2, 4, 4] and rows.tolist() == [1, 2, 0, 3, -1, -1]
    assert slots.tolist() == [[2, 0], [1, 3], [-1, -1]]
    w, *_ = ref.route(z, 2, False)
    assert torch.allclose(w[1], torch.full((2,), 1 / 3).double())


def test_reference_mxfp4_by_hand():
    x = torch.zeros(1, 32)
    x[0, :8] = torch.tensor([6.0, -0.25, 0.25, 0.75, -2.5, 5.0, 3.5, 0.26])
    codes, scales = ref.encode(x)
    assert scales.tolist() == [[127]]
    assert ref.decode(codes, scales)[0, :8].tolist() == [6.0, -0.0, 0.0, 1.0, -2.0, 4.0, 4.0, 0.5]
    assert codes[0, 0].item() == (8 << 4) + 7
    codes, scales = ref.encode(x * 4)
    assert scales.tolist() == [[129]] and ref.decode(codes, scales)[0, 0] == 24
    assert ref.encode(torch.zeros(1, 32))[1].item() == 0
    assert ref.encode(torch.full((1, 32), 7.9))[1].item() == 127  # 7.9 < 8: above 6 to 6
    assert ref.decode(*ref.encode(torch.full((1, 32), 7.9)))[0, 0] == 6


def test_reference_shard_rows():
    assert ref.shard_rows(12, 2, 3) == [[0, 1, 6, 7], [2, 3, 8, 9], [4, 5, 10, 11]]


def test_a_layer_taken_by_another_thread_is_left_to_it(monkeypatch):
    """Two threads release the layers given up: one may empty the list behind the other's look at it."""
    released = []

    class Lib:
        sg_experts_free = staticmethod(released.append)

    def other_thread():  # between the look and the taking
        if len(sg._freed) == 1:
            sg._freed.pop()
        return False

    monkeypatch.setattr(sg, "_lib", Lib)
    monkeypatch.setattr(sg, "_freed", ["a", "b", "c"])
    monkeypatch.setattr(sg.torch.cuda, "is_current_stream_capturing", other_thread)
    sg._free_experts()
    assert released == ["c", "b"] and not sg._freed


def test_missing_matrices_are_refused(L):
    """None where a (rows, width) tensor belongs, as for every other argument."""
    for call in (lambda: sg.moe_route(None, 2), lambda: sg.quantize_mxfp4(None),
                 lambda: sg._matrix(None, "x", 64)):
        with pytest.raises(sg.ShardGemmError, match="None") as e:
            call()
        assert e.value.code == sg.ERR_INVALID_ARG
