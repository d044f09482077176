"""Calls of the library on the stand-in runtime (host_stub.cpp), one function a test of
test_host_calls_cpu.py, each in a process of its own:

    python host_calls.py STUB LIBRARY FUNCTION
"""
import ctypes as C
import sys

BF16, F16 = 1, 2
COLUMN, ROW = 0, 1
INVALID, UNSUPPORTED, OOM = 1, 4, 6


class Stub(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("launches", "mallocs", "syncs", "device", "largest", "stream_captured",
                                         "other_capture", "ended", "live", "blocks")]


class Adapters(C.Structure):
    _fields_ = [("A", C.c_void_p), ("B", C.c_void_p), ("scale", C.c_void_p), ("n", C.c_int), ("rank", C.c_int)]


def ready(stub, library):
    global S, L, PTR
    S = Stub.in_dll(C.CDLL(stub, mode=C.RTLD_GLOBAL), "stub")
    L = C.CDLL(library)
    L.sg_last_error.restype = C.c_char_p
    # (integers travel as 64 bits: the callee reads as many as it declares)
    for name in ("sg_gated_mlp_workspace", "sg_gated_mlp_backward_workspace", "sg_adapted_workspace",
                 "sg_adapted_backward_workspace", "sg_adapter_plan_ints"):
        getattr(L, name).restype = C.c_size_t
    global memory
    memory = C.create_string_buffer(1 << 22)
    PTR = C.addressof(memory) // 256 * 256 + 256


def wide(args):
    """Integers as 64-bit ones (those that fit 32 bits alike), pointers as they are."""
    return [C.c_int64(a) if isinstance(a, int) else a for a in args]


def call(name, *args):
    return getattr(L, name)(*wide(args))


def error():
    return L.sg_last_error().decode()


def ok(status):
    assert status == 0, (status, error())


def experts(E, out, width, mode, segments, P):
    h = C.c_void_p()
    ok(call("sg_shard_experts", PTR, BF16, E, out, width, mode, segments, P, None, C.byref(h)))
    return h


def linear(out, width, mode, segments=1, P=1, bias=None, dtype=BF16):
    h = C.c_void_p()
    ok(call("sg_shard_linear", PTR, dtype, out, width, bias, mode, segments, P, None, C.byref(h)))
    return h


def block_backward_tokens():
    """A block's backward call refuses every T that its workspace is not sized for."""
    up, down = experts(1, 64, 32, COLUMN, 2, 1), experts(1, 32, 32, ROW, 1, 1)

    def back(T, R, dx, dwg, dwd, ws=PTR, n=1 << 20):
        return call("sg_gated_mlp_backward", up, down, PTR, PTR, T, PTR, PTR, PTR, None, None, 1, R, dx, BF16, dwg, dwd,
                    BF16, ws, n, None)

    before = S.launches
    for T in (-1, -(1 << 40), (1 << 30) + 1, 1 << 62):
        assert call("sg_gated_mlp_backward_workspace", up, down, T, 4) == 0
        for dx, dwg, dwd in ((PTR, None, None), (None, None, PTR), (PTR, None, PTR), (None, PTR, None)):
            for ws, n in ((None, 0), (PTR, 1 << 20)):
                st = back(T, 4, dx, dwg, dwd, ws, n)
                assert st == (INVALID if T < 0 else UNSUPPORTED), (T, st, error())
    assert S.launches == before
    assert back(4, 4, PTR, None, None, None, 0) == 5  # no workspace
    assert S.launches == before
    ok(back(4, 4, PTR, None, None))
    ok(back(0, 4, PTR, None, PTR))
    assert S.launches > before


def adapted(layer, mode, T=16, status=0, n=2, rank=8):
    ad = Adapters(PTR, PTR, None, n, rank)
    ref = C.byref(ad)
    need = call("sg_adapted_workspace", layer, ref, T)
    if mode == COLUMN:
        st = call("sg_adapted_all_to_sharded", layer, ref, PTR, PTR, T, PTR, 1, 0, BF16, PTR, need, None)
    else:
        st = call("sg_adapted_sharded_to_all", layer, ref, PTR, PTR, T, PTR, BF16, PTR, need, None)
    assert st == status, (st, error())


def adapted_backward(layer, mode, T=16, status=0, n=2, rank=8, dx=True):
    ad = Adapters(PTR, PTR, None, n, rank)
    ref = C.byref(ad)
    need = call("sg_adapted_backward_workspace", layer, ref, T)
    name = "sg_adapted_all_to_sharded_backward" if mode == COLUMN else "sg_adapted_sharded_to_all_backward"
    st = call(name, layer, ref, PTR, PTR, PTR, T, PTR if dx else None, BF16, PTR, PTR, BF16, PTR, need, None)
    assert st == status, (st, error())


# out, in, mode, P: stored row-major, and in fragments that are not the tiles'
COPIED = [(40, 72, COLUMN, 1), (48, 96, COLUMN, 2), (80, 32, ROW, 1)]


def first_adapted_call_beside_a_capture():
    """The copy of a layer's weights is built without ending a capture of another thread."""
    for out, width, mode, P in COPIED:
        for f in (adapted, adapted_backward):
            layer = linear(out, width, mode, P=P)
            mallocs = S.mallocs
            S.other_capture = 1
            f(layer, mode)
            S.other_capture = 0
            assert S.ended == 0 and S.mallocs > mallocs, (out, width, mode, P)
            mallocs = S.mallocs
            f(layer, mode)  # it is there
            assert S.mallocs == mallocs
    layer = linear(*COPIED[0][:2], COLUMN)
    mallocs, launches = S.mallocs, S.launches
    S.stream_captured = 1  # the call's own stream: nothing is built, the layer's own kernels run
    adapted(layer, COLUMN)
    assert S.ended == 0 and S.mallocs == mallocs and S.launches > launches


def backward(layer, mode, B=4):
    name = "sg_all_to_sharded_backward" if mode == COLUMN else "sg_sharded_to_all_backward"
    ok(call(name, layer, None, PTR, B, PTR, BF16, None, BF16, None, 0, None))


def first_backward_call_beside_a_capture():
    """The transposed copy, too; a call captured before it is there builds none."""
    for mode in (COLUMN, ROW):
        for f in (backward, lambda x, m: adapted_backward(x, m, T=4)):
            for out, width in ((64, 64), (64, 80)):  # stored in fragments and row-major
                layer = linear(out, width, mode)
                S.stream_captured, mallocs, launches = 1, S.mallocs, S.launches
                f(layer, mode)
                assert S.ended == 0 and S.mallocs == mallocs and S.launches > launches
                S.stream_captured, S.other_capture = 0, 1
                f(layer, mode)
                assert S.ended == 0 and S.mallocs > mallocs
                S.stream_captured, S.other_capture, mallocs = 1, 0, S.mallocs
                f(layer, mode)  # it is there
                S.stream_captured = 0
                assert S.ended == 0 and S.mallocs == mallocs


def no_memory_for_a_copy():
    """Without memory for the copy of its weights (or for the way there) a layer's own kernels run."""
    for out, width, mode, P in COPIED:
        weights = out * width * 2
        for f in (adapted, lambda x, m: adapted_backward(x, m, T=16)):
            for largest in (0, weights):  # (the copy is padded: larger)
                layer = linear(out, width, mode, P=P)
                live, launches = S.live, S.launches
                S.largest = largest
                f(layer, mode)
                f(layer, mode)  # (the failure is not found again by a launch)
                S.largest = 1 << 60
                assert S.live == live and S.launches > launches
                f(layer, mode)
                assert S.live == live + 1, (S.live, live)


def adapted_calls_on_another_device():
    """Refused, as the expert calls are: what they build and launch would lie on the wrong one."""
    for mode in (COLUMN, ROW):
        layer = linear(40, 72, mode)
        mallocs, launches = S.mallocs, S.launches
        for T in (0, 1, 16):
            for f in (adapted, adapted_backward):
                S.device = 1
                f(layer, mode, T=T, status=INVALID)
                assert "device 0" in error() and "device is 1" in error()
        assert S.mallocs == mallocs and S.launches == launches
        S.device = 0
        adapted(layer, mode)


def projections_that_cannot_be_launched():
    """What the projection's own call refuses is refused before anything is launched."""
    T = 1 << 25
    row = linear(200, 35, ROW, bias=PTR)  # (biases: the layer's own kernels)
    column = linear(200, 35, COLUMN, bias=PTR)
    for layer, mode in ((row, ROW), (column, COLUMN)):
        ad = Adapters(PTR, PTR, None, 1, 8)
        ref = C.byref(ad)
        launches, huge = S.launches, 1 << 60
        name = "sg_adapted_all_to_sharded" if mode == COLUMN else "sg_adapted_sharded_to_all"
        tail = (1, 0, BF16) if mode == COLUMN else (BF16,)
        assert call(name, layer, ref, PTR, PTR, T, PTR, *tail, PTR, huge, None) != 0
        assert S.launches == launches, (mode, "forward")
        for d in (PTR, None):
            assert call(name + "_backward", layer, ref, PTR, PTR, PTR, T, PTR, BF16, d, d, BF16, PTR, huge, None) != 0
            assert S.launches == launches, (mode, "backward")


def quantized(out, width, mode, P, bits, dtype=BF16):
    h = C.c_void_p()
    if bits == 8:
        ok(call("sg_shard_mxfp8_linear", PTR, PTR, out, width, dtype, None, mode, 1, P, None, C.byref(h)))
    else:
        ok(call("sg_shard_quantized_linear", PTR, PTR, PTR, out, width, 64, 4, dtype, None, mode, 1, P, None, C.byref(h)))
    return h


def workspace_of_decoded_weights():
    """MX FP8 weights become one 16-bit matrix, 4-bit ones two: the workspace holds no more."""
    T, n, rank = 22, 2, 8
    ad = Adapters(PTR, PTR, None, n, rank)
    for out, width, mode, P in ((416, 448, COLUMN, 1), (208, 896, ROW, 2)):
        ranks = P if mode == ROW else 1
        one = ranks * ((out + 15) // 16) * ((width // ranks + 63) // 64 * 2) * 1024
        for bits, matrices in ((8, 1), (4, 2)):
            layer = quantized(out, width, mode, P, bits)
            need = call("sg_adapted_workspace", layer, C.byref(ad), T)
            # beside them: x A^T in up to sixteen slabs of 16 floats a token, its operands and exponents
            rest = 16 * T * 16 * 4 + 32 * 64 + T * 4 + 4 * 256
            assert matrices * one <= need <= matrices * one + rest, (bits, need, one)
            adapted(layer, mode, T=T)


def input_gradients_beside_a_bias():
    """No bias enters dx: it takes the same kernels, and no transposed copy, as without one."""
    for mode, P in ((COLUMN, 1), (COLUMN, 2), (ROW, 1)):
        seen = []
        for bias in (None, PTR):
            layer = linear(64, 128, mode, P=P, bias=bias)
            mallocs, launches = S.mallocs, S.launches
            adapted_backward(layer, mode, T=16)
            seen.append((S.mallocs - mallocs, S.launches - launches, S.blocks))
            adapted(layer, mode, T=16)
        assert seen[0] == seen[1] and seen[0][0] == 0, seen


def layers_given_up_beside_a_capture():
    """A layer's release, its copies' too, does not end a capture of another thread."""
    live = S.live
    for make in (lambda: linear(48, 96, COLUMN, P=2, bias=PTR), lambda: linear(48, 96, COLUMN, P=2),
                 lambda: quantized(64, 256, ROW, 1, 4), lambda: quantized(64, 256, ROW, 1, 8)):
        layer = make()
        if S.live == live + 1:  # the dense one without a bias: its copies
            adapted(layer, COLUMN)
        S.other_capture = 1
        call("sg_layer_free", layer)
        S.other_capture = 0
        assert S.ended == 0 and S.live == live
    layer = linear(48, 96, COLUMN)
    S.device = 1
    call("sg_layer_free", layer)
    assert S.device == 1 and S.live == live
    call("sg_layer_free", None)


def weight_gradient_tiles():
    """Tiles of 256 x 256 from four times round the chip's 256 compute units on, and from
    three where an expert has many rows; else of 128 x 128."""
    for E, O, I, times in ((64, 1024, 768, 3), (8, 2560, 2560, 3.125), (1, 4096, 14336, 3.5), (16, 1792, 1792, 3.0625),
                           (16, 2048, 2048, 4), (8, 2048, 2048, 2)):
        layer = experts(E, O, I, COLUMN, 1, 1)

        def blocks(n):  # of an expert's tiles, in eights
            return E * ((-(-O // n) * -(-I // n) + 7) // 8 * 8)

        for m in (1, 32, 512, 2047, 2048, 4096):
            R = m * E
            if R * max(O, I) * 2 >= 0xffff0000:
                continue
            ok(call("sg_experts_all_to_sharded_backward", layer, PTR, R, I, PTR, PTR, None, 1, R, None, BF16, PTR, BF16,
                    None))
            wide = times >= 4 or (times >= 3 and m >= 2048)
            assert S.blocks == blocks(256 if wide else 128), (E, O, I, m, S.blocks)


if __name__ == "__main__":
    ready(*sys.argv[1:3])
    globals()[sys.argv[3]]()
    print("ok")
