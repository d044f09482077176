"""Python binding of libshardgemm: the sharded GEMMs of 1-D tensor parallelism
(all-to-sharded, sharded-to-all, their 4-bit affine variants) and SUMMA's
q-step block accumulation, with all P shards of a layer on one MI355X GPU.

This module only marshals arguments: torch supplies device memory and the
current HIP stream, every step of the computation runs in the library's
kernels.  The entry points mirror include/shardgemm.h one to one:

    shard_linear               sg_shard_linear
    shard_quantized_linear     sg_shard_quantized_linear
    shard_mxfp8_linear         sg_shard_mxfp8_linear
    all_to_sharded             sg_all_to_sharded_ex (sg_all_to_sharded's layouts + a sharded input)
    sharded_to_all             sg_sharded_to_all_ex (+ sg_sharded_to_all_workspace; all-reduce or
                               reduce-scatter output)
    mlp                        sg_mlp (+ sg_mlp_workspace): gate|up with SwiGLU, then down
    all_to_sharded_backward    sg_all_to_sharded_backward (dx = rank-order all_sum, dw)
    sharded_to_all_backward    sg_sharded_to_all_backward (sharded dx, dw)
    summa_matmul               sg_summa_matmul (+ sg_summa_workspace)
    summa_backward             sg_summa_backward (Matmul_ABT_2D / Matmul_ATB_2D)
    shard_experts              sg_shard_experts; Experts.update: sg_experts_update
    shard_mxfp4_experts        sg_shard_mxfp4_experts
    experts_all_to_sharded     sg_experts_all_to_sharded (+ _backward)
    experts_sharded_to_all     sg_experts_sharded_to_all (+ _backward)
    swiglu                     sg_swiglu (+ _backward)
    moe_route                  sg_moe_route (+ _backward): top-k experts and the grouping plan
    moe_combine                sg_moe_combine (+ _backward): the weighted sum over a token's experts
    moe_mlp                    sg_moe_mlp (+ sg_moe_mlp_workspace)
    quantize_mxfp4             sg_quantize_mxfp4; dequantize_mxfp4: sg_dequantize_mxfp4
    quantize_mxfp8             sg_quantize_mxfp8; dequantize_mxfp8: sg_dequantize_mxfp8
    experts_gated              sg_experts_gated (+ _backward): SwiGLU's half of the gated block, its
                               gate|up rows kept in MX FP8 for the backward pass
    gated_mlp                  sg_gated_mlp (+ _backward): the whole block
    adapter_plan               sg_adapter_plan: a step's tokens grouped by adapter
    adapted_all_to_sharded     sg_adapted_all_to_sharded (+ _backward): low-rank adapters beside a layer
    adapted_sharded_to_all     sg_adapted_sharded_to_all (+ _backward)
    Layer.info / Layer.shard   sg_layer_info / sg_layer_copy_shard
    time_next_launch           sg_time_next_launch (profiling)

There is no fallback: if the library is not built, importing works but the
first call raises.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libshardgemm.so")

ALL_TO_SHARDED, SHARDED_TO_ALL = 0, 1
IN_FULL, IN_SHARDED = 0, 1
OUT_FULL, OUT_SHARDED = 0, 1
_MODES = {"all-to-sharded": ALL_TO_SHARDED, "sharded-to-all": SHARDED_TO_ALL}
F32, BF16, F16 = 0, 1, 2
_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_TORCH_DT = {v: k for k, v in _DT.items()}
EPI_NONE, EPI_SWIGLU = 0, 1

OK, ERR_INVALID_ARG, ERR_BAD_MODE, ERR_NOT_DIVISIBLE, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_OOM, ERR_HIP = range(8)


class ShardGemmError(RuntimeError):
    """A non-zero sg_status; `code` holds it, the message is sg_last_error()."""

    def __init__(self, code: int, message: str):
        super().__init__(f"[sg_status {code}] {message}")
        self.code = code


class ShardGemmNotBuilt(RuntimeError):
    pass


_lib = None


def lib():
    """The loaded library (ctypes.CDLL) with every entry point typed."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ShardGemmNotBuilt(
                f"{LIB_PATH} is missing: build it first (python -m sharded_gemm_alltosharded_amd._build)")
        L = C.CDLL(LIB_PATH)
        P, I64, I, SZ = C.c_void_p, C.c_int64, C.c_int, C.c_size_t
        PP = C.POINTER(C.c_void_p)
        sig = {
            "sg_shard_linear": ([P, I, I64, I64, P, I, I, I, P, PP], I),
            "sg_shard_quantized_linear": ([P, P, P, I64, I64, I, I, I, P, I, I, I, P, PP], I),
            "sg_shard_mxfp8_linear": ([P, P, I64, I64, I, P, I, I, I, P, PP], I),
            "sg_all_to_sharded": ([P, P, I64, P, I, I, I, P], I),
            "sg_all_to_sharded_ex": ([P, P, I, I64, P, I, I, I, P], I),
            "sg_sharded_to_all": ([P, P, I64, P, I, P, SZ, P], I),
            "sg_sharded_to_all_ex": ([P, P, I64, P, I, I, P, SZ, P], I),
            "sg_all_to_sharded_backward": ([P, P, P, I64, P, I, P, I, P, SZ, P], I),
            "sg_sharded_to_all_backward": ([P, P, P, I64, P, I, P, I, P, SZ, P], I),
            "sg_layer_backward_workspace": ([P, I64], SZ),
            "sg_summa_backward": ([P, P, P, I, I64, I64, I64, I, P, P, P, SZ, P], I),
            "sg_summa_backward_workspace": ([I, I64, I64, I64, I], SZ),
            "sg_mlp": ([P, P, P, I64, P, I, P, SZ, P], I),
            "sg_mlp_workspace": ([P, P, I64], SZ),
            "sg_mlp_static": ([P, P, P, I64, P, I, P], I),
            "sg_sharded_to_all_workspace": ([P, I64], SZ),
            "sg_summa_matmul": ([P, P, I, I64, I64, I64, I, P, I, I, P, SZ, P], I),
            "sg_summa_workspace": ([I, I64, I64, I], SZ),
            "sg_layer_info": ([P, P, P, P, P, P, P, P], I),
            "sg_layer_copy_shard": ([P, I, I, P, SZ, P], I),
            "sg_layer_free": ([P], None),
            "sg_shard_experts": ([P, I, I64, I64, I64, I, I, I, P, PP], I),
            "sg_shard_mxfp4_experts": ([P, P, I64, I64, I64, I, I, I, P, PP], I),
            "sg_experts_update": ([P, P, P], I),
            "sg_experts_info": ([P, P, P, P, P, P, P, P, P], I),
            "sg_experts_free": ([P], None),
            "sg_experts_all_to_sharded": ([P, P, P, I64, I64, P, P, I, I64, P, I, I, P], I),
            "sg_experts_sharded_to_all": ([P, P, P, P, I64, P, I, P], I),
            "sg_experts_all_to_sharded_backward": ([P, P, I64, I64, P, P, P, I, I64, P, I, P, I, P], I),
            "sg_experts_sharded_to_all_backward": ([P, P, P, P, I64, P, I, P, I, P], I),
            "sg_swiglu": ([P, I, I64, I64, P, P], I),
            "sg_swiglu_backward": ([P, P, I, I64, I64, P, P], I),
            "sg_moe_route": ([P, I64, I, I64, I, I, I, P, P, P, P, P, P, SZ, P], I),
            "sg_moe_route_workspace": ([I64, I, I], SZ),
            "sg_moe_route_backward": ([P, I64, I, I64, I, I, I, P, P, P, P, P], I),
            "sg_moe_combine": ([P, I, I64, P, P, I64, I, I64, P, I, P], I),
            "sg_moe_combine_backward": ([P, P, I, I64, P, P, I64, I, I64, P, P, P], I),
            "sg_moe_mlp": ([P, P, P, I64, I64, P, P, P, P, I, P, I, P, SZ, P], I),
            "sg_moe_mlp_workspace": ([P, P, I64, I], SZ),
            "sg_quantize_mxfp4": ([P, I, I64, I64, I64, P, P, P], I),
            "sg_dequantize_mxfp4": ([P, P, I64, I64, P, I, P], I),
            "sg_quantize_mxfp8": ([P, I, I64, I64, I64, P, P, P], I),
            "sg_dequantize_mxfp8": ([P, P, I64, I64, P, I, P], I),
            "sg_experts_gated": ([P, P, I64, I64, P, P, I, I64, P, P, P, P, SZ, P], I),
            "sg_experts_gated_workspace": ([P, I64], SZ),
            "sg_experts_gated_backward": ([P, P, P, P, P, I64, P, P, P], I),
            "sg_gated_mlp": ([P, P, P, I64, I64, P, P, I, I64, P, I, P, P, P, P, P, SZ, P], I),
            "sg_gated_mlp_workspace": ([P, P, I64], SZ),
            "sg_gated_mlp_backward": ([P, P, P, P, I64, P, P, P, P, P, I, I64, P, I, P, P, I, P, SZ, P], I),
            "sg_gated_mlp_backward_workspace": ([P, P, I64, I64], SZ),
            "sg_adapter_plan_ints": ([I64, I], SZ),
            "sg_adapter_plan": ([P, I64, I, P, P], I),
            "sg_adapted_workspace": ([P, P, I64], SZ),
            "sg_adapted_all_to_sharded": ([P, P, P, P, I64, P, I, I, I, P, SZ, P], I),
            "sg_adapted_sharded_to_all": ([P, P, P, P, I64, P, I, P, SZ, P], I),
            "sg_adapted_backward_workspace": ([P, P, I64], SZ),
            "sg_adapted_all_to_sharded_backward": ([P, P, P, P, P, I64, P, I, P, P, I, P, SZ, P], I),
            "sg_adapted_sharded_to_all_backward": ([P, P, P, P, P, I64, P, I, P, P, I, P, SZ, P], I),
            "sg_time_next_launch": ([P, P], I),
            "sg_last_error": ([], C.c_char_p),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _check(rc: int):
    if rc != OK:
        raise ShardGemmError(rc, lib().sg_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(device=None):
    return C.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _mode(sharding) -> int:
    if isinstance(sharding, int):
        return sharding
    # unknown strings reach the library as an invalid mode, which rejects them
    return _MODES.get(sharding, -1)


def time_next_launch(start: "torch.cuda.Event", stop: "torch.cuda.Event"):
    """Arm two timing events for the next kernel this thread launches
    through the library (sg_time_next_launch): they are recorded at that
    kernel's own start and end."""
    for e in (start, stop):
        if e.cuda_event == 0:  # torch creates events lazily
            e.record()
    _check(lib().sg_time_next_launch(C.c_void_p(start.cuda_event), C.c_void_p(stop.cuda_event)))


_freed_layers: list = []


def _release(given_up: list, free):
    """Release the layers given up.  That waits for the device; those given up while
    this thread captures, whose graph may hold calls on them, stay until it ends."""
    while given_up and not torch.cuda.is_current_stream_capturing():
        try:
            h = given_up.pop()
        except IndexError:  # another thread took the last one since
            return
        free(h)


class Layer:
    """A sharded layer owned by the library (sg_layer*)."""

    def __init__(self, handle: C.c_void_p, device: torch.device):
        _release(_freed_layers, lib().sg_layer_free)
        self._h = handle
        self.device = device
        o, i, m, s, p, d, q = (C.c_int64(), C.c_int64(), C.c_int(), C.c_int(), C.c_int(), C.c_int(), C.c_int())
        _check(lib().sg_layer_info(self._h, C.byref(o), C.byref(i), C.byref(m), C.byref(s), C.byref(p),
                                   C.byref(d), C.byref(q)))
        self.out_dims, self.in_dims = o.value, i.value
        self.mode, self.segments, self.P = m.value, s.value, p.value
        self.dtype = _TORCH_DT[d.value]
        self.quantized = bool(q.value)
        self.mx = q.value == 2  # MX FP8 layer

    @property
    def handle(self):
        return self._h

    def free(self):
        h, self._h = self._h, None
        if h is not None and _lib is not None:
            _freed_layers.append(h)
            _release(_freed_layers, _lib.sg_layer_free)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass

    def shard(self, r: int, what: int = 0) -> torch.Tensor:
        """Copy of rank r's stored tensor: 0 weight, 1 bias, 2 scales, 3 biases."""
        if what == 0:
            if self.mx:
                shape, dt = self._wshape(1), torch.uint8
            elif self.quantized:
                shape, dt = self._wshape(8), torch.int32
            else:
                shape, dt = self._wshape(1), self.dtype
        elif what == 1:
            n = self.out_dims // self.P if self.mode == ALL_TO_SHARDED else self.out_dims
            shape, dt = (n,), self.dtype
        elif self.mx:
            shape, dt = self._wshape(32), torch.uint8
        else:
            shape, dt = self._wshape(64), torch.int16
        out = torch.empty(shape, dtype=dt, device=self.device)
        _check(lib().sg_layer_copy_shard(self._h, r, what, _ptr(out), out.numel() * out.element_size(),
                                         _stream(self.device)))
        return out

    def _wshape(self, per):
        if self.mode == ALL_TO_SHARDED:
            return (self.out_dims // self.P, self.in_dims // per)
        return (self.out_dims, self.in_dims // self.P // per)


def shard_linear(weight: torch.Tensor, sharding, segments: int = 1, P: int = 1, bias=None) -> Layer:
    """Shard a dense (out, in) weight over P ranks (sg_shard_linear)."""
    dt = _DT.get(weight.dtype, -1)
    out_dims, in_dims = weight.shape
    weight = weight.contiguous()
    bias = None if bias is None else bias.contiguous()
    h = C.c_void_p()
    dev = weight.device
    _check(lib().sg_shard_linear(_ptr(weight), dt, out_dims, in_dims, _ptr(bias), _mode(sharding), segments, P,
                                 _stream(dev) if dev.type == "cuda" else None, C.byref(h)))
    return Layer(h, dev if dev.type == "cuda" else torch.device("cuda", torch.cuda.current_device()))


def shard_mxfp8_linear(codes: torch.Tensor, scales: torch.Tensor, sharding, segments: int = 1, P: int = 1,
                       act_dtype=torch.bfloat16, bias=None) -> Layer:
    """Shard an MX FP8 layer (sg_shard_mxfp8_linear).  codes: (out, in) uint8
    E4M3; scales: (out, in/32) uint8 E8M0."""
    out_dims, in_dims = codes.shape
    codes, scales = codes.contiguous(), scales.contiguous()
    bias = None if bias is None else bias.contiguous()
    dev = codes.device
    h = C.c_void_p()
    _check(lib().sg_shard_mxfp8_linear(_ptr(codes), _ptr(scales), out_dims, in_dims, _DT.get(act_dtype, -1),
                                       _ptr(bias), _mode(sharding), segments, P,
                                       _stream(dev) if dev.type == "cuda" else None, C.byref(h)))
    return Layer(h, dev if dev.type == "cuda" else torch.device("cuda", torch.cuda.current_device()))


def shard_quantized_linear(wq: torch.Tensor, scales: torch.Tensor, qbiases: torch.Tensor, in_dims: int, sharding,
                           segments: int = 1, P: int = 1, group_size: int = 64, bits: int = 4,
                           act_dtype=torch.bfloat16, bias=None) -> Layer:
    """Shard a 4-bit affine layer (sg_shard_quantized_linear).  wq: (out, in/8)
    int32 words; scales, qbiases: (out, in/group_size) 16-bit fp16 patterns."""
    out_dims = wq.shape[0]
    wq, scales, qbiases = wq.contiguous(), scales.contiguous(), qbiases.contiguous()
    bias = None if bias is None else bias.contiguous()
    dev = wq.device
    h = C.c_void_p()
    _check(lib().sg_shard_quantized_linear(_ptr(wq), _ptr(scales), _ptr(qbiases), out_dims, in_dims, group_size, bits,
                                           _DT.get(act_dtype, -1), _ptr(bias), _mode(sharding), segments, P,
                                           _stream(dev) if dev.type == "cuda" else None, C.byref(h)))
    return Layer(h, dev if dev.type == "cuda" else torch.device("cuda", torch.cuda.current_device()))


def all_to_sharded(layer: Layer, x: torch.Tensor, gather: bool = False, swiglu: bool = False,
                   out_dtype=None, out: torch.Tensor | None = None, x_sharded: bool = False) -> torch.Tensor:
    """x (B, in) -> (P, B, n/P) sharded, or (B, n) gathered; n = out_dims, or
    out_dims/2 with the fused SwiGLU epilogue.  x_sharded: x is (P, B, in/P),
    all-gathered inside the matmul."""
    B = x.shape[1] if x_sharded else x.shape[0]
    n = layer.out_dims // 2 if swiglu else layer.out_dims
    out_dtype = out_dtype or layer.dtype
    if out is None:
        shape = (B, n) if gather else (layer.P, B, n // layer.P)
        out = torch.empty(shape, dtype=out_dtype, device=x.device)
    _check(lib().sg_all_to_sharded_ex(layer.handle, _ptr(x), IN_SHARDED if x_sharded else IN_FULL, B, _ptr(out),
                                      OUT_FULL if gather else OUT_SHARDED, EPI_SWIGLU if swiglu else EPI_NONE,
                                      _DT.get(out.dtype, -1), _stream(x.device)))
    return out


_workspaces: dict = {}


def workspace(layer: Layer, B: int, device) -> torch.Tensor | None:
    """A workspace shared by calls on one device (no initial contents needed)."""
    need = lib().sg_sharded_to_all_workspace(layer.handle, B)
    if need == 0:
        return None
    key = torch.device(device)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, dtype=torch.uint8, device=key)
        _workspaces[key] = ws
    return ws


def sharded_to_all(layer: Layer, x_partial: torch.Tensor, out_dtype=None, out: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None, scatter: bool = False) -> torch.Tensor:
    """x_partial (P, B, in/P) -> (B, out): the rank partials summed in rank
    order, bias added once; scatter: the reduce-scatter (P, B, out/P)."""
    B = x_partial.shape[1]
    out_dtype = out_dtype or layer.dtype
    if out is None:
        shape = (layer.P, B, layer.out_dims // layer.P) if scatter else (B, layer.out_dims)
        out = torch.empty(shape, dtype=out_dtype, device=x_partial.device)
    if ws is None:
        ws = workspace(layer, B, x_partial.device)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().sg_sharded_to_all_ex(layer.handle, _ptr(x_partial), B, _ptr(out), OUT_SHARDED if scatter else OUT_FULL,
                                      _DT.get(out.dtype, -1), _ptr(ws), nbytes, _stream(x_partial.device)))
    return out


_mlp_workspaces: dict = {}


def mlp_workspace(gate_up: Layer, down: Layer, B: int, device) -> torch.Tensor | None:
    """A workspace for mlp(), shared by calls on one device (None
    when the layers do not form a gate|up, down pair: sg_mlp then says why)."""
    need = int(lib().sg_mlp_workspace(gate_up.handle, down.handle, B))
    if need == 0:
        return None
    key = torch.device(device)
    ws = _mlp_workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, dtype=torch.uint8, device=key)
        _mlp_workspaces[key] = ws
    return ws


def mlp(gate_up: Layer, down: Layer, x: torch.Tensor, out_dtype=None, out: torch.Tensor | None = None,
        ws: torch.Tensor | None = None) -> torch.Tensor:
    """(B, in) -> (B, out): down(silu(x W_gate^T) * (x W_up^T)) through sg_mlp,
    the sharded h kept in the workspace."""
    B = x.shape[0]
    out_dtype = out_dtype or down.dtype
    if out is None:
        out = torch.empty((B, down.out_dims), dtype=out_dtype, device=x.device)
    if ws is None:
        ws = mlp_workspace(gate_up, down, B, x.device)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().sg_mlp(gate_up.handle, down.handle, _ptr(x), B, _ptr(out), _DT.get(out.dtype, -1), _ptr(ws),
                        nbytes, _stream(x.device)))
    return out


MLP_STATIC_SCRATCH_BYTES = 16 << 20  # SG_MLP_STATIC_SCRATCH_BYTES


def mlp_static(gate_up: Layer, down: Layer, x: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
    """sg_mlp_static: mlp() without a workspace, for callers that cannot
    allocate (the library's per-device static scratch holds h).  The caller
    passes the output; this wrapper allocates nothing."""
    _check(lib().sg_mlp_static(gate_up.handle, down.handle, _ptr(x), x.shape[0], _ptr(out), _DT.get(out.dtype, -1),
                               _stream(x.device)))
    return out


def _bwd_ws(layer: Layer, B: int, ws, device):
    """The weight-gradient workspace: "auto" takes sg_layer_backward_workspace
    bytes from torch's caching allocator (stream-ordered), None runs the
    weight gradient on the vector units, or a uint8 device tensor."""
    if isinstance(ws, str):
        n = int(lib().sg_layer_backward_workspace(layer.handle, B))
        ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None
    return ws, (0 if ws is None else ws.numel() * ws.element_size())


def all_to_sharded_backward(layer: Layer, x: torch.Tensor | None, dy: torch.Tensor, need_dx: bool = True,
                            need_dw: bool = True, dx_dtype=None, dw_dtype=torch.float32, ws="auto"):
    """Backward of an all-to-sharded layer (sg_all_to_sharded_backward): dy
    (P, B, out/P) -> (dx (B, in) = the rank-order all_sum of dy[r] W_r,
    dw (P, out/P, in), dw[r] = dy[r]^T x); either may be skipped (None)."""
    B = dy.shape[1]
    dx = torch.empty((B, layer.in_dims), dtype=dx_dtype or layer.dtype, device=dy.device) if need_dx else None
    dw = torch.empty((layer.P, layer.out_dims // layer.P, layer.in_dims), dtype=dw_dtype,
                     device=dy.device) if need_dw else None
    ws, nbytes = _bwd_ws(layer, B, ws if need_dw else None, dy.device)
    _check(lib().sg_all_to_sharded_backward(layer.handle, _ptr(x), _ptr(dy), B, _ptr(dx),
                                            _DT.get(dx.dtype if dx is not None else layer.dtype, -1), _ptr(dw),
                                            _DT.get(dw_dtype, -1), _ptr(ws), nbytes, _stream(dy.device)))
    return dx, dw


def sharded_to_all_backward(layer: Layer, x_partial: torch.Tensor | None, dy: torch.Tensor, need_dx: bool = True,
                            need_dw: bool = True, dx_dtype=None, dw_dtype=torch.float32, ws="auto"):
    """Backward of a sharded-to-all layer (sg_sharded_to_all_backward): dy
    (B, out) -> (dx_partial (P, B, in/P), slice r = dy W_r; dw (P, out, in/P),
    dw[r] = dy^T x_partial[r]); either may be skipped (None)."""
    B = dy.shape[0]
    dx = torch.empty((layer.P, B, layer.in_dims // layer.P), dtype=dx_dtype or layer.dtype,
                     device=dy.device) if need_dx else None
    dw = torch.empty((layer.P, layer.out_dims, layer.in_dims // layer.P), dtype=dw_dtype,
                     device=dy.device) if need_dw else None
    ws, nbytes = _bwd_ws(layer, B, ws if need_dw else None, dy.device)
    _check(lib().sg_sharded_to_all_backward(layer.handle, _ptr(x_partial), _ptr(dy), B, _ptr(dx),
                                            _DT.get(dx.dtype if dx is not None else layer.dtype, -1), _ptr(dw),
                                            _DT.get(dw_dtype, -1), _ptr(ws), nbytes, _stream(dy.device)))
    return dx, dw


def summa_backward(X: torch.Tensor, A: torch.Tensor, dY: torch.Tensor, q: int, need_dx: bool = True,
                   need_da: bool = True, ws="auto"):
    """Gradients of Y = X A in q SUMMA steps (sg_summa_backward): dX = dY A^T
    (M, K) and dA = X^T dY (K, N), both fp32; either may be skipped (None).
    ws: "auto" (sg_summa_backward_workspace bytes from torch's allocator), None
    (dA on the vector units) or a uint8 device tensor."""
    M, K = X.shape
    N = A.shape[1]
    dX = torch.empty((M, K), dtype=torch.float32, device=dY.device) if need_dx else None
    dA = torch.empty((K, N), dtype=torch.float32, device=dY.device) if need_da else None
    if isinstance(ws, str):
        n = int(lib().sg_summa_backward_workspace(_DT.get(X.dtype, -1), M, K, N, q)) if need_da else 0
        ws = torch.empty(n, dtype=torch.uint8, device=dY.device) if n else None
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().sg_summa_backward(_ptr(X), _ptr(A), _ptr(dY), _DT.get(X.dtype, -1), M, K, N, q, _ptr(dX), _ptr(dA),
                                   _ptr(ws), nbytes, _stream(dY.device)))
    return dX, dA


def summa_workspace(dtype: torch.dtype, K: int, N: int, q: int) -> int:
    """Bytes of workspace summa_matmul can use (0: it reads A in place)."""
    return int(lib().sg_summa_workspace(_DT.get(dtype, -1), K, N, q))


def summa_matmul(X: torch.Tensor, A: torch.Tensor, q: int, out: torch.Tensor | None = None,
                 accumulate: bool = False, fused: bool = True, workspace="auto") -> torch.Tensor:
    """Y (M, N) fp32 = X A (or Y += X A) on a q x q block grid.

    workspace: "auto" takes summa_workspace(...) bytes from torch's caching
    allocator for this call (stream-ordered, so the memory is reused only by
    later work on the same stream); None makes the kernels read A in place; or
    a uint8 device tensor of at least that size."""
    M, K = X.shape
    N = A.shape[1]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=X.device)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a tensor")
        need = summa_workspace(X.dtype, K, N, q)
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device) if need else None
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().sg_summa_matmul(_ptr(X), _ptr(A), _DT.get(X.dtype, -1), M, K, N, q, _ptr(out), int(accumulate),
                                 int(fused), ws_ptr, ws_bytes, _stream(X.device)))
    return out


# ---- mixture of experts and MXFP4 -------------------------------------------
# These calls run on the device of their tensors, whatever device is current,
# on that device's current stream; workspaces come from torch's caching
# allocator for each call, so calls on several streams, and captured graphs,
# never share one.

class Route(NamedTuple):
    """A router's choices and the plan that groups its slots by expert (sg_moe_route)."""
    weights: torch.Tensor   # (T, k) fp32
    experts: torch.Tensor   # (T, k) int32, -1: dropped
    offsets: torch.Tensor   # (E + 1) int32
    rows: torch.Tensor      # (T k) int32, -1 behind the last
    slots: torch.Tensor     # (T, k) int32, -1: dropped


def _bad(message: str):
    raise ShardGemmError(ERR_INVALID_ARG, message)


_FLOATS = tuple(_DT)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run(fn, dev: torch.device, *args):
    """fn(*args, stream) on dev's current stream, with dev current.  (These calls
    are short: with the public stream object and an unconditional device guard
    the binding took longer than the kernels of a decoding step.)"""
    i = dev.index
    if torch.cuda.current_device() != i:
        with torch.cuda.device(i):
            return _run(fn, dev, *args)
    rc = fn(*args, _raw_stream(i) if _raw_stream is not None else torch.cuda.current_stream(i).cuda_stream)
    if rc != OK:
        _check(rc)


def _at(t):
    return None if t is None else t.data_ptr()


def _want(t, name: str, shape=None, dtype=None, device=None, optional=False):
    """One tensor argument: packed, of the shape (None: any extent), dtype and device asked for."""
    if t is None:
        if not optional:
            _bad(f"{name} is None")
        return None
    if shape is not None and tuple(t.shape) != shape and (
            t.dim() != len(shape) or any(w is not None and w != h for w, h in zip(shape, t.shape))):
        _bad(f"{name} has shape {tuple(t.shape)}, not {tuple('any' if w is None else w for w in shape)}")
    if dtype is not None and t.dtype is not dtype and t.dtype not in (dtype if isinstance(dtype, tuple) else ()):
        _bad(f"{name} has dtype {t.dtype}")
    if not t.is_cuda:
        _bad(f"{name} is on {t.device}, not on a GPU")
    if device is not None and t.device != device:
        _bad(f"{name} is on {t.device}, not on {device}")
    if not t.is_contiguous():
        _bad(f"{name} is not contiguous")
    return t


def _matrix(t, name: str, width=None, dtype=_FLOATS, device=None):
    """A (rows, width) argument whose rows may be strided: its row stride."""
    if t is None:
        _bad(f"{name} is None")
    if t.dim() != 2 or (width is not None and t.shape[1] != width):
        _bad(f"{name} has shape {tuple(t.shape)}, not (any, {width})")
    if t.dtype is not dtype and t.dtype not in (dtype if isinstance(dtype, tuple) else ()):
        _bad(f"{name} has dtype {t.dtype}")
    if not t.is_cuda or (device is not None and t.device != device):
        _bad(f"{name} is on {t.device}, not on {device or 'a GPU'}")
    rows, cols = t.shape
    if t.is_contiguous():
        return cols
    if cols > 1 and t.stride(1) != 1 or rows > 1 and t.stride(0) < cols:
        _bad(f"{name} has strides {t.stride()}: its columns must be adjacent and its rows apart")
    return t.stride(0) if rows > 1 else cols


def _out(out, name: str, shape, dtype, device):
    if out is None:
        if dtype not in _DT:
            _bad(f"{name} cannot be {dtype}")
        return torch.empty(shape, dtype=dtype, device=device)
    return _want(out, name, shape, _FLOATS, device)


_freed: list = []


def _free_experts():
    _release(_freed, _lib.sg_experts_free)


class Experts:
    """E sharded linear layers owned by the library (sg_experts*)."""

    def __init__(self, handle: C.c_void_p, device: torch.device):
        self._h = handle
        self.device = device
        e, o, i = C.c_int64(), C.c_int64(), C.c_int64()
        m, s, p, d, q = C.c_int(), C.c_int(), C.c_int(), C.c_int(), C.c_int()
        _check(lib().sg_experts_info(handle, C.byref(e), C.byref(o), C.byref(i), C.byref(m), C.byref(s), C.byref(p),
                                     C.byref(d), C.byref(q)))
        self.E, self.out_dims, self.in_dims = e.value, o.value, i.value
        self.mode, self.segments, self.P = m.value, s.value, p.value
        self.dtype = _TORCH_DT[d.value]
        self.mx = bool(q.value)

    @property
    def handle(self):
        if self._h is None:
            _bad("the layer has been freed")
        return self._h

    def update(self, weight: torch.Tensor):
        """New weights (E, out, in) into the layer, on the current stream."""
        _want(weight, "weight", (self.E, self.out_dims, self.in_dims), self.dtype, self.device)
        _run(lib().sg_experts_update, self.device, self.handle, _at(weight))

    def free(self):
        h, self._h = self._h, None
        if h is not None and _lib is not None:
            _freed.append(h)
            _free_experts()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def _experts(make, device) -> Experts:
    device = device if device.type == "cuda" else torch.device("cuda", torch.cuda.current_device())
    h = C.c_void_p()
    with torch.cuda.device(device):
        _check(make(_stream(device), C.byref(h)))
    _free_experts()
    return Experts(h, device)


def shard_experts(weight: torch.Tensor, sharding, segments: int = 1, P: int = 1) -> Experts:
    """Shard E dense weights (E, out, in) over P ranks (sg_shard_experts)."""
    if weight.dim() != 3:
        _bad(f"weight has shape {tuple(weight.shape)}, not (E, out, in)")
    E, o, i = weight.shape
    weight = weight.contiguous()
    return _experts(lambda s, h: lib().sg_shard_experts(_ptr(weight), _DT.get(weight.dtype, -1), E, o, i,
                                                        _mode(sharding), segments, P, s, h), weight.device)


def shard_mxfp4_experts(codes: torch.Tensor, scales: torch.Tensor, sharding, segments: int = 1, P: int = 1) -> Experts:
    """Shard E MXFP4 weights (sg_shard_mxfp4_experts): codes (E, out, in / 2),
    scales (E, out, in / 32) uint8, as quantize_mxfp4 gives them for (E, out, in)."""
    if codes.dim() != 3 or scales.dim() != 3 or codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        _bad("codes and scales must be (E, out, in / 2) and (E, out, in / 32) uint8")
    E, o, half = codes.shape
    if scales.shape != (E, o, half * 2 // 32) or codes.device != scales.device:
        _bad(f"scales has shape {tuple(scales.shape)} for codes of shape {tuple(codes.shape)}")
    codes, scales = codes.contiguous(), scales.contiguous()
    return _experts(lambda s, h: lib().sg_shard_mxfp4_experts(_ptr(codes), _ptr(scales), E, o, half * 2,
                                                              _mode(sharding), segments, P, s, h), codes.device)


def _grouped(layer: Experts, offsets, rows, R, k=1):
    if rows is not None and (k is None or k < 1):
        _bad(f"rows are slots of k choices each: k is {k}")
    _want(offsets, "offsets", (layer.E + 1,), torch.int32, layer.device, optional=layer.E == 1)
    _want(rows, "rows", (R,), torch.int32, layer.device, optional=True)


def experts_all_to_sharded(layer: Experts, x: torch.Tensor, offsets=None, rows=None, k: int | None = None,
                           swiglu: bool = False, x_scales=None, out_dtype=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """x (T, in) -> (P, R, n / P), rows grouped by expert (sg_experts_all_to_sharded);
    n = out_dims, or out_dims / 2 with the SwiGLU epilogue.

    rows: None (R = T, row m is x[m]) or the plan's slots, row m is x[rows[m] // k].
    x_scales: x is MXFP4 codes (T, in / 2) with these scales (T, in / 32)."""
    dev = layer.device
    if x_scales is None:
        ld = _matrix(x, "x", layer.in_dims, layer.dtype, dev)
    else:
        _want(x, "x", (None, layer.in_dims // 2), torch.uint8, dev)
        _want(x_scales, "x_scales", (x.shape[0], layer.in_dims // 32), torch.uint8, dev)
        ld = layer.in_dims
    R = x.shape[0] if rows is None else rows.shape[0]
    _grouped(layer, offsets, rows, R, k)
    n = layer.out_dims // 2 if swiglu else layer.out_dims
    out = _out(out, "out", (layer.P, R, n // layer.P), out_dtype or layer.dtype, dev)
    _run(lib().sg_experts_all_to_sharded, dev, layer.handle, _at(x), _at(x_scales), x.shape[0], ld, _at(offsets),
         _at(rows), k or 1, R, _at(out), EPI_SWIGLU if swiglu else EPI_NONE, _DT[out.dtype])
    return out


def experts_sharded_to_all(layer: Experts, h: torch.Tensor, offsets=None, h_scales=None, out_dtype=None,
                           out: torch.Tensor | None = None) -> torch.Tensor:
    """h (P, R, in / P) -> (R, out): the ranks' partial sums added in rank order
    (sg_experts_sharded_to_all).  h_scales: h is MXFP4 codes (P, R, in / P / 2)."""
    dev, kr = layer.device, layer.in_dims // layer.P
    if h_scales is None:
        _want(h, "h", (layer.P, None, kr), layer.dtype, dev)
    else:
        _want(h, "h", (layer.P, None, kr // 2), torch.uint8, dev)
        _want(h_scales, "h_scales", (layer.P, h.shape[1], kr // 32), torch.uint8, dev)
    R = h.shape[1]
    _grouped(layer, offsets, None, R)
    out = _out(out, "out", (R, layer.out_dims), out_dtype or layer.dtype, dev)
    _run(lib().sg_experts_sharded_to_all, dev, layer.handle, _at(h), _at(h_scales), _at(offsets), R, _at(out),
         _DT[out.dtype])
    return out


def experts_all_to_sharded_backward(layer: Experts, x: torch.Tensor | None, dy: torch.Tensor, offsets=None, rows=None,
                                    k: int | None = None, need_dx: bool = True, need_dw: bool = True, dx_dtype=None,
                                    dw_dtype=torch.float32):
    """dy (P, R, out / P) -> (dx (R, in), one row for every grouped row,
    dw (E, P, out / P, in)); either may be skipped (None)."""
    dev, n = layer.device, layer.out_dims // layer.P
    _want(dy, "dy", (layer.P, None, n), layer.dtype, dev)
    R, T, ld = dy.shape[1], 0, layer.in_dims
    if need_dw:
        ld = _matrix(x, "x", layer.in_dims, layer.dtype, dev)
        T = x.shape[0]
    _grouped(layer, offsets, rows, R, k)
    dx = _out(None, "dx", (R, layer.in_dims), dx_dtype or layer.dtype, dev) if need_dx else None
    dw = _out(None, "dw", (layer.E, layer.P, n, layer.in_dims), dw_dtype, dev) if need_dw else None
    _run(lib().sg_experts_all_to_sharded_backward, dev, layer.handle, _at(x) if need_dw else None, T, ld, _at(dy),
         _at(offsets), _at(rows), k or 1, R, _at(dx), _DT.get(dx_dtype or layer.dtype, -1), _at(dw), _DT.get(dw_dtype, -1))
    return dx, dw


def experts_sharded_to_all_backward(layer: Experts, h: torch.Tensor | None, dy: torch.Tensor, offsets=None,
                                    need_dx: bool = True, need_dw: bool = True, dx_dtype=None,
                                    dw_dtype=torch.float32):
    """dy (R, out) -> (dh (P, R, in / P), dw (E, P, out, in / P)); either may be skipped (None)."""
    dev, kr = layer.device, layer.in_dims // layer.P
    _want(dy, "dy", (None, layer.out_dims), layer.dtype, dev)
    R = dy.shape[0]
    if need_dw:
        _want(h, "h", (layer.P, R, kr), layer.dtype, dev)
    _grouped(layer, offsets, None, R)
    dh = _out(None, "dx", (layer.P, R, kr), dx_dtype or layer.dtype, dev) if need_dx else None
    dw = _out(None, "dw", (layer.E, layer.P, layer.out_dims, kr), dw_dtype, dev) if need_dw else None
    _run(lib().sg_experts_sharded_to_all_backward, dev, layer.handle, _at(h) if need_dw else None, _at(dy),
         _at(offsets), R, _at(dh), _DT.get(dx_dtype or layer.dtype, -1), _at(dw), _DT.get(dw_dtype, -1))
    return dh, dw


def swiglu(gu: torch.Tensor) -> torch.Tensor:
    """(..., 2 f) rows [gate; up] -> (..., f) silu(gate) * up (sg_swiglu)."""
    _want(gu, "gu", None, _FLOATS)
    if gu.dim() < 1 or gu.shape[-1] % 2 or gu.shape[-1] == 0:
        _bad(f"gu has shape {tuple(gu.shape)}: its rows must be [gate; up]")
    f = gu.shape[-1] // 2
    h = torch.empty((*gu.shape[:-1], f), dtype=gu.dtype, device=gu.device)
    _run(lib().sg_swiglu, gu.device, _at(gu), _DT[gu.dtype], gu.numel() // (2 * f), f, _at(h))
    return h


def swiglu_backward(gu: torch.Tensor, dh: torch.Tensor) -> torch.Tensor:
    """Gradient of swiglu: dh (..., f) -> dgu (..., 2 f) (sg_swiglu_backward)."""
    _want(gu, "gu", None, _FLOATS)
    if gu.dim() < 1 or gu.shape[-1] % 2 or gu.shape[-1] == 0:
        _bad(f"gu has shape {tuple(gu.shape)}: its rows must be [gate; up]")
    f = gu.shape[-1] // 2
    _want(dh, "dh", (*gu.shape[:-1], f), gu.dtype, gu.device)
    dgu = torch.empty_like(gu)
    _run(lib().sg_swiglu_backward, gu.device, _at(gu), _at(dh), _DT[gu.dtype], gu.numel() // (2 * f), f, _at(dgu))
    return dgu


def moe_route(logits: torch.Tensor, k: int, normalize: bool = True) -> Route:
    """The k experts of every token and the plan that groups the slots
    (sg_moe_route).  logits (T, E), -inf where an expert is closed to a token."""
    ld = _matrix(logits, "logits")
    T, E = logits.shape
    dev, L = logits.device, lib()
    if not 1 <= k <= E:
        _bad(f"a router needs 1 <= k <= E (got k {k}, E {E})")
    n = T * k
    # one allocation; the workspace (none for few slots) may end it: only this call uses it
    need = L.sg_moe_route_workspace(T, E, k)
    buf = torch.empty((4 * n + E + 1 + need // 4,), dtype=torch.int32, device=dev)
    w, e, rows, slots, offsets, ws = buf.split_with_sizes((n, n, n, n, E + 1, need // 4))
    w, e, slots = w.view(torch.float32).view(T, k), e.view(T, k), slots.view(T, k)
    _run(L.sg_moe_route, dev, _at(logits), ld, _DT[logits.dtype], T, E, k, int(normalize), _at(w), _at(e), _at(offsets),
         _at(rows), _at(slots), _at(ws), need)
    return Route(w, e, offsets, rows, slots)


def moe_route_backward(logits: torch.Tensor, route: Route, dweights: torch.Tensor,
                       normalize: bool = True) -> torch.Tensor:
    """Gradient of the router's weights: dweights (T, k) -> dlogits (T, E) (sg_moe_route_backward)."""
    ld = _matrix(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    k = route.weights.shape[-1]
    _want(route.weights, "weights", (T, k), torch.float32, dev)
    _want(route.experts, "experts", (T, k), torch.int32, dev)
    _want(dweights, "dweights", (T, k), torch.float32, dev)
    dz = torch.empty((T, E), dtype=logits.dtype, device=dev)
    _run(lib().sg_moe_route_backward, dev, _at(logits), ld, _DT[logits.dtype], T, E, k, int(normalize),
         _at(route.weights), _at(route.experts), _at(dweights), _at(dz))
    return dz


def moe_combine(y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None, out_dtype=None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """(R, D) grouped rows -> (T, D): each token's rows, weighted and added
    (sg_moe_combine).  weights None: 1."""
    _want(y, "y", (None, None), _FLOATS)
    dev = y.device
    _want(slots, "slots", (None, None), torch.int32, dev)
    T, k = slots.shape
    _want(weights, "weights", (T, k), torch.float32, dev, optional=True)
    out = _out(out, "out", (T, y.shape[1]), out_dtype or y.dtype, dev)
    _run(lib().sg_moe_combine, dev, _at(y), _DT[y.dtype], y.shape[0], _at(slots), _at(weights), T, k, y.shape[1],
         _at(out), _DT[out.dtype])
    return out


def moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, slots: torch.Tensor,
                         weights: torch.Tensor | None = None, need_dy: bool = True, need_dweights: bool = True,
                         dy: torch.Tensor | None = None):
    """Gradient of moe_combine: dout (T, D) -> (dy (R, D), dweights (T, k));
    either may be skipped (None).  Rows of no slot are left as they were in a
    caller's dy, and are zero in a new one; a row may stand in slots once."""
    _want(dout, "dout", (None, None), _FLOATS)
    dev, (T, D) = dout.device, dout.shape
    _want(y, "y", (None, D), dout.dtype, dev)
    _want(slots, "slots", (T, None), torch.int32, dev)
    k = slots.shape[1]
    _want(weights, "weights", (T, k), torch.float32, dev, optional=True)
    if need_dy:
        dy = torch.zeros_like(y) if dy is None else _want(dy, "dy", tuple(y.shape), y.dtype, dev)
    else:
        dy = None
    dw = torch.empty((T, k), dtype=torch.float32, device=dev) if need_dweights else None
    _run(lib().sg_moe_combine_backward, dev, _at(dout), _at(y), _DT[y.dtype], y.shape[0], _at(slots), _at(weights), T, k,
         D, _at(dy), _at(dw))
    return dy, dw


def moe_mlp(gate_up: Experts, down: Experts, x: torch.Tensor, route: Route, out_dtype=None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """The gated MLP over experts: (T, in) -> (T, out) (sg_moe_mlp)."""
    dev = gate_up.device
    ld = _matrix(x, "x", gate_up.in_dims, gate_up.dtype, dev)
    T, k = x.shape[0], route.slots.shape[-1]
    _want(route.weights, "weights", (T, k), torch.float32, dev)
    _want(route.slots, "slots", (T, k), torch.int32, dev)
    _want(route.rows, "rows", (T * k,), torch.int32, dev)
    _want(route.offsets, "offsets", (gate_up.E + 1,), torch.int32, dev)
    out = _out(out, "out", (T, down.out_dims), out_dtype or down.dtype, dev)
    L = lib()
    need = L.sg_moe_mlp_workspace(gate_up.handle, down.handle, T, k)
    ws = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    _run(L.sg_moe_mlp, dev, gate_up.handle, down.handle, _at(x), T, ld, _at(route.weights), _at(route.offsets),
         _at(route.rows), _at(route.slots), k, _at(out), _DT[out.dtype], _at(ws), need)
    return out


def quantize_mxfp4(x: torch.Tensor):
    """(..., n) values -> MXFP4 codes (..., n / 2) and scales (..., n / 32), uint8 (sg_quantize_mxfp4)."""
    if x is None or x.dim() < 1:
        _bad("x is None" if x is None else "x has no columns")
    n = x.shape[-1]
    if x.dim() == 2:
        ld = _matrix(x, "x")
    else:
        _want(x, "x", None, _FLOATS)
        ld = n
    rows = x.numel() // n if n else 0
    codes = torch.empty((*x.shape[:-1], n // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((*x.shape[:-1], n // 32), dtype=torch.uint8, device=x.device)
    _run(lib().sg_quantize_mxfp4, x.device, _at(x), _DT[x.dtype], rows, n, ld, _at(codes), _at(scales))
    return codes, scales


def dequantize_mxfp4(codes: torch.Tensor, scales: torch.Tensor, out_dtype=torch.float32) -> torch.Tensor:
    """The values that codes (..., n / 2) and scales (..., n / 32) stand for (sg_dequantize_mxfp4)."""
    _want(codes, "codes", None, torch.uint8)
    if codes.dim() < 1:
        _bad("codes has no columns")
    n = codes.shape[-1] * 2
    _want(scales, "scales", (*codes.shape[:-1], n // 32), torch.uint8, codes.device)
    x = _out(None, "out", (*codes.shape[:-1], n), out_dtype, codes.device)
    _run(lib().sg_dequantize_mxfp4, codes.device, _at(codes), _at(scales), x.numel() // n if n else 0, n, _at(x),
         _DT[out_dtype])
    return x


# ---- the gated block on activations kept in 8 bits --------------------------

def quantize_mxfp8(x: torch.Tensor):
    """(..., n) values -> MX FP8 codes (..., n) and scales (..., ceil(n / 32)), uint8 (sg_quantize_mxfp8)."""
    if x is None or x.dim() < 1:
        _bad("x is None" if x is None else "x has no columns")
    n = x.shape[-1]
    if x.dim() == 2:
        ld = _matrix(x, "x")
    else:
        _want(x, "x", None, _FLOATS)
        ld = n
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty((*x.shape[:-1], (n + 31) // 32), dtype=torch.uint8, device=x.device)
    _run(lib().sg_quantize_mxfp8, x.device, _at(x), _DT[x.dtype], x.numel() // n if n else 0, n, ld, _at(codes),
         _at(scales))
    return codes, scales


def dequantize_mxfp8(codes: torch.Tensor, scales: torch.Tensor, out_dtype=torch.float32) -> torch.Tensor:
    """The values that codes (..., n) and scales (..., ceil(n / 32)) stand for (sg_dequantize_mxfp8)."""
    _want(codes, "codes", None, torch.uint8)
    if codes.dim() < 1:
        _bad("codes has no columns")
    n = codes.shape[-1]
    _want(scales, "scales", (*codes.shape[:-1], (n + 31) // 32), torch.uint8, codes.device)
    x = _out(None, "out", tuple(codes.shape), out_dtype, codes.device)
    _run(lib().sg_dequantize_mxfp8, codes.device, _at(codes), _at(scales), x.numel() // n if n else 0, n, _at(x),
         _DT[out_dtype])
    return x


class GatedSaved(NamedTuple):
    """What a gated block keeps for its backward pass, in MX FP8 (sg_gated_mlp)."""
    x_codes: torch.Tensor    # (T, in) uint8
    x_scales: torch.Tensor   # (T, ceil(in / 32)) uint8
    gu_codes: torch.Tensor   # (P, R, 2, f) uint8: the gate rows, the up rows
    gu_scales: torch.Tensor  # (P, R, 2, ceil(f / 32)) uint8


def _scratch(need: int, dev):
    return torch.empty((need,), dtype=torch.uint8, device=dev) if need else None


def _kept(P, R, f, dev):
    return (torch.empty((P, R, 2, f), dtype=torch.uint8, device=dev),
            torch.empty((P, R, 2, (f + 31) // 32), dtype=torch.uint8, device=dev))


def _want_kept(codes, scales, P, R, f, dev):
    _want(codes, "codes", (P, R, 2, f), torch.uint8, dev)
    _want(scales, "scales", (P, R, 2, (f + 31) // 32), torch.uint8, dev)


def experts_gated(layer: Experts, x: torch.Tensor, offsets=None, rows=None, k: int | None = None):
    """x (T, in) -> (h (P, R, f), codes (P, R, 2, f), scales): SwiGLU of the gate|up
    product, and its gate and up rows kept in MX FP8 (sg_experts_gated).  rows, k as
    in experts_all_to_sharded; f = out_dims / 2 / P."""
    dev = layer.device
    ld = _matrix(x, "x", layer.in_dims, layer.dtype, dev)
    R = x.shape[0] if rows is None else rows.shape[0]
    _grouped(layer, offsets, rows, R, k)
    f = layer.out_dims // 2 // layer.P
    h = torch.empty((layer.P, R, f), dtype=layer.dtype, device=dev)
    codes, scales = _kept(layer.P, R, f, dev)
    L = lib()
    need = L.sg_experts_gated_workspace(layer.handle, R)
    ws = _scratch(need, dev)
    _run(L.sg_experts_gated, dev, layer.handle, _at(x), x.shape[0], ld, _at(offsets), _at(rows), k or 1, R, _at(h),
         _at(codes), _at(scales), _at(ws), need)
    return h, codes, scales


def experts_gated_backward(down: Experts, dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, offsets=None,
                           need_h: bool = True):
    """dy (R, out) and the kept gate and up rows -> (dgu (P, R, 2 f), h (P, R, f) or
    None): the gradient of the gate|up rows, and the down layer's input again
    (sg_experts_gated_backward)."""
    dev, f = down.device, down.in_dims // down.P
    _want(dy, "dy", (None, down.out_dims), down.dtype, dev)
    R = dy.shape[0]
    _grouped(down, offsets, None, R)
    _want_kept(codes, scales, down.P, R, f, dev)
    dgu = torch.empty((down.P, R, 2 * f), dtype=down.dtype, device=dev)
    h = torch.empty((down.P, R, f), dtype=down.dtype, device=dev) if need_h else None
    _run(lib().sg_experts_gated_backward, dev, down.handle, _at(dy), _at(codes), _at(scales), _at(offsets), R, _at(dgu),
         _at(h))
    return dgu, h


def gated_mlp(gate_up: Experts, down: Experts, x: torch.Tensor, offsets=None, rows=None, k: int | None = None,
              out_dtype=None, out: torch.Tensor | None = None):
    """The gated block for training: x (T, in) -> (y (R, out), GatedSaved), y[m] =
    down(silu(x W_gate^T) * (x W_up^T)) for every grouped row (sg_gated_mlp).  A dense
    block is one expert: shard_experts(weight[None], ...), offsets None."""
    dev = gate_up.device
    ld = _matrix(x, "x", gate_up.in_dims, gate_up.dtype, dev)
    T = x.shape[0]
    R = T if rows is None else rows.shape[0]
    _grouped(gate_up, offsets, rows, R, k)
    out = _out(out, "out", (R, down.out_dims), out_dtype or down.dtype, dev)
    x_codes = torch.empty((T, gate_up.in_dims), dtype=torch.uint8, device=dev)
    x_scales = torch.empty((T, (gate_up.in_dims + 31) // 32), dtype=torch.uint8, device=dev)
    gu_codes, gu_scales = _kept(gate_up.P, R, gate_up.out_dims // 2 // gate_up.P, dev)
    L = lib()
    need = L.sg_gated_mlp_workspace(gate_up.handle, down.handle, R)
    ws = _scratch(need, dev)
    _run(L.sg_gated_mlp, dev, gate_up.handle, down.handle, _at(x), T, ld, _at(offsets), _at(rows), k or 1, R, _at(out),
         _DT[out.dtype], _at(x_codes), _at(x_scales), _at(gu_codes), _at(gu_scales), _at(ws), need)
    return out, GatedSaved(x_codes, x_scales, gu_codes, gu_scales)


def gated_mlp_backward(gate_up: Experts, down: Experts, saved: GatedSaved, dy: torch.Tensor, offsets=None, rows=None,
                       k: int | None = None, need_dx: bool = True, need_dw: bool = True, dx_dtype=None,
                       dw_dtype=torch.float32):
    """Gradients of gated_mlp from what it kept: dy (R, out) -> (dx (R, in), one row
    for every grouped row, dw_gate_up (E, P, 2 f, in), dw_down (E, P, out, f)); dx, or
    both weights', may be skipped (None) (sg_gated_mlp_backward)."""
    dev = gate_up.device
    _want(dy, "dy", (None, down.out_dims), down.dtype, dev)
    R, f, D = dy.shape[0], gate_up.out_dims // 2 // gate_up.P, gate_up.in_dims
    _grouped(gate_up, offsets, rows, R, k)
    _want(saved.x_codes, "x_codes", (None, D), torch.uint8, dev)
    T = saved.x_codes.shape[0]
    _want(saved.x_scales, "x_scales", (T, (D + 31) // 32), torch.uint8, dev)
    _want_kept(saved.gu_codes, saved.gu_scales, gate_up.P, R, f, dev)
    dx = _out(None, "dx", (R, D), dx_dtype or gate_up.dtype, dev) if need_dx else None
    dwg = _out(None, "dw", (gate_up.E, gate_up.P, 2 * f, D), dw_dtype, dev) if need_dw else None
    dwd = _out(None, "dw", (down.E, down.P, down.out_dims, down.in_dims // down.P), dw_dtype, dev) if need_dw else None
    L = lib()
    need = L.sg_gated_mlp_backward_workspace(gate_up.handle, down.handle, T, R)
    ws = _scratch(need, dev)
    _run(L.sg_gated_mlp_backward, dev, gate_up.handle, down.handle, _at(saved.x_codes), _at(saved.x_scales), T,
         _at(saved.gu_codes), _at(saved.gu_scales), _at(dy), _at(offsets), _at(rows), k or 1, R, _at(dx),
         _DT.get(dx_dtype or gate_up.dtype, -1), _at(dwg), _at(dwd), _DT.get(dw_dtype, -1), _at(ws), need)
    return dx, dwg, dwd


# ---- low-rank adapters beside a shared projection ----------------------------

class Adapters(NamedTuple):
    """n low-rank adapters of one layer: y += scale[a] (x A[a]^T) B[a]^T (sg_adapters)."""
    A: torch.Tensor                    # (n, rank, in_dims) of the layer's dtype
    B: torch.Tensor                    # (n, out_dims, rank)
    scale: torch.Tensor | None = None  # (n,) fp32; None: 1


class AdapterPlan(NamedTuple):
    """A step's tokens grouped by adapter (sg_adapter_plan)."""
    data: torch.Tensor
    T: int
    n: int


class _AdaptersArg(C.Structure):
    _fields_ = [("A", C.c_void_p), ("B", C.c_void_p), ("scale", C.c_void_p), ("n", C.c_int), ("rank", C.c_int)]


def adapter_plan(which: torch.Tensor, n: int) -> AdapterPlan:
    """which (T,) int32, the adapter of each token (0 .. n - 1, anything else: none)
    -> the plan that every layer's calls of the step take."""
    _want(which, "which", (None,), torch.int32)
    T, dev, L = which.shape[0], which.device, lib()
    # (out of range: sg_adapter_plan says so)
    data = torch.empty((max(1, L.sg_adapter_plan_ints(T, n)),), dtype=torch.int32, device=dev)
    _run(L.sg_adapter_plan, dev, _at(which), T, n, _at(data))
    return AdapterPlan(data, T, n)


def _adapters(layer: Layer, ad: Adapters, plan: AdapterPlan, T: int):
    if layer.handle is None:
        _bad("the layer has been freed")
    dev = layer.device
    _want(ad.A, "A", (None, None, layer.in_dims), layer.dtype, dev)
    n, rank = ad.A.shape[0], ad.A.shape[1]
    _want(ad.B, "B", (n, layer.out_dims, rank), layer.dtype, dev)
    _want(ad.scale, "scale", (n,), torch.float32, dev, optional=True)
    if plan.T != T or plan.n != n:
        _bad(f"the plan is of {plan.T} tokens and {plan.n} adapters, the call of {T} and {n}")
    _want(plan.data, "plan", (max(1, lib().sg_adapter_plan_ints(T, n)),), torch.int32, dev)
    return C.byref(_AdaptersArg(_at(ad.A), _at(ad.B), _at(ad.scale), n, rank))


def adapted_all_to_sharded(layer: Layer, x: torch.Tensor, adapters: Adapters, plan: AdapterPlan, gather: bool = False,
                           swiglu: bool = False, out_dtype=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """all_to_sharded with each token's adapter beside the layer: x (T, in) ->
    (P, T, n / P) sharded, or (T, n) gathered (sg_adapted_all_to_sharded)."""
    dev = layer.device
    _want(x, "x", (None, layer.in_dims), layer.dtype, dev)
    T = x.shape[0]
    ad = _adapters(layer, adapters, plan, T)
    n = layer.out_dims // 2 if swiglu else layer.out_dims
    out = _out(out, "out", (T, n) if gather else (layer.P, T, n // layer.P), out_dtype or layer.dtype, dev)
    L = lib()
    need = L.sg_adapted_workspace(layer.handle, ad, T)
    ws = _scratch(need, dev)
    _run(L.sg_adapted_all_to_sharded, dev, layer.handle, ad, _at(plan.data), _at(x), T, _at(out),
         OUT_FULL if gather else OUT_SHARDED, EPI_SWIGLU if swiglu else EPI_NONE, _DT[out.dtype], _at(ws), need)
    return out


def adapted_sharded_to_all(layer: Layer, x_partial: torch.Tensor, adapters: Adapters, plan: AdapterPlan, out_dtype=None,
                           out: torch.Tensor | None = None) -> torch.Tensor:
    """sharded_to_all with each token's adapter beside the layer: x_partial
    (P, T, in / P) -> (T, out) (sg_adapted_sharded_to_all)."""
    dev = layer.device
    _want(x_partial, "x_partial", (layer.P, None, layer.in_dims // layer.P), layer.dtype, dev)
    T = x_partial.shape[1]
    ad = _adapters(layer, adapters, plan, T)
    out = _out(out, "out", (T, layer.out_dims), out_dtype or layer.dtype, dev)
    L = lib()
    need = L.sg_adapted_workspace(layer.handle, ad, T)
    ws = _scratch(need, dev)
    _run(L.sg_adapted_sharded_to_all, dev, layer.handle, ad, _at(plan.data), _at(x_partial), T, _at(out), _DT[out.dtype],
         _at(ws), need)
    return out


def _adapted_backward(fn, layer, x, x_shape, dy, T, adapters, plan, need_dx, need_d, dx_dtype, d_dtype):
    dev = layer.device
    if need_d:
        _want(x, "x", x_shape, layer.dtype, dev)
    ad = _adapters(layer, adapters, plan, T)
    dx = _out(None, "dx", x_shape, dx_dtype or layer.dtype, dev) if need_dx else None
    dA = _out(None, "dA", tuple(adapters.A.shape), d_dtype, dev) if need_d else None
    dB = _out(None, "dB", tuple(adapters.B.shape), d_dtype, dev) if need_d else None
    need = lib().sg_adapted_backward_workspace(layer.handle, ad, T)
    ws = _scratch(need, dev)
    _run(fn, dev, layer.handle, ad, _at(plan.data), _at(x) if need_d else None, _at(dy), T, _at(dx),
         _DT.get(dx_dtype or layer.dtype, -1), _at(dA), _at(dB), _DT.get(d_dtype, -1), _at(ws), need)
    return dx, dA, dB


def adapted_all_to_sharded_backward(layer: Layer, x: torch.Tensor | None, dy: torch.Tensor, adapters: Adapters,
                                    plan: AdapterPlan, need_dx: bool = True, need_d: bool = True, dx_dtype=None,
                                    d_dtype=torch.float32):
    """Gradients of adapted_all_to_sharded (no SwiGLU) with the layer frozen: dy
    (P, T, out / P) -> (dx (T, in), dA, dB); dx, or the adapters', may be skipped (None)."""
    _want(dy, "dy", (layer.P, None, layer.out_dims // layer.P), layer.dtype, layer.device)
    T = dy.shape[1]
    return _adapted_backward(lib().sg_adapted_all_to_sharded_backward, layer, x, (T, layer.in_dims), dy, T, adapters, plan,
                             need_dx, need_d, dx_dtype, d_dtype)


def adapted_sharded_to_all_backward(layer: Layer, x_partial: torch.Tensor | None, dy: torch.Tensor, adapters: Adapters,
                                    plan: AdapterPlan, need_dx: bool = True, need_d: bool = True, dx_dtype=None,
                                    d_dtype=torch.float32):
    """Gradients of adapted_sharded_to_all with the layer frozen: dy (T, out) ->
    (dx (P, T, in / P), dA, dB); dx, or the adapters', may be skipped (None)."""
    _want(dy, "dy", (None, layer.out_dims), layer.dtype, layer.device)
    T = dy.shape[0]
    return _adapted_backward(lib().sg_adapted_sharded_to_all_backward, layer, x_partial,
                             (layer.P, T, layer.in_dims // layer.P), dy, T, adapters, plan, need_dx, need_d, dx_dtype,
                             d_dtype)
