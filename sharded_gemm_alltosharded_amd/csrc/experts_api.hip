// C-ABI entry points of the mixture of experts, of MXFP4 and of the gated block on
// activations kept in MX FP8: validation, the expert layers, and what each call
// hands to the grouped kernels.  Every check runs on the host before any device work.
#include <stdarg.h>
#include <stdio.h>

#include <new>

#include "gated.h"

struct sg_experts {
    sg::ExpertsLayout l;
    sg_dtype dtype;
    int mx;
    uint8_t* w;
    uint8_t* wsc;
    int device;
    int64_t w_expert() const { return l.blocks * l.steps * 1024; }
    int64_t wsc_expert() const { return l.blocks * sg::mx4_scale_runs(l.steps) * 256; }
};

namespace {

sg_status fail(sg_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    sg::last_error() = buf;
    return st;
}

sg_status launched(hipError_t e, const char* what) {
    if (e == hipSuccess) return SG_OK;
    if (e == hipErrorInvalidConfiguration)
        return fail(SG_ERR_UNSUPPORTED, "%s: more workgroups than one launch may have", what);
    return fail(e == hipErrorOutOfMemory ? SG_ERR_OOM : SG_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool is16(int dt) { return dt == SG_BF16 || dt == SG_F16; }
bool known(int dt) { return dt == SG_F32 || is16(dt); }
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxTokens = (int64_t)1 << 25;  // of a router's launch, a wave each
constexpr int64_t kMaxBytes = 0xffff0000;  // what a 32-bit buffer offset reaches

// device memory as it is, host memory through a copy that `tmp` then owns
sg_status on_device(const void* src, size_t bytes, hipStream_t s, const void** out, void** tmp) {
    hipPointerAttribute_t at;
    *out = src;
    if (hipPointerGetAttributes(&at, src) == hipSuccess &&
        (at.type == hipMemoryTypeDevice || at.type == hipMemoryTypeManaged))
        return SG_OK;
    (void)hipGetLastError();
    hipError_t e = hipMalloc(tmp, bytes);
    if (e == hipSuccess) e = hipMemcpyAsync(*tmp, src, bytes, hipMemcpyDefault, s);
    *out = *tmp;
    return launched(e, "weight copy");
}

sg_status layout_of(int64_t E, int64_t out_dims, int64_t in_dims, int mode, int segments, int P, bool mx,
                    sg::ExpertsLayout* l) {
    if (mode != SG_ALL_TO_SHARDED && mode != SG_SHARDED_TO_ALL)
        return fail(SG_ERR_BAD_MODE,
                    "Sharding type %d not supported, choose one of 'all-to-sharded' or 'sharded-to-all'", mode);
    if (segments < 1 || P < 1) return fail(SG_ERR_INVALID_ARG, "segments and P must be >= 1");
    if (E < 1 || out_dims < 1 || in_dims < 1) return fail(SG_ERR_INVALID_ARG, "layer dimensions must be >= 1");
    if (E > sg::kRouteMaxExperts || out_dims > (1 << 24) || in_dims > (1 << 24))
        return fail(SG_ERR_UNSUPPORTED, "more than %d experts, or dimensions above 2^24, are not supported",
                    sg::kRouteMaxExperts);
    const bool col = mode == SG_ALL_TO_SHARDED;
    const int64_t dim = col ? out_dims : in_dims;
    if (dim % segments)
        return fail(SG_ERR_NOT_DIVISIBLE, "Cannot split the %s of size %lld into %d segments.",
                    col ? "output" : "input", (long long)dim, segments);
    if (dim / segments % P)
        return fail(SG_ERR_NOT_DIVISIBLE, "Cannot shard the %s of size %lld across %d devices.",
                    col ? "output" : "input", (long long)dim, P);
    if (mx && in_dims % 32)
        return fail(SG_ERR_NOT_DIVISIBLE, "in_dims %lld is not a multiple of the scale block of 32", (long long)in_dims);
    if (mx && !col && (in_dims / segments / P) % 32)
        return fail(SG_ERR_NOT_DIVISIBLE,
                    "Cannot shard the input of size %lld across %d devices: a scale block of 32 would straddle two "
                    "ranks.", (long long)in_dims, P);
    l->mode = mode;
    l->S = segments;
    l->P = P;
    l->E = E;
    l->out = out_dims;
    l->in = in_dims;
    l->f = col ? out_dims / segments / P : out_dims;
    l->bps = up(l->f, 16) / 16;
    l->blocks = col ? l->bps * segments * P : l->bps;
    l->kl = col ? in_dims : in_dims / P;
    l->kpad = up(l->kl, mx ? 128 : 64);
    l->steps = (col ? 1 : P) * l->kpad / (mx ? 128 : 32);
    if (E * l->blocks * l->steps >= sg::kMaxBlocks * 4)
        return fail(SG_ERR_UNSUPPORTED, "an expert layer above 64 GiB is not supported");
    if (l->blocks * l->steps * 1024 > kMaxBytes)
        return fail(SG_ERR_UNSUPPORTED, "an expert above 4 GiB is not supported");
    return SG_OK;
}

sg_status pack(sg_experts* x, const void* weight, const uint8_t* codes, const uint8_t* scales, hipStream_t hs) {
    const size_t n = (size_t)(x->l.E * x->l.out * x->l.in);
    const void *a = nullptr, *b = nullptr;
    void *ta = nullptr, *tb = nullptr;
    sg_status st;
    if (x->mx) {
        st = on_device(codes, n / 2, hs, &a, &ta);
        if (!st) st = on_device(scales, n / 32, hs, &b, &tb);
        if (!st) st = launched(sg::experts_pack_mx4(x->w, x->wsc, (const uint8_t*)a, (const uint8_t*)b, x->l, hs),
                               "weight layout");
    } else {
        st = on_device(weight, n * 2, hs, &a, &ta);
        if (!st) st = launched(sg::experts_pack(x->w, a, x->l, hs), "weight layout");
    }
    if (ta || tb) {
        (void)hipStreamSynchronize(hs);
        if (ta) (void)hipFree(ta);
        if (tb) (void)hipFree(tb);
    }
    return st;
}

sg_status build(const sg::ExpertsLayout& l, sg_dtype dtype, bool mx, const void* weight, const uint8_t* codes,
                const uint8_t* scales, void* stream, sg_experts** out) {
    sg_experts* x = new (std::nothrow) sg_experts{};
    if (!x) return fail(SG_ERR_OOM, "out of host memory");
    x->l = l;
    x->dtype = dtype;
    x->mx = mx;
    (void)hipGetDevice(&x->device);
    hipError_t e = hipMalloc((void**)&x->w, (size_t)(l.E * x->w_expert()));
    if (e == hipSuccess && mx) e = hipMalloc((void**)&x->wsc, (size_t)(l.E * x->wsc_expert()));
    sg_status st = launched(e, "weight allocation");
    if (!st) st = pack(x, weight, codes, scales, (hipStream_t)stream);
    if (!st) st = launched(hipStreamSynchronize((hipStream_t)stream), "weight layout");
    if (st) {
        const std::string msg = sg::last_error();
        sg_experts_free(x);
        sg::last_error() = msg;
        return st;
    }
    *out = x;
    return SG_OK;
}

sg_status check_layer(const sg_experts* x, int mode, const char* what) {
    if (!x) return fail(SG_ERR_INVALID_ARG, "layer is NULL");
    if (x->l.mode != mode)
        return fail(SG_ERR_BAD_MODE, "%s needs an %s layer", what,
                    mode == SG_ALL_TO_SHARDED ? "all-to-sharded" : "sharded-to-all");
    int d = -1;
    if (hipGetDevice(&d) != hipSuccess || d != x->device) {
        (void)hipGetLastError();
        return fail(SG_ERR_INVALID_ARG, "the layer lives on device %d, the current device is %d", x->device, d);
    }
    return SG_OK;
}

// the rows of a grouped call
sg_status check_rows(const sg_experts* x, const int32_t* offsets, int64_t R) {
    if (R < 0) return fail(SG_ERR_INVALID_ARG, "R must be >= 0");
    if (R > kMaxRows) return fail(SG_ERR_UNSUPPORTED, "more than 2^30 rows are not supported");
    if (!offsets && x->l.E != 1) return fail(SG_ERR_INVALID_ARG, "offsets is NULL for a layer of %lld experts",
                                             (long long)x->l.E);
    return SG_OK;
}

sg_status check_tokens(int64_t T) {
    if (T < 0) return fail(SG_ERR_INVALID_ARG, "T must be >= 0");
    if (T > kMaxRows) return fail(SG_ERR_UNSUPPORTED, "more than 2^30 tokens are not supported");
    return SG_OK;
}

sg_status check_gather(int64_t T, int64_t ldx, int64_t width, const int32_t* rows, int k, int64_t R) {
    if (sg_status st = check_tokens(T)) return st;
    if (k < 1) return fail(SG_ERR_INVALID_ARG, "k must be >= 1");
    if (ldx < width) return fail(SG_ERR_INVALID_ARG, "row stride %lld of x is below its width %lld", (long long)ldx,
                                 (long long)width);
    if (!rows && R > T) return fail(SG_ERR_INVALID_ARG, "%lld rows of %lld tokens need a row map", (long long)R,
                                    (long long)T);
    return SG_OK;
}

sg_status check_bytes(int64_t rows, int64_t ld, int64_t bytes2) {
    if ((double)rows * (double)ld * (double)bytes2 / 2 > (double)kMaxBytes)
        return fail(SG_ERR_UNSUPPORTED, "an activation slice above 4 GiB is not supported");
    return SG_OK;
}

void set_weights(sg::Grouped& p, const sg_experts* x) {
    p.W = x->w;
    p.w_expert = x->w_expert();
    p.wsc = x->wsc;
    p.wsc_expert = x->wsc_expert();
    p.wsteps = (int)x->l.steps;
    p.E = (int)x->l.E;
}

int mode_of(const sg_experts* x, const uint8_t* a_scales) {
    return x->mx ? (a_scales ? sg::G_MX4A4 : sg::G_MX4) : x->dtype == SG_F16 ? sg::G_F16 : sg::G_BF16;
}

void set_out(sg::Grouped& p, void* y, sg_dtype dt) {
    p.out = y;
    p.out_dtype = dt;
}

// x (T, in) -> ranks' columns; ldh: columns of a rank's output row that are
// stored (the layer's own, and zeros behind them: products with its zero-padded
// rows would be NaN there for an infinite x)
sg::Grouped column(const sg_experts* x, const void* a, const uint8_t* a_scales, int64_t T, int64_t ldx,
                   const int32_t* offsets, const int32_t* rows, int k, int64_t R, void* y, int swiglu, int64_t ldh,
                   sg_dtype dt) {
    sg::Grouped p{};
    p.mode = mode_of(x, a_scales);
    p.A = a;
    p.a_scales = a_scales;
    p.lda = ldx;
    p.a_pieces = 1;
    p.nseg = 1;
    p.kl = (int)x->l.kl;
    p.kpad = (int)x->l.kpad;
    p.offsets = offsets;
    p.rows = rows;
    p.kdiv = rows ? k : 1;
    p.T = (int)T;
    p.R = (int)R;
    set_weights(p, x);
    p.swiglu = swiglu;
    p.bps = (int)x->l.bps;
    p.f = (int)(swiglu ? ldh : x->l.f);
    p.pad = (int)(p.f - x->l.f);
    p.S = swiglu ? 1 : x->l.S;
    p.nout = (int)(swiglu ? x->l.bps * x->l.P : x->l.blocks);
    p.ldo = swiglu ? ldh : x->l.f * x->l.S;
    p.o_rank = R * p.ldo;
    set_out(p, y, dt);
    return p;
}

// h (P, R, ldh) -> the rank-order sum (R, out)
sg::Grouped row(const sg_experts* x, const void* h, const uint8_t* h_scales, int64_t ldh, const int32_t* offsets,
                int64_t R, void* y, sg_dtype dt) {
    sg::Grouped p{};
    p.mode = mode_of(x, h_scales);
    p.A = h;
    p.a_scales = h_scales;
    p.lda = ldh;
    p.a_rank = R * ldh;
    p.a_pieces = 1;
    p.nseg = x->l.P;
    p.kl = (int)ldh;
    p.kpad = (int)x->l.kpad;
    p.offsets = offsets;
    p.kdiv = 1;
    p.T = p.R = (int)R;
    set_weights(p, x);
    p.bps = (int)x->l.bps;
    p.f = (int)x->l.f;
    p.S = 1;
    p.nout = (int)x->l.blocks;
    p.ldo = x->l.f;
    set_out(p, y, dt);
    return p;
}

// dh_r = dy W_r of a sharded-to-all layer
sg::Grouped row_dx(const sg_experts* x, const void* dy, const int32_t* offsets, int64_t R, void* dh,
                          sg_dtype dh_dtype) {
    const sg::ExpertsLayout& l = x->l;
    sg::Grouped p{};
    p.mode = mode_of(x, nullptr);
    p.A = dy;
    p.lda = l.out;
    p.a_pieces = p.nseg = 1;
    p.kl = (int)l.out;
    p.kpad = (int)(l.bps * 16);
    p.offsets = offsets;
    p.kdiv = 1;
    p.T = p.R = (int)R;
    set_weights(p, x);
    p.transposed = 1;
    p.bps = (int)(l.kpad / 16);
    p.f = (int)l.kl;
    p.S = 1;
    p.nout = p.bps * l.P;
    p.ldo = l.kl;
    p.o_rank = R * l.kl;
    set_out(p, dh, dh_dtype);
    return p;
}

// dx = the ranks' sum of dy_r W_r of an all-to-sharded layer; dy (P, R, S, fp), each
// piece's columns behind the layer's f zeros
sg::Grouped column_dx(const sg_experts* x, const void* dy, int64_t fp, const int32_t* offsets, int64_t R, void* dx,
                      sg_dtype dx_dtype) {
    const sg::ExpertsLayout& l = x->l;
    sg::Grouped p{};
    p.mode = mode_of(x, nullptr);
    p.A = dy;
    p.lda = fp * l.S;
    p.a_rank = R * fp * l.S;
    p.a_pieces = l.S;
    p.nseg = l.P * l.S;
    p.kl = (int)fp;
    p.kpad = (int)(l.bps * 16);
    p.offsets = offsets;
    p.kdiv = 1;
    p.T = p.R = (int)R;
    set_weights(p, x);
    p.transposed = 1;
    p.nout = p.bps = (int)(l.steps * 2);
    p.f = (int)l.in;
    p.S = 1;
    p.ldo = l.in;
    set_out(p, dx, dx_dtype);
    return p;
}

// the weight gradients of the two layers
sg::GroupedDw column_dw(const sg_experts* x, const void* a, int64_t T, int64_t ldx, const void* dy, const int32_t* offsets,
                        const int32_t* rows, int k, int64_t R, void* dw, sg_dtype dw_dtype) {
    const sg::ExpertsLayout& l = x->l;
    const int64_t n = l.f * l.S;  // columns of a rank
    sg::GroupedDw p{};
    p.f16 = x->dtype == SG_F16;
    p.G = dy;
    p.ldg = n;
    p.g_rank = R * n;
    p.X = a;
    p.ldx = ldx;
    p.offsets = offsets;
    p.rows = rows;
    p.kdiv = rows ? k : 1;
    p.T = (int)T;
    p.R = (int)R;
    p.E = (int)l.E;
    p.P = l.P;
    p.O = (int)n;
    p.I = (int)l.in;
    p.out = dw;
    p.out_dtype = dw_dtype;
    return p;
}
sg::GroupedDw row_dw(const sg_experts* x, const void* h, const void* dy, const int32_t* offsets, int64_t R, void* dw,
                     sg_dtype dw_dtype) {
    const sg::ExpertsLayout& l = x->l;
    sg::GroupedDw p{};
    p.f16 = x->dtype == SG_F16;
    p.G = dy;
    p.ldg = l.out;
    p.X = h;
    p.ldx = l.kl;
    p.x_rank = R * l.kl;
    p.offsets = offsets;
    p.kdiv = 1;
    p.T = p.R = (int)R;
    p.E = (int)l.E;
    p.P = l.P;
    p.O = (int)l.out;
    p.I = (int)l.kl;
    p.out = dw;
    p.out_dtype = dw_dtype;
    return p;
}

// activations of a call on an MXFP4 layer
sg_status check_acts(const sg_experts* x, const void* a, const uint8_t* scales, int64_t ldx) {
    if (scales && !x->mx) return fail(SG_ERR_INVALID_ARG, "MXFP4 activations need an MXFP4 layer");
    if (scales && (ldx != x->l.kl || !aligned(a, 16)))
        return fail(SG_ERR_INVALID_ARG, "MXFP4 activations must be packed rows, 16-byte aligned");
    return SG_OK;
}

int64_t h_stride(const sg_experts* gate_up) { return up(gate_up->l.f, 8); }

sg_status check_pair(const sg_experts* g, const sg_experts* d) {
    if (!g || !d) return fail(SG_ERR_INVALID_ARG, "layer is NULL");
    if (g->l.mode != SG_ALL_TO_SHARDED || g->l.S != 2)
        return fail(SG_ERR_INVALID_ARG, "gate_up must be an all-to-sharded layer with segments = 2");
    if (d->l.mode != SG_SHARDED_TO_ALL || d->l.S != 1)
        return fail(SG_ERR_INVALID_ARG, "down must be a sharded-to-all layer with segments = 1");
    if (g->l.P != d->l.P || g->l.E != d->l.E || g->dtype != d->dtype || g->device != d->device)
        return fail(SG_ERR_INVALID_ARG, "gate_up and down must have the same ranks, experts, dtype and device");
    if (d->l.in * 2 != g->l.out)
        return fail(SG_ERR_INVALID_ARG, "down's input %lld is not half of gate_up's output %lld", (long long)d->l.in,
                    (long long)g->l.out);
    return SG_OK;
}

sg_status check_route(const sg::Route& r, int64_t T, int64_t ld) {
    if (!known(r.dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dtype %d", r.dtype);
    if (T < 0 || r.E < 1 || r.k < 1 || r.k > r.E)
        return fail(SG_ERR_INVALID_ARG, "a router needs T >= 0 tokens and 1 <= k <= E (got k %d, E %d)", r.k, r.E);
    if (r.E > sg::kRouteMaxExperts || r.k > sg::kRouteMaxK)
        return fail(SG_ERR_UNSUPPORTED, "more than %d experts, or %d choices, are not supported", sg::kRouteMaxExperts,
                    sg::kRouteMaxK);
    if (T > kMaxTokens || T > kMaxRows / r.k)
        return fail(SG_ERR_UNSUPPORTED, "more than 2^25 tokens, or 2^30 slots, are not supported");
    if (ld < r.E) return fail(SG_ERR_INVALID_ARG, "row stride %lld of the logits is below E", (long long)ld);
    return SG_OK;
}

sg_status check_slots(int64_t T, int k, int64_t D, int64_t R) {
    if (T < 0 || k < 1 || D < 1 || R < 0) return fail(SG_ERR_INVALID_ARG, "need T >= 0, k >= 1, D >= 1, R >= 0");
    if (k > sg::kRouteMaxK) return fail(SG_ERR_UNSUPPORTED, "more than %d choices are not supported", sg::kRouteMaxK);
    if (D > kMaxRows || T > kMaxRows / k || R > kMaxRows || T * (D / 512 + 1) >= sg::kMaxBlocks)
        return fail(SG_ERR_UNSUPPORTED, "more rows than one launch takes");
    return SG_OK;
}

}  // namespace

extern "C" {

sg_status sg_shard_experts(const void* weight, sg_dtype dtype, int64_t E, int64_t out_dims, int64_t in_dims, int mode,
                           int segments, int P, void* stream, sg_experts** out) {
    sg::last_error().clear();
    if (!out) return fail(SG_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    sg::ExpertsLayout l;
    if (sg_status st = layout_of(E, out_dims, in_dims, mode, segments, P, false, &l)) return st;
    if (!weight) return fail(SG_ERR_INVALID_ARG, "weight is NULL");
    if (dtype == SG_F32) return fail(SG_ERR_UNSUPPORTED, "experts hold bf16 or fp16 weights");
    if (!is16(dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    return build(l, dtype, false, weight, nullptr, nullptr, stream, out);
}

sg_status sg_shard_mxfp4_experts(const uint8_t* codes, const uint8_t* scales, int64_t E, int64_t out_dims,
                                 int64_t in_dims, int mode, int segments, int P, void* stream, sg_experts** out) {
    sg::last_error().clear();
    if (!out) return fail(SG_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    sg::ExpertsLayout l;
    if (sg_status st = layout_of(E, out_dims, in_dims, mode, segments, P, true, &l)) return st;
    if (!codes || !scales) return fail(SG_ERR_INVALID_ARG, "codes and scales must not be NULL");
    return build(l, SG_BF16, true, nullptr, codes, scales, stream, out);
}

sg_status sg_experts_update(sg_experts* x, const void* weight, void* stream) {
    sg::last_error().clear();
    if (!x || !weight) return fail(SG_ERR_INVALID_ARG, "layer and weight must not be NULL");
    if (x->mx) return fail(SG_ERR_UNSUPPORTED, "only bf16 and fp16 experts take new weights");
    if (sg_status st = check_layer(x, x->l.mode, "")) return st;
    return pack(x, weight, nullptr, nullptr, (hipStream_t)stream);
}

sg_status sg_experts_info(const sg_experts* x, int64_t* E, int64_t* out_dims, int64_t* in_dims, int* mode,
                          int* segments, int* P, sg_dtype* dtype, int* mxfp4) {
    sg::last_error().clear();
    if (!x) return fail(SG_ERR_INVALID_ARG, "layer is NULL");
    if (E) *E = x->l.E;
    if (out_dims) *out_dims = x->l.out;
    if (in_dims) *in_dims = x->l.in;
    if (mode) *mode = x->l.mode;
    if (segments) *segments = x->l.S;
    if (P) *P = x->l.P;
    if (dtype) *dtype = x->dtype;
    if (mxfp4) *mxfp4 = x->mx;
    return SG_OK;
}

void sg_experts_free(sg_experts* x) {
    if (!x) return;
    int d = x->device;
    (void)hipGetDevice(&d);
    if (d != x->device) (void)hipSetDevice(x->device);
    // Kernels queued on any stream may still read the weights: hipFree waits for
    // the device.  In relaxed mode it does so beside a capture of any thread, which
    // hipDeviceSynchronize would end.
    hipStreamCaptureMode mode = hipStreamCaptureModeRelaxed;
    (void)hipThreadExchangeStreamCaptureMode(&mode);
    if (x->w) (void)hipFree(x->w);
    if (x->wsc) (void)hipFree(x->wsc);
    (void)hipThreadExchangeStreamCaptureMode(&mode);
    if (d != x->device) (void)hipSetDevice(d);
    delete x;
}

sg_status sg_experts_all_to_sharded(const sg_experts* x, const void* a, const uint8_t* a_scales, int64_t T, int64_t ldx,
                                    const int32_t* offsets, const int32_t* rows, int k, int64_t R, void* y,
                                    int epilogue, sg_dtype y_dtype, void* stream) {
    sg::last_error().clear();
    sg_status st = check_layer(x, SG_ALL_TO_SHARDED, "sg_experts_all_to_sharded");
    if (!st) st = check_rows(x, offsets, R);
    if (!st) st = check_gather(T, ldx, x->l.in, rows, k, R);
    if (!st) st = check_acts(x, a, a_scales, ldx);
    if (!st) st = check_bytes(T, ldx, a_scales ? 1 : 4);
    if (st) return st;
    if (!known(y_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown output dtype %d", (int)y_dtype);
    if (epilogue != SG_EPI_NONE && epilogue != SG_EPI_SWIGLU)
        return fail(SG_ERR_INVALID_ARG, "unknown epilogue %d", epilogue);
    if (epilogue == SG_EPI_SWIGLU && x->l.S != 2)
        return fail(SG_ERR_INVALID_ARG, "the SwiGLU epilogue needs a layer with segments = 2");
    if (R == 0) return SG_OK;
    if (!y || (!a && T)) return fail(SG_ERR_INVALID_ARG, "x and y must not be NULL");
    if (T == 0) return fail(SG_ERR_INVALID_ARG, "%lld rows of no tokens", (long long)R);
    return launched(sg::launch_grouped(column(x, a, a_scales, T, ldx, offsets, rows, k, R, y,
                                              epilogue == SG_EPI_SWIGLU, x->l.f, y_dtype), (hipStream_t)stream),
                    "sg_experts_all_to_sharded");
}

sg_status sg_experts_sharded_to_all(const sg_experts* x, const void* h, const uint8_t* h_scales,
                                    const int32_t* offsets, int64_t R, void* y, sg_dtype y_dtype, void* stream) {
    sg::last_error().clear();
    sg_status st = check_layer(x, SG_SHARDED_TO_ALL, "sg_experts_sharded_to_all");
    if (!st) st = check_rows(x, offsets, R);
    if (!st) st = check_acts(x, h, h_scales, x->l.kl);
    if (!st) st = check_bytes(R, x->l.kl, h_scales ? 1 : 4);
    if (st) return st;
    if (!known(y_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown output dtype %d", (int)y_dtype);
    if (R == 0) return SG_OK;
    if (!h || !y) return fail(SG_ERR_INVALID_ARG, "x and y must not be NULL");
    return launched(sg::launch_grouped(row(x, h, h_scales, x->l.kl, offsets, R, y, y_dtype), (hipStream_t)stream),
                    "sg_experts_sharded_to_all");
}

size_t sg_moe_mlp_workspace(const sg_experts* g, const sg_experts* d, int64_t T, int k) {
    if (check_pair(g, d) || T <= 0 || k < 1 || T > kMaxRows / k) return 0;
    const size_t R = (size_t)(T * k);
    return (size_t)up((int64_t)(R * g->l.P * h_stride(g) * 2), 256) + R * d->l.out * 4;
}

sg_status sg_moe_mlp(const sg_experts* g, const sg_experts* d, const void* x, int64_t T, int64_t ldx,
                     const float* weights, const int32_t* offsets, const int32_t* rows, const int32_t* slots, int k,
                     void* y, sg_dtype y_dtype, void* workspace, size_t ws_bytes, void* stream) {
    sg::last_error().clear();
    sg_status st = check_pair(g, d);
    if (!st) st = check_layer(g, SG_ALL_TO_SHARDED, "sg_moe_mlp");
    if (!st) st = check_slots(T, k, d->l.out, 0);
    if (st) return st;
    const int64_t R = T * k;
    if (!st) st = check_gather(T, ldx, g->l.in, rows, k, 0);
    if (!st) st = check_bytes(T, ldx, 4);
    if (!st) st = check_bytes(R, h_stride(g), 4);
    if (st) return st;
    if (!known(y_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown output dtype %d", (int)y_dtype);
    if (T == 0) return SG_OK;
    if (!x || !y || !weights || !offsets || !rows || !slots)
        return fail(SG_ERR_INVALID_ARG, "x, y and the routing plan must not be NULL");
    const size_t need = sg_moe_mlp_workspace(g, d, T, k);
    if (!workspace || ws_bytes < need || !aligned(workspace, 16))
        return fail(SG_ERR_WORKSPACE, "sg_moe_mlp needs %zu bytes of 16-byte aligned workspace (got %zu)", need,
                    workspace ? ws_bytes : (size_t)0);
    hipStream_t s = (hipStream_t)stream;
    const int64_t ldh = h_stride(g);
    // h is rounded to the layers' 16 bits: the matrix instruction multiplies values
    // of one type, and h in two parts would cost every down product a second pass.
    // One rounding of each h beside one of each y, of the same size and independent:
    // sqrt(2) times the error of h in 32 bits (rms 0.0023 to 0.0017 of y in bf16,
    // 0.00030 to 0.00021 in fp16; 0.0026 at most, on a few hundred outputs).  An h
    // beyond 65504 is infinite in fp16.
    void* h = workspace;
    float* yr = (float*)((char*)workspace + up(R * g->l.P * ldh * 2, 256));
    st = launched(sg::launch_grouped(column(g, x, nullptr, T, ldx, offsets, rows, k, R, h, 1, ldh, g->dtype), s),
                  "sg_moe_mlp gate_up");
    if (!st) st = launched(sg::launch_grouped(row(d, h, nullptr, ldh, offsets, R, yr, SG_F32), s), "sg_moe_mlp down");
    if (!st) st = launched(sg::launch_combine(yr, SG_F32, slots, weights, T, k, d->l.out, R, y, y_dtype, s),
                           "sg_moe_mlp combine");
    return st;
}

static sg_status check_backward(const sg_experts* x, const void* in, int64_t T, const void* dy, int64_t R, const void* dx,
                                sg_dtype dx_dtype, const void* dw, sg_dtype dw_dtype) {
    if (x->mx) return fail(SG_ERR_UNSUPPORTED, "MXFP4 experts have no backward pass");
    if (!dx && !dw) return fail(SG_ERR_INVALID_ARG, "dx and dw are both NULL");
    if (dx && !known(dx_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dx dtype %d", (int)dx_dtype);
    if (dw && !known(dw_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dw dtype %d", (int)dw_dtype);
    if (R > 0 && !dy) return fail(SG_ERR_INVALID_ARG, "dy is NULL");
    if (R > 0 && dw && !in) return fail(SG_ERR_INVALID_ARG, "dw needs x");
    if (R > 0 && dw && T == 0) return fail(SG_ERR_INVALID_ARG, "%lld rows of no tokens", (long long)R);
    return SG_OK;
}

sg_status sg_experts_all_to_sharded_backward(const sg_experts* x, const void* a, int64_t T, int64_t ldx,
                                             const void* dy, const int32_t* offsets, const int32_t* rows, int k,
                                             int64_t R, void* dx, sg_dtype dx_dtype, void* dw, sg_dtype dw_dtype,
                                             void* stream) {
    sg::last_error().clear();
    sg_status st = check_layer(x, SG_ALL_TO_SHARDED, "sg_experts_all_to_sharded_backward");
    if (!st) st = check_rows(x, offsets, R);
    if (!st && dw) st = check_gather(T, ldx, x->l.in, rows, k, R);
    if (!st) st = check_backward(x, a, T, dy, R, dx, dx_dtype, dw, dw_dtype);
    if (!st) st = check_bytes(R, x->l.f * x->l.S, 4);
    if (!st && dw) st = check_bytes(T, ldx, 4);
    if (st) return st;
    const sg::ExpertsLayout& l = x->l;
    hipStream_t s = (hipStream_t)stream;
    if (dx && R > 0)
        st = launched(sg::launch_grouped(column_dx(x, dy, l.f, offsets, R, dx, dx_dtype), s),
                      "sg_experts_all_to_sharded_backward dx");
    if (!st && dw)
        st = launched(sg::launch_grouped_dw(column_dw(x, a, T, ldx, dy, offsets, rows, k, R, dw, dw_dtype), s),
                      "sg_experts_all_to_sharded_backward dw");
    return st;
}

sg_status sg_experts_sharded_to_all_backward(const sg_experts* x, const void* h, const void* dy,
                                             const int32_t* offsets, int64_t R, void* dh, sg_dtype dh_dtype, void* dw,
                                             sg_dtype dw_dtype, void* stream) {
    sg::last_error().clear();
    sg_status st = check_layer(x, SG_SHARDED_TO_ALL, "sg_experts_sharded_to_all_backward");
    if (!st) st = check_rows(x, offsets, R);
    if (!st) st = check_backward(x, h, R, dy, R, dh, dh_dtype, dw, dw_dtype);
    if (!st) st = check_bytes(R, x->l.out, 4);
    if (!st && dw) st = check_bytes(R, x->l.kl, 4);
    if (st) return st;
    hipStream_t s = (hipStream_t)stream;
    if (dh && R > 0)
        st = launched(sg::launch_grouped(row_dx(x, dy, offsets, R, dh, dh_dtype), s),
                      "sg_experts_sharded_to_all_backward dx");
    if (!st && dw)
        st = launched(sg::launch_grouped_dw(row_dw(x, h, dy, offsets, R, dw, dw_dtype), s),
                      "sg_experts_sharded_to_all_backward dw");
    return st;
}

size_t sg_moe_route_workspace(int64_t T, int E, int k) {
    if (T <= 0 || E < 1 || k < 1 || E > sg::kRouteMaxExperts || k > sg::kRouteMaxK || T > kMaxRows / k) return 0;
    return sg::route_workspace_ints(T, E, k) * 4;
}

sg_status sg_moe_route(const void* logits, int64_t ld, sg_dtype dtype, int64_t T, int E, int k, int normalize,
                       float* weights, int32_t* experts, int32_t* offsets, int32_t* rows, int32_t* slots,
                       void* workspace, size_t ws_bytes, void* stream) {
    sg::last_error().clear();
    sg::Route r{};
    r.dtype = dtype;
    r.E = E;
    r.k = k;
    if (sg_status st = check_route(r, T, ld)) return st;
    if (!offsets || (T && (!logits || !weights || !experts || !rows || !slots)))
        return fail(SG_ERR_INVALID_ARG, "the logits and every output must not be NULL");
    const size_t need = sg_moe_route_workspace(T, E, k);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 4)))
        return fail(SG_ERR_WORKSPACE, "sg_moe_route needs %zu bytes of workspace (got %zu)", need,
                    workspace ? ws_bytes : (size_t)0);
    r.logits = logits;
    r.ld = ld;
    r.T = (int)T;
    r.normalize = normalize != 0;
    r.weights = weights;
    r.experts = experts;
    r.offsets = offsets;
    r.rows = rows;
    r.slots = slots;
    r.ws = (int32_t*)workspace;
    return launched(sg::launch_route(r, (hipStream_t)stream), "sg_moe_route");
}

sg_status sg_moe_route_backward(const void* logits, int64_t ld, sg_dtype dtype, int64_t T, int E, int k, int normalize,
                                const float* weights, const int32_t* experts, const float* dweights, void* dlogits,
                                void* stream) {
    sg::last_error().clear();
    sg::Route r{};
    r.dtype = dtype;
    r.E = E;
    r.k = k;
    if (sg_status st = check_route(r, T, ld)) return st;
    if (T == 0) return SG_OK;
    if ((!logits && !normalize) || !weights || !experts || !dweights || !dlogits)
        return fail(SG_ERR_INVALID_ARG, "the inputs and dlogits must not be NULL");
    r.logits = logits;
    r.ld = ld;
    r.T = (int)T;
    r.normalize = normalize != 0;
    r.weights = (float*)weights;
    r.experts = (int32_t*)experts;
    return launched(sg::launch_route_backward(r, dweights, dlogits, E, (hipStream_t)stream), "sg_moe_route_backward");
}

sg_status sg_moe_combine(const void* y, sg_dtype y_dtype, int64_t R, const int32_t* slots, const float* weights,
                         int64_t T, int k, int64_t D, void* out, sg_dtype out_dtype, void* stream) {
    sg::last_error().clear();
    if (sg_status st = check_slots(T, k, D, R)) return st;
    if (!known(y_dtype) || !known(out_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dtype");
    if (T == 0) return SG_OK;
    if (!slots || !out || (R && !y)) return fail(SG_ERR_INVALID_ARG, "y, slots and out must not be NULL");
    return launched(sg::launch_combine(y, y_dtype, slots, weights, T, k, D, R, out, out_dtype, (hipStream_t)stream),
                    "sg_moe_combine");
}

sg_status sg_moe_combine_backward(const void* dout, const void* y, sg_dtype dtype, int64_t R, const int32_t* slots,
                                  const float* weights, int64_t T, int k, int64_t D, void* dy, float* dweights,
                                  void* stream) {
    sg::last_error().clear();
    if (sg_status st = check_slots(T, k, D, R)) return st;
    if (!known(dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (!dy && !dweights) return fail(SG_ERR_INVALID_ARG, "dy and dweights are both NULL");
    if (T == 0) return SG_OK;
    if (!dout || !slots || (R && dweights && !y))
        return fail(SG_ERR_INVALID_ARG, "dout, slots and (for dweights) y must not be NULL");
    return launched(sg::launch_combine_backward(dout, y, dtype, slots, weights, T, k, D, R, dy, dweights,
                                                (hipStream_t)stream), "sg_moe_combine_backward");
}

static sg_status check_swiglu(sg_dtype dtype, int64_t rows, int64_t f) {
    if (!known(dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (rows < 0 || f < 1) return fail(SG_ERR_INVALID_ARG, "need rows >= 0 and f >= 1");
    if ((double)rows * (double)((f + 7) / 8) >= (double)(sg::kMaxBlocks - 1) * 256)
        return fail(SG_ERR_UNSUPPORTED, "more values than one launch takes");
    return SG_OK;
}

sg_status sg_swiglu(const void* gu, sg_dtype dtype, int64_t rows, int64_t f, void* h, void* stream) {
    sg::last_error().clear();
    if (sg_status st = check_swiglu(dtype, rows, f)) return st;
    if (rows == 0) return SG_OK;
    if (!gu || !h) return fail(SG_ERR_INVALID_ARG, "gu and h must not be NULL");
    return launched(sg::launch_swiglu(gu, dtype, rows, f, h, (hipStream_t)stream), "sg_swiglu");
}

sg_status sg_swiglu_backward(const void* gu, const void* dh, sg_dtype dtype, int64_t rows, int64_t f, void* dgu,
                             void* stream) {
    sg::last_error().clear();
    if (sg_status st = check_swiglu(dtype, rows, f)) return st;
    if (rows == 0) return SG_OK;
    if (!gu || !dh || !dgu) return fail(SG_ERR_INVALID_ARG, "gu, dh and dgu must not be NULL");
    return launched(sg::launch_swiglu_backward(gu, dh, dtype, rows, f, dgu, (hipStream_t)stream), "sg_swiglu_backward");
}

static sg_status check_mx(sg_dtype dtype, int64_t rows, int64_t cols) {
    if (!known(dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (rows < 0 || cols < 0) return fail(SG_ERR_INVALID_ARG, "rows and cols must be >= 0");
    if (cols % 32) return fail(SG_ERR_NOT_DIVISIBLE, "%lld columns are not a multiple of the scale block of 32",
                               (long long)cols);
    if ((double)rows * (double)cols / 8 >= (double)(sg::kMaxBlocks - 1) * 256)
        return fail(SG_ERR_UNSUPPORTED, "more values than one launch takes");
    return SG_OK;
}

sg_status sg_quantize_mxfp4(const void* x, sg_dtype dtype, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes,
                            uint8_t* scales, void* stream) {
    sg::last_error().clear();
    if (sg_status st = check_mx(dtype, rows, cols)) return st;
    if (ldx < cols) return fail(SG_ERR_INVALID_ARG, "row stride %lld is below the width %lld", (long long)ldx,
                                (long long)cols);
    if (rows == 0 || cols == 0) return SG_OK;
    if (!x || !codes || !scales) return fail(SG_ERR_INVALID_ARG, "x, codes and scales must not be NULL");
    if (!aligned(codes, 4)) return fail(SG_ERR_INVALID_ARG, "codes must be 4-byte aligned");
    return launched(sg::launch_quantize_mxfp4(x, dtype, rows, cols, ldx, codes, scales, (hipStream_t)stream),
                    "sg_quantize_mxfp4");
}

sg_status sg_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* x,
                              sg_dtype dtype, void* stream) {
    sg::last_error().clear();
    if (sg_status st = check_mx(dtype, rows, cols)) return st;
    if (rows == 0 || cols == 0) return SG_OK;
    if (!x || !codes || !scales) return fail(SG_ERR_INVALID_ARG, "x, codes and scales must not be NULL");
    if (!aligned(codes, 4) || !aligned(x, 16))
        return fail(SG_ERR_INVALID_ARG, "codes must be 4-byte, x 16-byte aligned");
    return launched(sg::launch_dequantize_mxfp4(codes, scales, rows, cols, x, dtype, (hipStream_t)stream),
                    "sg_dequantize_mxfp4");
}

// ---- the gated block on activations kept in 8 bits ---------------------------

static sg_status check_mx8(sg_dtype dtype, int64_t rows, int64_t cols) {
    if (!known(dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (rows < 0 || cols < 0) return fail(SG_ERR_INVALID_ARG, "rows and cols must be >= 0");
    if ((double)rows * (double)sg::mx8_blocks(cols) * 4 >= (double)(sg::kMaxBlocks - 1) * 256)
        return fail(SG_ERR_UNSUPPORTED, "more values than one launch takes");
    return SG_OK;
}

sg_status sg_quantize_mxfp8(const void* x, sg_dtype dtype, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes,
                            uint8_t* scales, void* stream) {
    sg::last_error().clear();
    if (sg_status st = check_mx8(dtype, rows, cols)) return st;
    if (ldx < cols) return fail(SG_ERR_INVALID_ARG, "row stride %lld is below the width %lld", (long long)ldx,
                                (long long)cols);
    if (rows == 0 || cols == 0) return SG_OK;
    if (!x || !codes || !scales) return fail(SG_ERR_INVALID_ARG, "x, codes and scales must not be NULL");
    return launched(sg::launch_quantize_mxfp8(x, dtype, rows, cols, ldx, codes, scales, (hipStream_t)stream),
                    "sg_quantize_mxfp8");
}

sg_status sg_dequantize_mxfp8(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* x,
                              sg_dtype dtype, void* stream) {
    sg::last_error().clear();
    if (sg_status st = check_mx8(dtype, rows, cols)) return st;
    if (rows == 0 || cols == 0) return SG_OK;
    if (!x || !codes || !scales) return fail(SG_ERR_INVALID_ARG, "x, codes and scales must not be NULL");
    return launched(sg::launch_dequantize_mxfp8(codes, scales, rows, cols, x, cols, dtype, false, (hipStream_t)stream),
                    "sg_dequantize_mxfp8");
}

static sg_status check_gate_up(const sg_experts* g) {
    if (sg_status st = check_layer(g, SG_ALL_TO_SHARDED, "a gated block")) return st;
    if (g->mx) return fail(SG_ERR_UNSUPPORTED, "a gated block that keeps its activations needs bf16 or fp16 layers");
    if (g->l.S != 2) return fail(SG_ERR_INVALID_ARG, "gate_up must be an all-to-sharded layer with segments = 2");
    return SG_OK;
}
static sg_status check_down(const sg_experts* d) {
    if (sg_status st = check_layer(d, SG_SHARDED_TO_ALL, "a gated block")) return st;
    if (d->mx) return fail(SG_ERR_UNSUPPORTED, "a gated block that keeps its activations needs bf16 or fp16 layers");
    if (d->l.S != 1) return fail(SG_ERR_INVALID_ARG, "down must be a sharded-to-all layer with segments = 1");
    return SG_OK;
}
static sg_status check_ws(const char* what, const void* ws, size_t bytes, size_t need) {
    if (need && (!ws || bytes < need || !aligned(ws, 16)))
        return fail(SG_ERR_WORKSPACE, "%s needs %zu bytes of 16-byte aligned workspace (got %zu)", what, need,
                    ws ? bytes : (size_t)0);
    return SG_OK;
}
// rows of the block: f columns of P ranks, as many threads as a launch may have
static sg_status check_gated_rows(int64_t P, int64_t R, int64_t f) {
    if ((double)P * (double)R * (double)sg::mx8_blocks(f) * 4 >= (double)(sg::kMaxBlocks - 1) * 256)
        return fail(SG_ERR_UNSUPPORTED, "more values than one launch takes");
    return SG_OK;
}

static bool fused(const sg_experts* g) { return sg::gated_fits(g->l.P, g->l.bps); }

size_t sg_experts_gated_workspace(const sg_experts* g, int64_t R) {
    if (!g || g->l.mode != SG_ALL_TO_SHARDED || g->l.S != 2 || g->mx || R <= 0 || R > kMaxRows) return 0;
    return fused(g) ? 0 : (size_t)up(R * g->l.out * 4, 256);
}

// h's rows are ldh >= f columns apart, zeros behind f
static sg_status gated(const sg_experts* g, const void* x, int64_t T, int64_t ldx, const int32_t* offsets,
                       const int32_t* rows, int k, int64_t R, void* h, int64_t ldh, uint8_t* codes, uint8_t* scales,
                       void* workspace, hipStream_t s) {
    if (fused(g)) {
        sg::Gated kept{};
        kept.codes = codes;
        kept.scales = scales;
        kept.f = (int)g->l.f;
        return launched(sg::launch_gated(column(g, x, nullptr, T, ldx, offsets, rows, k, R, h, 1, ldh, g->dtype), kept, s),
                        "gated block");
    }
    sg_status st = launched(sg::launch_grouped(column(g, x, nullptr, T, ldx, offsets, rows, k, R, workspace, 0, 0, SG_F32), s),
                            "gated block");
    if (!st) st = launched(sg::launch_gated_keep((const float*)workspace, g->l.P, R, g->l.f, ldh, offsets, (int)g->l.E, h,
                                                 g->dtype == SG_F16, codes, scales, s), "gated block");
    return st;
}

// dgu's pieces and h's rows are fp >= f columns, zeros behind f
static sg_status gated_backward(const sg_experts* d, const void* dy, const uint8_t* codes, const uint8_t* scales,
                                const int32_t* offsets, int64_t R, void* dgu, void* h, int64_t fp, hipStream_t s) {
    sg::Gated kept{};
    kept.codes = (uint8_t*)codes;
    kept.scales = (uint8_t*)scales;
    kept.f = (int)d->l.kl;
    kept.h = h;
    sg::Grouped p = row_dx(d, dy, offsets, R, dgu, d->dtype);
    p.f = (int)fp;
    return launched(sg::launch_gated_backward(p, kept, s), "gated block");
}

sg_status sg_experts_gated(const sg_experts* g, const void* x, int64_t T, int64_t ldx, const int32_t* offsets,
                           const int32_t* rows, int k, int64_t R, void* h, uint8_t* codes, uint8_t* scales,
                           void* workspace, size_t ws_bytes, void* stream) {
    sg::last_error().clear();
    sg_status st = check_gate_up(g);
    if (!st) st = check_rows(g, offsets, R);
    if (!st) st = check_gather(T, ldx, g->l.in, rows, k, R);
    if (!st) st = check_bytes(T, ldx, 4);
    if (!st) st = check_gated_rows(g->l.P, R, g->l.f);
    if (st) return st;
    if (R == 0) return SG_OK;
    if (T == 0) return fail(SG_ERR_INVALID_ARG, "%lld rows of no tokens", (long long)R);
    if (!x || !h || !codes || !scales) return fail(SG_ERR_INVALID_ARG, "x, h, codes and scales must not be NULL");
    if ((st = check_ws("sg_experts_gated", workspace, ws_bytes, sg_experts_gated_workspace(g, R)))) return st;
    return gated(g, x, T, ldx, offsets, rows, k, R, h, g->l.f, codes, scales, workspace, (hipStream_t)stream);
}

sg_status sg_experts_gated_backward(const sg_experts* d, const void* dy, const uint8_t* codes, const uint8_t* scales,
                                    const int32_t* offsets, int64_t R, void* dgu, void* h, void* stream) {
    sg::last_error().clear();
    sg_status st = check_down(d);
    if (!st) st = check_rows(d, offsets, R);
    if (!st) st = check_bytes(R, d->l.out, 4);
    if (!st) st = check_gated_rows(d->l.P, R, d->l.kl);
    if (st) return st;
    if (R == 0) return SG_OK;
    if (!dy || !codes || !scales || !dgu) return fail(SG_ERR_INVALID_ARG, "dy, codes, scales and dgu must not be NULL");
    return gated_backward(d, dy, codes, scales, offsets, R, dgu, h, d->l.kl, (hipStream_t)stream);
}

// A product of few rows and few tiles is split over its inputs (up to eight rows of an
// expert it streams the weights, and splits them there)
static int splits_of(const sg::Grouped& p) { return p.R > (int64_t)8 * p.E ? sg::grouped_splits(p) : 1; }
static size_t split_bytes(const sg::Grouped& p) {
    const int n = splits_of(p);
    return n > 1 ? (size_t)up((int64_t)n * p.R * p.ldo * 4, 256) : 0;
}
static sg_status product(const sg::Grouped& p, void* workspace, const char* what, hipStream_t s) {
    const int n = splits_of(p);
    return launched(n > 1 ? sg::launch_grouped_split(p, n, (float*)workspace, s) : sg::launch_grouped(p, s), what);
}

size_t sg_gated_mlp_workspace(const sg_experts* g, const sg_experts* d, int64_t R) {
    if (check_pair(g, d) || R <= 0 || R > kMaxRows) return 0;
    const size_t a = sg_experts_gated_workspace(g, R);
    const size_t b = split_bytes(row(d, nullptr, nullptr, h_stride(g), nullptr, R, nullptr, SG_F32));
    return (size_t)up(R * g->l.P * h_stride(g) * 2, 256) + (a > b ? a : b);
}

sg_status sg_gated_mlp(const sg_experts* g, const sg_experts* d, const void* x, int64_t T, int64_t ldx,
                       const int32_t* offsets, const int32_t* rows, int k, int64_t R, void* y, sg_dtype y_dtype,
                       uint8_t* x_codes, uint8_t* x_scales, uint8_t* gu_codes, uint8_t* gu_scales, void* workspace,
                       size_t ws_bytes, void* stream) {
    sg::last_error().clear();
    sg_status st = check_pair(g, d);
    if (!st) st = check_gate_up(g);
    if (!st) st = check_down(d);
    if (!st) st = check_rows(g, offsets, R);
    if (!st) st = check_gather(T, ldx, g->l.in, rows, k, R);
    if (!st) st = check_bytes(T, ldx, 4);
    if (!st) st = check_bytes(R, h_stride(g), 4);
    if (!st) st = check_gated_rows(g->l.P, R, g->l.f);
    if (!st) st = check_mx8(g->dtype, T, g->l.in);
    if (st) return st;
    if (!known(y_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown output dtype %d", (int)y_dtype);
    if (R > 0 && T == 0) return fail(SG_ERR_INVALID_ARG, "%lld rows of no tokens", (long long)R);
    if (T > 0 && (!x || !x_codes || !x_scales)) return fail(SG_ERR_INVALID_ARG, "x, x_codes and x_scales must not be NULL");
    if (R > 0 && (!y || !gu_codes || !gu_scales))
        return fail(SG_ERR_INVALID_ARG, "y, gu_codes and gu_scales must not be NULL");
    if ((st = check_ws("sg_gated_mlp", workspace, ws_bytes, sg_gated_mlp_workspace(g, d, R)))) return st;
    hipStream_t s = (hipStream_t)stream;
    const int64_t ldh = h_stride(g);
    if (T) st = launched(sg::launch_quantize_mxfp8(x, g->dtype, T, g->l.in, ldx, x_codes, x_scales, s), "sg_gated_mlp");
    if (st || R == 0) return st;
    // h is rounded to the layers' 16 bits, as in sg_moe_mlp and for its reason: it is the
    // down product's operand, whose two halves would cost a second pass (sqrt(2) times the
    // error of y that h in 32 bits would leave)
    void* rest = (char*)workspace + up(R * g->l.P * ldh * 2, 256);
    st = gated(g, x, T, ldx, offsets, rows, k, R, workspace, ldh, gu_codes, gu_scales, rest, s);
    if (!st) st = product(row(d, workspace, nullptr, ldh, offsets, R, y, y_dtype), rest, "sg_gated_mlp down", s);
    return st;
}

// dgu (P, R, 2, fp), h (P, R, fp), x in 16 bits, and a split dx's parts
size_t sg_gated_mlp_backward_workspace(const sg_experts* g, const sg_experts* d, int64_t T, int64_t R) {
    if (check_pair(g, d) || R <= 0 || R > kMaxRows || T < 0 || T > kMaxRows) return 0;
    const int64_t fp = h_stride(g), n = R * g->l.P * fp * 2;
    return (size_t)up(2 * n, 256) + (size_t)up(n, 256) + (size_t)up(T * up(g->l.in, 8) * 2, 256) +
           split_bytes(column_dx(g, nullptr, fp, nullptr, R, nullptr, SG_F32));
}

sg_status sg_gated_mlp_backward(const sg_experts* g, const sg_experts* d, const uint8_t* x_codes,
                                const uint8_t* x_scales, int64_t T, const uint8_t* gu_codes, const uint8_t* gu_scales,
                                const void* dy, const int32_t* offsets, const int32_t* rows, int k, int64_t R, void* dx,
                                sg_dtype dx_dtype, void* dw_gate_up, void* dw_down, sg_dtype dw_dtype, void* workspace,
                                size_t ws_bytes, void* stream) {
    sg::last_error().clear();
    sg_status st = check_pair(g, d);
    if (!st) st = check_gate_up(g);
    if (!st) st = check_down(d);
    const int64_t fp = st ? 0 : h_stride(g), ldx = st ? 0 : up(g->l.in, 8);
    if (!st) st = check_rows(g, offsets, R);
    if (!st) st = check_tokens(T);  // the workspace holds x whatever is asked for
    if (!st && dw_gate_up) st = check_gather(T, ldx, g->l.in, rows, k, R);
    if (!st && dw_gate_up) st = check_bytes(T, ldx, 4);
    if (!st && dw_gate_up) st = check_mx8(g->dtype, T, g->l.in);
    if (!st) st = check_bytes(R, fp * 2, 4);
    if (!st) st = check_bytes(R, d->l.out, 4);
    if (!st) st = check_gated_rows(g->l.P, R, g->l.f);
    if (st) return st;
    if (!dx && !dw_gate_up && !dw_down) return fail(SG_ERR_INVALID_ARG, "dx, dw_gate_up and dw_down are all NULL");
    if (dx && !known(dx_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dx dtype %d", (int)dx_dtype);
    if ((dw_gate_up || dw_down) && !known(dw_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dw dtype %d", (int)dw_dtype);
    if (R > 0 && dw_gate_up && T == 0) return fail(SG_ERR_INVALID_ARG, "%lld rows of no tokens", (long long)R);
    if (R > 0 && (!dy || !gu_codes || !gu_scales))
        return fail(SG_ERR_INVALID_ARG, "dy, gu_codes and gu_scales must not be NULL");
    if (R > 0 && dw_gate_up && (!x_codes || !x_scales))
        return fail(SG_ERR_INVALID_ARG, "dw_gate_up needs x_codes and x_scales");
    if ((st = check_ws("sg_gated_mlp_backward", workspace, ws_bytes, sg_gated_mlp_backward_workspace(g, d, T, R))))
        return st;
    hipStream_t s = (hipStream_t)stream;
    const int64_t n = R * g->l.P * fp * 2;
    char* dgu = (char*)workspace;
    char* h = dgu + up(2 * n, 256);
    char* x = h + up(n, 256);
    char* rest = x + up(T * ldx * 2, 256);
    // dgu is stored in the layers' 16 bits, once, the operand of both products behind it,
    // and h again (a matrix instruction multiplies values of one type; two halves would cost
    // each product a second pass): sqrt(2) times the error of dx and dW.  Rows of it, of h
    // and of x begin on 16 bytes whatever f and in are.
    if (R > 0) {
        st = gated_backward(d, dy, gu_codes, gu_scales, offsets, R, dgu, dw_down ? h : nullptr, fp, s);
        if (!st && dx) st = product(column_dx(g, dgu, fp, offsets, R, dx, dx_dtype), rest, "sg_gated_mlp_backward dx", s);
        if (!st && dw_gate_up)
            st = launched(sg::launch_dequantize_mxfp8(x_codes, x_scales, T, g->l.in, x, ldx, g->dtype, true, s),
                          "sg_gated_mlp_backward");
    }
    if (!st && dw_gate_up) {
        sg::GroupedDw p = column_dw(g, x, T, ldx, dgu, offsets, rows, k, R, dw_gate_up, dw_dtype);
        p.ldg = p.O = (int)(2 * fp);
        p.g_rank = R * 2 * fp;
        p.of = (int)g->l.f;
        p.ofp = (int)fp;
        p.xw = (int)ldx;
        st = launched(sg::launch_grouped_dw(p, s), "sg_gated_mlp_backward dw_gate_up");
    }
    if (!st && dw_down) {
        sg::GroupedDw p = row_dw(d, h, dy, offsets, R, dw_down, dw_dtype);
        p.ldx = p.xw = (int)fp;
        p.x_rank = R * fp;
        st = launched(sg::launch_grouped_dw(p, s), "sg_gated_mlp_backward dw_down");
    }
    return st;
}

}  // extern "C"
