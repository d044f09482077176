// C-ABI entry points of the low-rank adapters: validation, workspaces, and the order
// of the launches beside the shared projection's own call.  Every check runs on the
// host before any device work.
#include <stdarg.h>
#include <stdio.h>

#include "adapters.h"
#include "gated.h"

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
    return fail(e == hipErrorOutOfMemory ? SG_ERR_OOM : SG_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool known(int dt) { return dt == SG_F32 || dt == SG_BF16 || dt == SG_F16; }
size_t up256(int64_t n) { return (size_t)((n + 255) / 256 * 256); }

constexpr int64_t kMaxTokens = (int64_t)1 << 25;

struct Geometry {
    int64_t out, in;
    int mode, S, P, quantized;
    sg_dtype dtype;
    bool column() const { return mode == SG_ALL_TO_SHARDED; }
    int64_t part() const { return (column() ? out : in) / S / P; }
};

// the rank-sharded side's activation, (P, T, S part), and the replicated one's
sg::Pieces sharded(const Geometry& g, int64_t T) {
    const int64_t ld = g.S * g.part();
    return {T * ld, ld, g.S, g.P, (int)g.part()};
}
sg::Pieces full(int64_t width) { return {0, width, 1, 1, (int)width}; }
sg::Pieces x_pieces(const Geometry& g, int64_t T) { return g.column() ? full(g.in) : sharded(g, T); }
sg::Pieces y_pieces(const Geometry& g, int64_t T) { return g.column() ? sharded(g, T) : full(g.out); }

sg::Plan plan_of(const int32_t* plan, int64_t T, int n) {
    const sg::PlanLayout l = sg::plan_layout(T, n);
    return {plan + l.offsets, plan + l.rows, plan + l.ids, plan + l.tiles, (int)T, n, (int)sg::adapter_tiles(T, n),
            sg::adapter_tile_rows(T, n)};
}

sg_status check_adapters(const sg_adapters* ad) {
    if (!ad) return fail(SG_ERR_INVALID_ARG, "adapters is NULL");
    if (ad->n < 1 || ad->rank < 1) return fail(SG_ERR_INVALID_ARG, "need n >= 1 adapters of rank >= 1 (got %d, %d)", ad->n,
                                               ad->rank);
    if (ad->n > sg::kMaxAdapters || ad->rank > sg::kMaxRank)
        return fail(SG_ERR_UNSUPPORTED, "more than %d adapters, or ranks above %d, are not supported", sg::kMaxAdapters,
                    sg::kMaxRank);
    return SG_OK;
}

sg_status check_call(const sg_layer* l, int mode, const sg_adapters* ad, int64_t T, Geometry* g) {
    if (!l) return fail(SG_ERR_INVALID_ARG, "layer is NULL");
    if (sg_status st = sg_layer_info(l, &g->out, &g->in, &g->mode, &g->S, &g->P, &g->dtype, &g->quantized)) return st;
    if (g->mode != mode)
        return fail(SG_ERR_INVALID_ARG, mode == SG_ALL_TO_SHARDED ? "layer is sharded-to-all" : "layer is all-to-sharded");
    int d = -1;
    if (hipGetDevice(&d) != hipSuccess || d != sg::layer_device(l)) {
        (void)hipGetLastError();
        return fail(SG_ERR_INVALID_ARG, "the layer lives on device %d, the current device is %d", sg::layer_device(l), d);
    }
    if (g->dtype == SG_F32) return fail(SG_ERR_UNSUPPORTED, "adapters stand beside layers of bf16 or fp16 activations");
    if (sg_status st = check_adapters(ad)) return st;
    if (T < 0) return fail(SG_ERR_INVALID_ARG, "T must be >= 0");
    if (T > kMaxTokens) return fail(SG_ERR_UNSUPPORTED, "more than 2^25 tokens are not supported");
    const int64_t groups = (g->part() + 31) / 32 * g->S * g->P + ((g->column() ? g->in : g->out) + 31) / 32;
    if (groups > 4 * 65535 || (double)(sg::adapter_tiles(T, ad->n) * 4) * (double)groups >= (double)sg::kMaxBlocks * 4)
        return fail(SG_ERR_UNSUPPORTED, "more columns or tokens than one launch takes");
    if (!ad->A || !ad->B) return fail(SG_ERR_INVALID_ARG, "A and B must not be NULL");
    return SG_OK;
}

// U = X M^T in `slabs` parts, then used through M2
struct Half {
    sg::LowRank p;
    size_t bytes;
};
Half half(const Geometry& g, const sg_adapters* ad, const int32_t* plan, int64_t T, bool of_x) {
    Half h{};
    sg::LowRank& p = h.p;
    p.plan = plan_of(plan, T, ad->n);
    p.f16 = g.dtype == SG_F16;
    p.rank = ad->rank;
    p.rp = (ad->rank + 15) / 16 * 16;
    p.M = of_x ? ad->A : ad->B;
    p.transposed = !of_x;
    p.width = of_x ? g.in : g.out;
    p.x = of_x ? x_pieces(g, T) : y_pieces(g, T);
    p.slabs = T ? sg::shrink_slabs(p.plan, p.width, p.rank) : 1;
    p.slab = T * p.rp;
    p.scale = ad->scale;
    h.bytes = up256(p.slab * p.slabs * 4);
    return h;
}


sg_status check_ws(const char* what, const void* ws, size_t bytes, size_t need) {
    if (need && (!ws || bytes < need || (uintptr_t)ws % 16))
        return fail(SG_ERR_WORKSPACE, "%s needs %zu bytes of 16-byte aligned workspace (got %zu)", what, need,
                    ws ? bytes : (size_t)0);
    return SG_OK;
}

// The projection's product on the grouped tiles, x W^T or (transposed) dy W: what it is
// but for its weights.  False where they, or the tokens, do not suit the tiles.
bool tile_product(const sg_layer* l, const Geometry& g, int64_t T, bool transposed, bool swiglu, sg::Grouped* to) {
    sg::Grouped& p = *to;
    p = sg::Grouped{};
    const int64_t f = g.part(), rank_width = g.S * f;  // of the sharded side
    // (a rank's segments of a sharded-to-all layer lie side by side in its matrix: of whole
    // blocks and without padding behind them, where there are several)
    if ((T <= 8 && !g.quantized) || (g.quantized && (transposed || !sg::layer_codes(l, T).any())) ||
        (!g.column() && g.S > 1 && (f % 16 || rank_width % 64)) ||
        (double)T * (double)(g.in > g.out ? g.in : g.out) * 2 >= (double)0xffff0000ll ||
        (double)((g.out + 15 + 16 * g.S * g.P) * (g.in + 63 + 64 * g.P)) * (g.quantized ? 4 : 2) >= (double)0xffff0000ll)
        return false;
    p.mode = g.dtype == SG_F16 ? sg::G_F16 : sg::G_BF16;
    p.kdiv = 1;
    p.T = p.R = (int)T;
    p.E = 1;
    p.transposed = transposed;
    p.swiglu = swiglu;
    const bool in_sharded = g.column() == transposed;  // the product's input is the sharded side
    const int64_t width = transposed ? g.out : g.in, cols = transposed ? g.in : g.out;
    const int64_t rows16 = ((g.column() ? f : g.out) + 15) / 16 * 16;  // of a part, or of a rank's matrix
    const int64_t cols64 = ((g.column() ? g.in : rank_width) + 63) / 64 * 64;
    // input: the parts of an all-to-sharded layer's output, the ranks' rows of a
    // sharded-to-all layer's input, or whole rows
    p.a_pieces = in_sharded && g.column() ? g.S : 1;
    p.nseg = !in_sharded ? 1 : g.column() ? g.S * g.P : g.P;
    p.kl = (int)(!in_sharded ? width : g.column() ? f : rank_width);
    p.kpad = (int)(transposed ? rows16 : cols64);
    p.lda = in_sharded ? rank_width : width;
    p.a_rank = in_sharded ? T * rank_width : 0;
    // output: parts of f columns each; the one of a rank of a sharded-to-all layer with the
    // padding of its matrix
    const bool parts = !in_sharded && (g.column() || g.S > 1);
    p.S = swiglu || !parts ? 1 : g.S;
    p.f = (int)(parts ? f : in_sharded ? cols : rank_width);
    p.bps = (int)(parts ? (f + 15) / 16 : transposed ? cols64 / 16 : rows16 / 16);
    p.nout = (int)(p.bps * (in_sharded ? 1 : g.P) * (parts && !swiglu ? g.S : 1));
    p.ldo = in_sharded ? cols : swiglu ? f : rank_width;
    p.o_rank = in_sharded ? 0 : T * p.ldo;
    return true;
}

// 16-bit matrices that a layer's weights make up: hi and lo of a 4-bit one's
int halves(const Geometry& g) { return g.quantized == 1 ? 2 : 1; }
size_t weight_bytes(const Geometry& g) {
    if (!g.quantized) return 0;
    const int64_t blocks = g.column() ? (g.part() + 15) / 16 * g.S * g.P : (g.out + 15) / 16;
    return (size_t)(halves(g) * (g.column() ? 1 : g.P) * blocks * (((g.column() ? g.in : g.in / g.P) + 63) / 64 * 2) * 1024);
}

// Its weights; of a quantized layer at `at` (weight_bytes).  p.W stays null where there are none.
sg_status tile_weights(const sg_layer* l, const Geometry& g, void* at, hipStream_t s, sg::Grouped* to, sg::Adapted* d) {
    sg::Grouped& p = *to;
    sg::LayerTiles v{};
    if (g.quantized) {
        const int64_t cols = g.column() ? g.in : g.in / g.P;
        v.blocks = g.column() ? (g.part() + 15) / 16 * g.S * g.P : (g.out + 15) / 16;
        v.steps = (cols + 63) / 64 * 2;
        v.w = at;
        const sg::LayerCodes codes = sg::layer_codes(l, to->T);
        if (sg_status st = launched(sg::launch_code_tiles(codes, g.dtype == SG_F16, g.column() ? 1 : g.P, g.out,
                                                          g.column() ? g.part() : g.out, cols, at, s), "weight codes"))
            return st;
        if (codes.codes) {  // the same inputs through the lo halves
            d->again = p.nseg;
            p.nseg *= 2;
        }
    } else if (sg_status st = launched(sg::layer_tiles(l, !p.transposed, s, &v), "weight layout")) {
        return st;
    }
    if (!v.w) return SG_OK;
    const int64_t matrix = v.blocks * v.steps * 1024;
    p.W = (const uint8_t*)v.w;
    p.w_expert = matrix * (g.column() ? 1 : g.P) * halves(g);
    p.wsteps = (int)v.steps;
    d->wseg = d->wrank = (uint32_t)matrix;
    return SG_OK;
}

// the adapters' part of the epilogue
void set_adapted(const Geometry& g, const sg_adapters* ad, const sg::Plan& plan, sg::Grouped* p, sg::Adapted* d) {
    const bool in_sharded = g.column() == (bool)p->transposed;
    p->rows = plan.rows;
    d->plan = plan;
    d->rank = ad->rank;
    d->M = p->transposed ? ad->A : ad->B;
    d->width = p->transposed ? g.in : g.out;
    d->P = in_sharded ? 1 : g.P;
}

// Fewer tiles than fill the chip: the projection's part by itself, its sums split over
// the inputs, in fp32.  (A transposed product's weights and a sharded-to-all layer's
// ranks lie as the plain tiles have them only where there is one matrix.)
bool split_product(const Geometry& g, const sg::Grouped& p) {
    return !g.quantized && (g.column() || g.P == 1) && !sg::adapted_fills(p);
}
size_t split_bytes(const sg::Grouped& p) {
    const int n = sg::grouped_splits(p);
    return n > 1 ? up256(n * sg::grouped_outputs(p) * 4) : 0;
}
sg_status launch_split(sg::Grouped p, const void* a, float* out, void* ws, const char* what, hipStream_t s) {
    p.A = a;
    p.out = out;
    p.out_dtype = SG_F32;
    const int n = sg::grouped_splits(p);
    return launched(n > 1 ? sg::launch_grouped_split(p, n, (float*)ws, s) : sg::launch_grouped(p, s), what);
}

// U's sums, and its operands for the tiles, at `at` (operands_bytes)
size_t operands_bytes(int64_t T, int rank) { return up256((int64_t)sg::operand_bytes(T, rank)) + up256(T * 4); }
sg_status finish(const sg::LowRank& p, sg::Adapted* d, char* at, int64_t T, const char* what, hipStream_t s) {
    int32_t* ex = (int32_t*)(at + up256((int64_t)sg::operand_bytes(T, p.rank)));
    d->operands = (decltype(d->operands))at;
    d->exponents = ex;
    return launched(sg::launch_finish(p, at, ex, s), what);
}

sg_status forward(const char* what, const sg_layer* l, const Geometry& g, const sg_adapters* ad, const int32_t* plan,
                  const void* x, int64_t T, void* y, int out_layout, int epilogue, sg_dtype y_dtype, void* workspace,
                  size_t ws_bytes, void* stream) {
    if (!known(y_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown output dtype %d", (int)y_dtype);
    if (T == 0) return SG_OK;
    if (!plan || !x || !y) return fail(SG_ERR_INVALID_ARG, "plan, x and y must not be NULL");
    if (sg_status st = check_ws(what, workspace, ws_bytes, sg_adapted_workspace(l, ad, T))) return st;
    hipStream_t s = (hipStream_t)stream;
    Half u = half(g, ad, plan, T, true);
    sg::LowRank& p = u.p;
    p.U = (float*)workspace;
    p.X = x;
    sg_status st = SG_OK;
    const int64_t n = g.column() ? (epilogue == SG_EPI_SWIGLU ? g.out / 2 : g.out) / g.P : g.out;  // columns of a rank
    const bool gathered = g.column() && out_layout == SG_OUT_FULL;
    const bool swiglu = epilogue == SG_EPI_SWIGLU;
    char* rest = (char*)workspace + u.bytes;
    sg::Grouped q;
    sg::Adapted d{};
    bool tiles = tile_product(l, g, T, false, swiglu, &q), split = false;
    if (tiles && !g.quantized && !sg::adapted_fills(q))
        tiles = false, split = tile_product(l, g, T, false, false, &q) && split_product(g, q);
    if (tiles || split) {
        if ((st = tile_weights(l, g, rest + operands_bytes(T, ad->rank), s, &q, &d))) return st;
        if (!q.W) tiles = split = false;
    }
    if (tiles) {
        set_adapted(g, ad, p.plan, &q, &d);
        q.A = x;
        q.out = y;
        q.out_dtype = y_dtype;
        if (gathered) q.ldo = n * g.P, q.o_rank = n;
        st = launched(sg::launch_shrink(p, s), what);
        if (!st) st = finish(p, &d, rest, T, what, s);
        return st ? st : launched(sg::launch_adapted(q, d, s), what);
    }
    // The projection first: its own call may refuse what this one lets through.  The
    // projection's result stays in fp32 until the adapters' part is added, so that y
    // is rounded once; an fp32 y holds it itself
    const bool in_y = y_dtype == SG_F32 && !swiglu && !(split && gathered);
    char* at = rest;
    float* base = in_y ? (float*)y : (float*)at;
    at += up256(T * g.out * 4);
    // (sharded unless y is both gathered and the sum's own place)
    if (split) {
        st = launch_split(q, x, base, at, what, s);
    } else if (g.column()) {
        st = sg_all_to_sharded_ex(l, x, SG_IN_FULL, T, base, in_y ? out_layout : SG_OUT_SHARDED, SG_EPI_NONE, SG_F32, stream);
    } else {
        st = sg_sharded_to_all_ex(l, x, T, base, SG_OUT_FULL, SG_F32, at, ws_bytes - (size_t)(at - (char*)workspace), stream);
    }
    if (!st) st = launched(sg::launch_shrink(p, s), what);
    // (many rows' sums are added up once, few by every workgroup that wants them)
    if (!st && p.plan.tile_rows > 16) {
        st = launched(sg::launch_finish(p, nullptr, nullptr, s), what);
        p.slabs = 1;
    }
    if (st) return st;
    p.M = ad->B;
    p.width = g.out;
    p.x = y_pieces(g, T);
    p.base = base;
    p.swiglu = swiglu;
    p.out = y;
    p.out_dtype = y_dtype;
    p.out_ld = n;
    p.out_rank = g.column() ? T * n : 0;
    if (gathered) {
        p.out_ld = n * g.P;
        p.out_rank = n;
        if (in_y) p.x.ld = p.out_ld, p.x.rank = p.out_rank;
    }
    return launched(sg::launch_expand(p, s), what);
}

sg_status backward(const char* what, const sg_layer* l, const Geometry& g, const sg_adapters* ad, const int32_t* plan,
                   const void* x, const void* dy, int64_t T, void* dx, sg_dtype dx_dtype, void* dA, void* dB,
                   sg_dtype d_dtype, void* workspace, size_t ws_bytes, void* stream) {
    if (!dx && !dA && !dB) return fail(SG_ERR_INVALID_ARG, "dx, dA and dB are all NULL");
    if (dx && !known(dx_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown dx dtype %d", (int)dx_dtype);
    if ((dA || dB) && !known(d_dtype)) return fail(SG_ERR_INVALID_ARG, "unknown gradient dtype %d", (int)d_dtype);
    if (dx && g.quantized) return fail(SG_ERR_UNSUPPORTED, "the input gradient is implemented for dense layers only");
    if (T == 0 && !dA && !dB) return SG_OK;
    if (!plan || (T && !dy)) return fail(SG_ERR_INVALID_ARG, "plan and dy must not be NULL");
    if (T && (dA || dB) && !x) return fail(SG_ERR_INVALID_ARG, "dA and dB need x");
    if (sg_status st = check_ws(what, workspace, ws_bytes, sg_adapted_backward_workspace(l, ad, T))) return st;
    hipStream_t s = (hipStream_t)stream;
    Half u = half(g, ad, plan, T, true), v = half(g, ad, plan, T, false);
    u.p.U = (float*)workspace;
    u.p.X = x;
    v.p.U = (float*)((char*)workspace + u.bytes);
    v.p.X = dy;
    char* rest = (char*)workspace + u.bytes + v.bytes;
    sg::Grouped q{};
    sg::Adapted d{};
    sg_status st = SG_OK;
    bool tiles = T && dx && tile_product(l, g, T, true, false, &q), split = false;
    if (tiles) {
        split = split_product(g, q);
        tiles = sg::adapted_fills(q);
        if (tiles || split)
            if ((st = tile_weights(l, g, nullptr, s, &q, &d))) return st;
        if (!q.W) tiles = split = false;
    }
    // as forward: the frozen projection's part in fp32, rounded once with the adapters',
    // and before any other launch
    float* base = dx_dtype == SG_F32 ? (float*)dx : (float*)rest;
    if (T && dx && !tiles) {
        if (split) st = launch_split(q, dy, base, rest + up256(T * g.in * 4), what, s);
        else st = g.column() ? sg_all_to_sharded_backward(l, nullptr, dy, T, base, SG_F32, nullptr, SG_F32, nullptr, 0, stream)
                             : sg_sharded_to_all_backward(l, nullptr, dy, T, base, SG_F32, nullptr, SG_F32, nullptr, 0, stream);
    }
    if (!st && T && (dx || dA)) {
        st = launched(sg::launch_shrink(v.p, s), what);
        if (!st) st = tiles ? finish(v.p, &d, rest, T, what, s) : launched(sg::launch_finish(v.p, nullptr, nullptr, s), what);
        v.p.slabs = 1;
    }
    if (!st && T && dB) {
        st = launched(sg::launch_shrink(u.p, s), what);
        if (!st) st = launched(sg::launch_finish(u.p, nullptr, nullptr, s), what);
        u.p.slabs = 1;
    }
    if (!st && dA) {
        sg::LowRank p = v.p;
        p.M = ad->A;
        p.transposed = 0;
        p.width = g.in;
        p.X = x;
        p.x = x_pieces(g, T);
        p.out = dA;
        p.out_dtype = d_dtype;
        st = launched(sg::launch_grad(p, s), what);
    }
    if (!st && dB) {
        sg::LowRank p = u.p;
        p.M = ad->B;
        p.transposed = 1;
        p.width = g.out;
        p.X = dy;
        p.x = y_pieces(g, T);
        p.out = dB;
        p.out_dtype = d_dtype;
        st = launched(sg::launch_grad(p, s), what);
    }
    if (!st && tiles) {
        set_adapted(g, ad, v.p.plan, &q, &d);
        q.A = dy;
        q.out = dx;
        q.out_dtype = dx_dtype;
        st = launched(sg::launch_adapted(q, d, s), what);
    } else if (!st && T && dx) {
        sg::LowRank p = v.p;
        p.M = ad->A;
        p.transposed = 1;  // (rank, in), its columns the output's
        p.width = g.in;
        p.x = x_pieces(g, T);
        p.base = base;
        p.out = dx;
        p.out_dtype = dx_dtype;
        p.out_ld = p.x.ld;
        p.out_rank = p.x.rank;
        st = launched(sg::launch_expand(p, s), what);
    }
    return st;
}

}  // namespace

extern "C" {

size_t sg_adapter_plan_ints(int64_t T, int n) {
    if (T < 0 || T > kMaxTokens || n < 1 || n > sg::kMaxAdapters) return 0;
    return (size_t)sg::plan_layout(T, n).ints;
}

sg_status sg_adapter_plan(const int32_t* which, int64_t T, int n, int32_t* plan, void* stream) {
    sg::last_error().clear();
    if (T < 0 || n < 1) return fail(SG_ERR_INVALID_ARG, "need T >= 0 and n >= 1");
    if (T > kMaxTokens || n > sg::kMaxAdapters)
        return fail(SG_ERR_UNSUPPORTED, "more than 2^25 tokens or %d adapters are not supported", sg::kMaxAdapters);
    if (!plan || (T && !which)) return fail(SG_ERR_INVALID_ARG, "which and plan must not be NULL");
    return launched(sg::launch_adapter_plan(which, T, n, plan, (hipStream_t)stream), "sg_adapter_plan");
}

size_t sg_adapted_workspace(const sg_layer* l, const sg_adapters* ad, int64_t T) {
    Geometry g;
    if (!l || !ad || T <= 0 || check_adapters(ad) || sg_layer_info(l, &g.out, &g.in, &g.mode, &g.S, &g.P, &g.dtype, &g.quantized))
        return 0;
    // the projection's fp32 result and what its own call needs, or the operands of U
    size_t own = g.column() ? 0 : up256((int64_t)sg_sharded_to_all_workspace(l, T)), ops = operands_bytes(T, ad->rank);
    sg::Grouped q;
    if (tile_product(l, g, T, false, false, &q)) {
        if (split_product(g, q) && split_bytes(q) > own) own = split_bytes(q);
        ops += weight_bytes(g);
    }
    const size_t base = up256(T * g.out * 4) + own;
    return half(g, ad, nullptr, T, true).bytes + (base > ops ? base : ops);
}

sg_status sg_adapted_all_to_sharded(const sg_layer* l, const sg_adapters* ad, const int32_t* plan, const void* x, int64_t T,
                                    void* y, int out_layout, int epilogue, sg_dtype y_dtype, void* workspace,
                                    size_t ws_bytes, void* stream) {
    sg::last_error().clear();
    Geometry g;
    if (sg_status st = check_call(l, SG_ALL_TO_SHARDED, ad, T, &g)) return st;
    if (out_layout != SG_OUT_FULL && out_layout != SG_OUT_SHARDED)
        return fail(SG_ERR_INVALID_ARG, "unknown output layout %d", out_layout);
    if (epilogue != SG_EPI_NONE && epilogue != SG_EPI_SWIGLU) return fail(SG_ERR_INVALID_ARG, "unknown epilogue %d", epilogue);
    if (epilogue == SG_EPI_SWIGLU && g.S != 2)
        return fail(SG_ERR_INVALID_ARG, "the SwiGLU epilogue needs a layer with segments = 2");
    return forward("sg_adapted_all_to_sharded", l, g, ad, plan, x, T, y, out_layout, epilogue, y_dtype, workspace, ws_bytes,
                   stream);
}

sg_status sg_adapted_sharded_to_all(const sg_layer* l, const sg_adapters* ad, const int32_t* plan, const void* x_partial,
                                    int64_t T, void* y, sg_dtype y_dtype, void* workspace, size_t ws_bytes, void* stream) {
    sg::last_error().clear();
    Geometry g;
    if (sg_status st = check_call(l, SG_SHARDED_TO_ALL, ad, T, &g)) return st;
    return forward("sg_adapted_sharded_to_all", l, g, ad, plan, x_partial, T, y, SG_OUT_FULL, SG_EPI_NONE, y_dtype,
                   workspace, ws_bytes, stream);
}

size_t sg_adapted_backward_workspace(const sg_layer* l, const sg_adapters* ad, int64_t T) {
    Geometry g;
    if (!l || !ad || T <= 0 || check_adapters(ad) || sg_layer_info(l, &g.out, &g.in, &g.mode, &g.S, &g.P, &g.dtype, &g.quantized))
        return 0;
    const size_t ops = operands_bytes(T, ad->rank);
    size_t base = up256(T * g.in * 4);
    sg::Grouped q;
    if (tile_product(l, g, T, true, false, &q) && split_product(g, q)) base += split_bytes(q);
    return half(g, ad, nullptr, T, true).bytes + half(g, ad, nullptr, T, false).bytes + (base > ops ? base : ops);
}

sg_status sg_adapted_all_to_sharded_backward(const sg_layer* l, const sg_adapters* ad, const int32_t* plan, const void* x,
                                             const void* dy, int64_t T, void* dx, sg_dtype dx_dtype, void* dA, void* dB,
                                             sg_dtype d_dtype, void* workspace, size_t ws_bytes, void* stream) {
    sg::last_error().clear();
    Geometry g;
    if (sg_status st = check_call(l, SG_ALL_TO_SHARDED, ad, T, &g)) return st;
    return backward("sg_adapted_all_to_sharded_backward", l, g, ad, plan, x, dy, T, dx, dx_dtype, dA, dB, d_dtype, workspace,
                    ws_bytes, stream);
}

sg_status sg_adapted_sharded_to_all_backward(const sg_layer* l, const sg_adapters* ad, const int32_t* plan,
                                             const void* x_partial, const void* dy, int64_t T, void* dx_partial,
                                             sg_dtype dx_dtype, void* dA, void* dB, sg_dtype d_dtype, void* workspace,
                                             size_t ws_bytes, void* stream) {
    sg::last_error().clear();
    Geometry g;
    if (sg_status st = check_call(l, SG_SHARDED_TO_ALL, ad, T, &g)) return st;
    return backward("sg_adapted_sharded_to_all_backward", l, g, ad, plan, x_partial, dy, T, dx_partial, dx_dtype, dA, dB,
                    d_dtype, workspace, ws_bytes, stream);
}

}  // extern "C"
