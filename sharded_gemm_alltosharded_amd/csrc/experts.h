// Mixture-of-experts products: what the entry points (experts_api.hip) hand to
// the grouped kernels (experts.hip, experts_dw.hip).
#pragma once

#include "internal.h"

namespace sg {

// ---------------------------------------------------------------------------
// One grouped product.  The rows m = 0 .. R-1 come grouped by expert: rows
// offsets[e] .. offsets[e+1] - 1 belong to expert e (offsets null: E == 1 and
// every row is its).  For a row m of expert e
//
//   out[m][n] = sum_s sum_{k < kl} A_s[row(m)][k] W_e[n][s kpad + k]
//
//  * A_s: segment s of the input, part s % a_pieces (each kl columns) of rank
//    s / a_pieces, whose rows start at A + rank * a_rank elements, row stride
//    lda; row(m) = m, or rows[m] / kdiv with a gather map (an index
//    outside 0 .. T-1 reads zeros).  Rows are read below T.
//  * W_e: fragment-major, 16-row blocks of `wsteps` steps: 16-bit weights,
//    32 inputs a step (frag_offset); MXFP4 weights, 128 inputs a step
//    (mx4_offset, mx4_scale_offset).  A segment's inputs are padded with zero
//    weights to kpad, a multiple of 128 (MXFP4) or 64.
//  * transposed (dx of the layer): W_e's rows are the contracted dimension:
//    out[m][n] = sum_s sum_{k < kl} A_s[m][k] W_e[s kpad + k][n], kpad a
//    multiple of 16 and segment s stored in rows s kpad .. + kl.
//  * Output columns come in 16-column blocks: block b lies in piece b / bps at
//    column 16 (b % bps) of its f columns; piece i is part i % S of rank i / S.
//    Rank r's columns start at out + r * o_rank, row stride ldo.  The last `pad`
//    of the f columns are stored as zeros.
//  * swiglu: pieces 2r and 2r + 1 are rank r's gate and up rows; output block b
//    is block b % bps of rank b / bps.
// Rows behind offsets[E] are not written.
// ---------------------------------------------------------------------------
enum GroupedMode { G_BF16 = 0, G_F16 = 1, G_MX4 = 2, G_MX4A4 = 3 };

struct Grouped {
    int mode;  // GroupedMode: 16-bit x 16-bit, MXFP4 weights x bf16, MXFP4 x MXFP4
    const void* A;
    const uint8_t* a_scales;  // G_MX4A4: E8M0, one per 32 inputs, row stride kl / 32
    int64_t lda, a_rank;      // elements
    int a_pieces, nseg, kl, kpad;
    const int32_t* offsets;
    const int32_t* rows;
    int kdiv, T, R, E;
    const uint8_t* W;
    int64_t w_expert;  // bytes from one expert's weights to the next
    const uint8_t* wsc;
    int64_t wsc_expert;
    int wsteps;  // steps of a 16-row block
    int transposed, swiglu;
    int bps, f, pad, S, nout;  // output blocks (of pairs with swiglu): nout
    void* out;
    int out_dtype;
    int64_t ldo, o_rank;
};

// Codes of an MXFP4 layer: the 16-row x 128-input block (block b, step st) is
// 1 KB, lane l owning 16 bytes: the 32 codes of row l & 15, inputs 128 st + 32
// (l >> 4) .. + 31, which is one scale block and its operand of one
// v_mfma_scale_f32_16x16x128; input 2i in the low half of byte i.
__host__ __device__ inline int64_t mx4_offset(int64_t block, int64_t st, int64_t nsteps) {
    return (block * nsteps + st) * 1024;
}
// Their scales: for a 16-row block and a run of four steps 16 rows x 16 bytes,
// a row's four steps adjacent, four scale blocks (bytes) each.
__host__ __device__ inline int64_t mx4_scale_runs(int64_t nsteps) { return (nsteps + 3) / 4; }
__host__ __device__ inline int64_t mx4_scale_offset(int64_t block, int64_t st, int row, int64_t nsteps) {
    return ((block * mx4_scale_runs(nsteps) + (st >> 2)) * 16 + row) * 16 + (st & 3) * 4;
}

// workgroups of 256 threads that one launch may have (2^32 threads)
constexpr int64_t kMaxBlocks = 1 << 24;
// hipErrorInvalidConfiguration: more workgroups than a launch may have
hipError_t launch_grouped(const Grouped& p, hipStream_t s);

// Weight gradients of a grouped layer: out[e][r][o][i] = sum over expert e's
// rows m of G_r[m][o] X_r[row(m)][i]; zeros for an expert without rows.
struct GroupedDw {
    int f16;
    const void* G;
    int64_t ldg, g_rank;
    const void* X;
    int64_t ldx, x_rank;
    const int32_t* offsets;
    const int32_t* rows;
    int kdiv, T, R, E, P, O, I;
    uint32_t kmul;  // set by the launch
    int kshift;
    int xw;         // columns of X that may be read: I, or more where its rows are padded
    int of, ofp;    // pieces of the O columns of G: of of each ofp are the layer's (ofp 0: all)
    void* out;
    int out_dtype;
};
hipError_t launch_grouped_dw(const GroupedDw& p, hipStream_t s);

// Row-major expert weights -> the kernels' layout.
struct ExpertsLayout {
    int mode, S, P;       // sg_mode, segments, ranks
    int64_t E, out, in;   // the unsharded layer
    int64_t f, bps;       // columns and 16-row blocks of a piece (all-to-sharded: out / S / P; else out)
    int64_t kl, kpad;     // inputs of a segment, padded
    int64_t blocks, steps;
};
hipError_t experts_pack(void* dst, const void* src, const ExpertsLayout& l, hipStream_t s);
hipError_t experts_pack_mx4(uint8_t* codes, uint8_t* scales, const uint8_t* src_codes, const uint8_t* src_scales,
                            const ExpertsLayout& l, hipStream_t s);

// Routing (route.hip)
struct Route {
    const void* logits;
    int64_t ld;
    int dtype, T, E, k, normalize;
    float* weights;
    int32_t *experts, *offsets, *rows, *slots;
    int32_t* ws;
};
constexpr int kRouteMaxExperts = 1024, kRouteMaxK = 16;
size_t route_workspace_ints(int64_t T, int E, int k);
hipError_t launch_route(const Route& r, hipStream_t s);
hipError_t launch_route_backward(const Route& r, const float* dweights, void* dlogits, int64_t ldd, hipStream_t s);
hipError_t launch_combine(const void* y, int y_dtype, const int32_t* slots, const float* weights, int64_t T, int k,
                          int64_t D, int64_t R, void* out, int out_dtype, hipStream_t s);
hipError_t launch_combine_backward(const void* dout, const void* y, int dtype, const int32_t* slots,
                                   const float* weights, int64_t T, int k, int64_t D, int64_t R, void* dy, float* dw,
                                   hipStream_t s);
// swiglu on (rows, 2 f) -> (rows, f)
hipError_t launch_swiglu(const void* gu, int dtype, int64_t rows, int64_t f, void* h, hipStream_t s);
hipError_t launch_swiglu_backward(const void* gu, const void* dh, int dtype, int64_t rows, int64_t f, void* dgu,
                                  hipStream_t s);

// MXFP4 (mxfp4.hip)
hipError_t launch_quantize_mxfp4(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s);
hipError_t launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* x,
                                   int dtype, hipStream_t s);

// MX FP8 activations (mxfp8.hip); a row of n values has mx8_blocks(n) scales
__host__ __device__ inline int64_t mx8_blocks(int64_t n) { return (n + 31) / 32; }
hipError_t launch_quantize_mxfp8(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s);
// kept16: values that were kept from dtype's own (what E4M3 rounds beyond fp16 is fp16's largest)
hipError_t launch_dequantize_mxfp8(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* x,
                                   int64_t ld, int dtype, bool kept16, hipStream_t s);
// gate|up rows to h (rows of fp >= f columns, those behind f zeros) and what is kept,
// where the product's epilogue does not do it
hipError_t launch_gated_keep(const float* gu, int64_t P, int64_t R, int64_t f, int64_t fp, const int32_t* offsets, int E,
                             void* h, int f16, uint8_t* codes, uint8_t* scales, hipStream_t s);

#ifdef __HIPCC__
#define ALWAYS_INLINE __attribute__((always_inline))

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// ---- device helpers --------------------------------------------------------
// D = rows x columns of 16: lane l gives 32 (k) / 4 = 8 values of row l & 15 of
// w and of column l & 15 of a, and holds rows 4 (l >> 4) .. + 3 of column l & 15
template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 w, u32x4 a, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, a), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, a),
                                                       c, 0, 0, 0);
}

constexpr uint32_t kOutside = 0xfffffff0u;  // byte offset past every buffer: reads zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)(uint32_t)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// one load of 16 (4) bytes a lane straight into LDS at to + 16 (4) lane
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint8_t* to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint8_t* to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 4, voff, soff, 0, 0);
}
// every load of this wave but the last N, and every LDS write, has landed
template <int N = 0>
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}
// ... and, behind the barrier, of every wave of the workgroup; no access to
// memory is moved over it
template <int N = 0>
__device__ __forceinline__ void stage_barrier() {
    asm volatile("" ::: "memory");
    wait_loads<N>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ u32x2 read_tr(const uint8_t* p) {
    return __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// eight 16-bit inputs k .. k + 7 of a row, zeros from n on and for row < 0; any
// alignment (a global load takes every address).  Row 0 is there, n >= 1.  The
// last chunk of a row is read from the row's last eight inputs and shifted, so
// that no lane branches and no load leaves its row.
__device__ __forceinline__ u32x4 load8_any(const uint16_t* a, int64_t row, int64_t ld, int k, int n) {
    const bool in = row >= 0 && k < n;
    if (n < 8) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = in && k + e < n ? a[row * ld + k + e] : 0;
        return u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
    }
    const int over = max(k + 8 - n, 0);  // inputs of the chunk past the row's end
    uint64_t v[2];
    __builtin_memcpy(v, a + (in ? row * ld + k - over : 0), 16);
    const uint64_t lo = over & 4 ? v[1] : v[0], hi = over & 4 ? 0 : v[1];
    const int sh = 16 * (over & 3);
    const uint64_t x = in ? (lo >> sh) | ((hi << 1) << (63 - sh)) : 0, y = in ? hi >> sh : 0;
    return u32x4{(uint32_t)x, (uint32_t)(x >> 32), (uint32_t)y, (uint32_t)(y >> 32)};
}

// four (eight) results in adjacent columns, `left` of them in the row; any alignment
template <int DT, int N>
__device__ __forceinline__ void store_cols(void* out, int64_t at, const float (&v)[N], int left) {
    if (left < N) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < left) store_from_f32(out, DT, at + e, v[e]);
    } else if constexpr (DT == SG_F32) {
        __builtin_memcpy((float*)out + at, v, 4 * N);
    } else {
        uint32_t w[N / 2];
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            const uint32_t lo = DT == SG_BF16 ? f32_to_bf16(v[2 * e]) : f32_to_f16(v[2 * e]);
            const uint32_t hi = DT == SG_BF16 ? f32_to_bf16(v[2 * e + 1]) : f32_to_f16(v[2 * e + 1]);
            w[e] = lo | (hi << 16);
        }
        __builtin_memcpy((uint16_t*)out + at, w, 2 * N);
    }
}

// eight values of any type in adjacent columns, `left` of them in the row (the
// others zero); any alignment
template <int DT>
__device__ __forceinline__ void load_cols(const void* x, int64_t at, float (&v)[8], int64_t left) {
    if (left < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < left ? load_as_f32(x, DT, at + e) : 0.f;
    } else if constexpr (DT == SG_F32) {
        __builtin_memcpy(v, (const float*)x + at, 32);
    } else {
        uint16_t h[8];
        __builtin_memcpy(h, (const uint16_t*)x + at, 16);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = DT == SG_BF16 ? bf16_to_f32(h[e]) : f16_to_f32(h[e]);
    }
}

// ---- MX FP8 blocks (mxfp8.hip has the format) -------------------------------
// magnitudes compare like their bit patterns; infinities and NaNs are the largest
__device__ __forceinline__ uint32_t mx8_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ bool mx8_bad(uint32_t m) { return m >= 0x7f800000u; }
// exponent of a block whose largest magnitude has the bits m: 448 = 1.75 2^8
// (zeros and subnormals fall below -127)
__device__ __forceinline__ int mx8_exponent(uint32_t m) {
    return max((int)(m >> 23) - 135 + ((m & 0x7fffffu) > 0x600000u), -127);
}
__device__ __forceinline__ uint8_t mx8_scale(uint32_t m) { return mx8_bad(m) ? 255 : (uint8_t)(mx8_exponent(m) + 127); }
// four codes: x 2^-e is exact (a power of two) unless it falls below 2^-126, where
// the code is 0 anyway
__device__ __forceinline__ uint32_t mx8_codes(float a, float b, float c, float d, int e) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(a, -e), ldexpf(b, -e), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(c, -e), ldexpf(d, -e), w, true);
}
__device__ __forceinline__ void mx8_values(uint32_t w, int s, float& a, float& b, float& c, float& d) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    const float nan = __builtin_nanf("");
    a = s == 255 ? nan : ldexpf(lo[0], s - 127), b = s == 255 ? nan : ldexpf(lo[1], s - 127);
    c = s == 255 ? nan : ldexpf(hi[0], s - 127), d = s == 255 ? nan : ldexpf(hi[1], s - 127);
}

// h = g s u with s = 1 / (1 + e^-g), and its gradient, for 16-bit results:
// dg = dh u s (1 + g (1 - s)), du = dh g s.  s from e^-|g|, which cannot overflow, on
// the hardware's exponential: the square of 2^(t / 2), t = -|g| log2 e rounded, so that
// it is not flushed before it leaves fp32's subnormals, times 1 + r ln 2 for the r that
// t's rounding left.  Off by 2^-19 of itself at most (grouped_tile.h, swiglu4).  e^-|g| is
// 0 long before |g| = 256; beyond 2^127.5 t would be infinite, and r not a number.
__device__ __forceinline__ void swiglu_grad(float g, float u, float dh, float& dg, float& du, float& h) {
    const float z = fminf(fabsf(g), 256.f), t = -1.44269504f * z, half = __builtin_amdgcn_exp2f(0.5f * t), e2 = half * half;
    const float e = fmaf(e2 * fmaf(-1.44269504f, z, -t), 0.693147181f, e2);
    const float s = (g < 0.f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e), a = g * s;
    dg = dh * u * s * (1.0f + g * (1.0f - s));
    du = dh * a;
    h = a * u;
}

struct Slot {
    int e, row0, nrows;  // expert (-1: none), first row, rows of the tile (at most TM)
};

// The tiles of TM rows that the experts' rows make up, counting expert after
// expert.  Every lane of the wave takes part and gets the same answers; the
// offsets are clamped to 0 .. R, so that no content of theirs leads out of the
// arrays.  Up to 64 experts the offsets are read once, one a lane.
struct SlotMap {
    const int32_t* offsets;
    int E, R, TM;
    int b, n, t, sum;  // this lane's expert: first row, rows, tiles, tiles up to and with it

    __device__ __forceinline__ SlotMap(const int32_t* o, int experts, int rows, int tile)
        : offsets(o), E(experts), R(rows), TM(tile), b(0), n(0), t(0), sum(0) {
        if (offsets) read(0);
    }
    __device__ __forceinline__ void read(int e0) {
        const int lane = threadIdx.x & 63, e = e0 + lane;
        b = n = 0;
        if (e < E) {
            b = min(max(offsets[e], 0), R);
            n = max(min(offsets[e + 1], R) - b, 0);
        }
        t = (n + TM - 1) / TM;
        sum = t;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int v = __shfl_up(sum, d);
            if (lane >= d) sum += v;
        }
    }
    __device__ __forceinline__ int count() {
        if (!offsets) return (R + TM - 1) / TM;
        int total = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            if (E > 64) read(e0);
            total += __shfl(sum, 63);
        }
        return __builtin_amdgcn_readfirstlane(total);
    }
    __device__ __forceinline__ Slot find(int slot) {
        if (!offsets) {
            const int r0 = slot * TM;
            return r0 < R ? Slot{0, r0, min(TM, R - r0)} : Slot{-1, 0, 0};
        }
        int before = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            if (E > 64) read(e0);
            const uint64_t hit = __ballot(before + sum > slot);
            if (hit) {
                const int l = __builtin_ctzll(hit);
                const int first = before + __shfl(sum, l) - __shfl(t, l);
                const int row = __builtin_amdgcn_readfirstlane((slot - first) * TM);
                const int bb = __builtin_amdgcn_readfirstlane(__shfl(b, l));
                const int nn = __builtin_amdgcn_readfirstlane(__shfl(n, l));
                // (falling offsets can count more tiles than an int holds)
                if (row < 0 || row >= nn) return Slot{-1, 0, 0};
                return Slot{__builtin_amdgcn_readfirstlane(e0 + l), bb + row, min(TM, nn - row)};
            }
            before += __shfl(sum, 63);
        }
        return Slot{-1, 0, 0};
    }
};

// input row of grouped row m (-1: reads zeros)
__device__ __forceinline__ int grouped_row(const int32_t* rows, int kdiv, int T, int m) {
    if (!rows) return m < T ? m : -1;
    const int s = rows[m];
    const int t = s / kdiv;
    return s >= 0 && t < T ? t : -1;
}
#endif

}  // namespace sg
