// Grouped products of a mixture of experts (experts.h, Grouped), and the
// layout of an expert layer's weights.
#include "experts.h"

namespace sg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

namespace {

// D = W (16 rows) x A (16 tokens): lane l holds column (token) l & 15 and rows
// 4 (l >> 4) .. + 3 of the 16 x 16 block
template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 w, u32x4 a, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, a), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, a),
                                                       c, 0, 0, 0);
}

// MXFP4 x MXFP4: 16 bytes a lane are 32 codes of one scale block; the scales
// are the low bytes of sw and sa
__device__ __forceinline__ f32x4 mfma_mx4(u32x4 w, uint32_t sw, u32x4 a, uint32_t sa, f32x4 c) {
    const i32x8 wv = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, c, 4, 4, 0, (int)sw, 0, (int)sa);
}

// eight E2M1 codes (one word, k order) times 2^(s - 127) -> eight bf16; exact
// but where the product leaves bf16's range.  Scale 255 (NaN) gives NaNs.
__device__ __forceinline__ u32x4 mx4_to_bf16(uint32_t w, float scale) {
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    return r;
}

constexpr uint32_t kOutside = 0xfffffff0u;  // byte offset past every buffer: reads zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)(uint32_t)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// eight 16-bit inputs k .. k + 7 of a row, zeros from kl on and for row < 0;
// any alignment
__device__ __forceinline__ u32x4 load8_any(const uint16_t* a, int64_t row, int64_t lda, int k, int kl) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = row >= 0 && k + e < kl ? a[row * lda + k + e] : 0;
    return u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
}

// the 16-column output block ob of row m: this lane's columns 4 (lane >> 4) .. + 3
__device__ __forceinline__ void store_block(const Grouped& p, int ob, int m, f32x4 v) {
    const int piece = ob / p.bps, j = ob - piece * p.bps;
    const int r = p.swiglu ? piece : piece / p.S;
    const int s = p.swiglu ? 0 : piece - r * p.S;
    const int c = 16 * j + 4 * ((threadIdx.x & 63) >> 4);
    if (c >= p.f) return;
    const int64_t o = (int64_t)r * p.o_rank + (int64_t)m * p.ldo + s * p.f + c;
    if (p.vec) {  // f is a multiple of 4
        if (p.out_dtype == SG_F32) {
            *(f32x4*)((float*)p.out + o) = v;
            return;
        }
        u32x2 w;
        if (p.out_dtype == SG_BF16) {
            w[0] = f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16);
            w[1] = f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16);
        } else {
            w[0] = f32_to_f16(v[0]) | ((uint32_t)f32_to_f16(v[1]) << 16);
            w[1] = f32_to_f16(v[2]) | ((uint32_t)f32_to_f16(v[3]) << 16);
        }
        *(u32x2*)((uint16_t*)p.out + o) = w;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (c + e < p.f) store_from_f32(p.out, p.out_dtype, o + e, v[e]);
}

// segment's first element of A
__device__ __forceinline__ int64_t seg_offset(const Grouped& p, int seg) {
    const int r = seg / p.a_pieces;
    return r * p.a_rank + (int64_t)(seg - r * p.a_pieces) * p.kl;
}

// weight block i of output block ob (swiglu: i 0 the gate rows, 1 the up rows)
__device__ __forceinline__ int weight_block(const Grouped& p, int ob, int i) {
    if (!p.swiglu) return ob;
    const int r = ob / p.bps;
    return 2 * r * p.bps + (ob - r * p.bps) + i * p.bps;
}

// ---------------------------------------------------------------------------
// Streaming kernel: few rows for each expert.  Bound by HBM, by reading the
// weights of the experts that have rows once.  Weights go from memory straight
// into the registers of the MFMA that uses them (a step of a 16-row block is 1
// KB contiguous, 16 bytes a lane); the rows of up to 16 MB tokens are the
// other operand.  Four waves: KS of them split the inputs of one group of NB
// output blocks (their sums are added in wave order through LDS), 4 / KS groups
// stand side by side.  Steps come in runs of four, a run of loads ahead.
// ---------------------------------------------------------------------------
template <int MODE, bool SWIGLU, int MB, int NB, int KS, bool AL>
__global__ __launch_bounds__(256) void grouped_stream_kernel(Grouped p) {
    constexpr int NG = 4 / KS, NW = SWIGLU ? 2 * NB : NB;
    constexpr bool MX = MODE >= G_MX4;
    constexpr int KST = MX ? 128 : 32;               // inputs of a step
    constexpr int AF = MODE == G_MX4 ? 4 : 1;        // 16-byte operands of a step and 16 rows
    __shared__ f32x4 red[KS > 1 ? (KS - 1) * NG * NW * MB * 64 : 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kw = wave % KS, ng = wave / KS;
    const int groups = (p.nout + NG * NB - 1) / (NG * NB);
    const int si = blockIdx.x / groups;
    const Slot s = find_slot(p.offsets, p.E, p.R, si, 16 * MB);
    if (s.e < 0) return;
    const int ob0 = ((blockIdx.x - si * groups) * NG + ng) * NB;

    const uint8_t* w[NW];
    const uint8_t* ws[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const int ob = min(ob0 + (SWIGLU ? i / 2 : i), p.nout - 1);
        const int wb = weight_block(p, ob, SWIGLU ? i & 1 : 0);
        w[i] = p.W + (int64_t)s.e * p.w_expert + (int64_t)wb * p.wsteps * 1024 + lane * 16;
        if constexpr (MX)
            ws[i] = p.wsc + (int64_t)s.e * p.wsc_expert + (int64_t)wb * mx4_scale_runs(p.wsteps) * 256 + lane * 4;
    }
    int row[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int m = 16 * b + (lane & 15);
        row[b] = m < s.nrows ? grouped_row(p.rows, p.kdiv, p.T, s.row0 + m) : -1;
    }

    const int sps = p.kpad / KST;  // steps of a segment
    const int steps = p.nseg * sps, runs = (steps + 3) / 4;
    const int run0 = runs * kw / KS, run1 = runs * (kw + 1) / KS;
    const int64_t a_bytes = MODE == G_MX4A4 ? (int64_t)p.T * (p.lda / 2) : ((int64_t)(p.T - 1) * p.lda + p.kl) * 2;

    auto load_a = [&](int st, int b, u32x4 (&a)[AF], uint32_t& sa) {
        const int seg = st / sps, k0 = (st - seg * sps) * KST;
        if constexpr (MODE == G_MX4A4) {
            const int k = k0 + 32 * (lane >> 4);
            const bool in = row[b] >= 0 && k < p.kl;
            const uint8_t* base = (const uint8_t*)p.A + seg_offset(p, seg) / 2;
            a[0] = load16(buffer(base, a_bytes), in ? (uint32_t)(row[b] * (p.lda / 2) + k / 2) : kOutside);
            const uint8_t* sb = p.a_scales + (int64_t)seg * p.T * (p.kl / 32);
            sa = in ? sb[(int64_t)row[b] * (p.kl / 32) + k / 32] : 127u;
        } else {
            const uint16_t* base = (const uint16_t*)p.A + seg_offset(p, seg);
            const int k = k0 + (MODE == G_MX4 ? 32 : 8) * (lane >> 4);
#pragma unroll
            for (int j = 0; j < AF; ++j) {
                if constexpr (AL)
                    a[j] = load16(buffer(base, a_bytes), row[b] >= 0 && k + 8 * j < p.kl
                                                             ? (uint32_t)((row[b] * p.lda + k + 8 * j) * 2)
                                                             : kOutside);
                else
                    a[j] = load8_any(base, row[b], p.lda, k + 8 * j, p.kl);
            }
        }
    };

    f32x4 acc[NW][MB];
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    u32x4 wf[4][NW], af[4][MB][AF];
    uint32_t as[4][MB], wsc[NW], wsn[NW];
    auto load_step = [&](int st, int u) {
        const int c = min(st, steps - 1);
#pragma unroll
        for (int i = 0; i < NW; ++i) wf[u][i] = __builtin_nontemporal_load((const u32x4*)(w[i] + (int64_t)c * 1024));
#pragma unroll
        for (int b = 0; b < MB; ++b) load_a(c, b, af[u][b], as[u][b]);
    };
    auto load_scales = [&](int run) {
        if constexpr (MX) {
            const int c = min(run, runs - 1);
#pragma unroll
            for (int i = 0; i < NW; ++i) wsn[i] = *(const uint32_t*)(ws[i] + (int64_t)c * 256);
        }
    };
    if (run0 < run1) {
        load_scales(run0);
#pragma unroll
        for (int u = 0; u < 4; ++u) load_step(run0 * 4 + u, u);
    }
    for (int run = run0; run < run1; ++run) {
#pragma unroll
        for (int i = 0; i < NW; ++i) wsc[i] = wsn[i];
        load_scales(run + 1);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (run * 4 + u < steps) {
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    if constexpr (MODE == G_MX4) {
                        const uint32_t sb = (wsc[i] >> (8 * u)) & 255u;
                        const float sc = e8m0_to_f32(sb);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const u32x4 wv = mx4_to_bf16(wf[u][i][j], sc);
#pragma unroll
                            for (int b = 0; b < MB; ++b) acc[i][b] = mfma16<false>(wv, af[u][b][j], acc[i][b]);
                        }
                    } else if constexpr (MODE == G_MX4A4) {
#pragma unroll
                        for (int b = 0; b < MB; ++b)
                            acc[i][b] = mfma_mx4(wf[u][i], wsc[i] >> (8 * u), af[u][b][0], as[u][b], acc[i][b]);
                    } else {
#pragma unroll
                        for (int b = 0; b < MB; ++b) acc[i][b] = mfma16<MODE == G_F16>(wf[u][i], af[u][b][0], acc[i][b]);
                    }
                }
            }
            if (run + 1 < run1) load_step((run + 1) * 4 + u, u);
        }
    }

    if constexpr (KS > 1) {
        if (kw > 0)
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int b = 0; b < MB; ++b)
                    red[((((kw - 1) * NG + ng) * NW + i) * MB + b) * 64 + lane] = acc[i][b];
        __syncthreads();
        if (kw > 0) return;
        for (int q = 0; q < KS - 1; ++q)
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int b = 0; b < MB; ++b) acc[i][b] += red[(((q * NG + ng) * NW + i) * MB + b) * 64 + lane];
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        if (ob0 + n >= p.nout) continue;
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            const int m = 16 * b + (lane & 15);
            if (m >= s.nrows) continue;
            f32x4 v;
            if constexpr (SWIGLU) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = silu_f32(acc[2 * n][b][e]) * acc[2 * n + 1][b][e];
            } else {
                v = acc[n][b];
            }
            store_block(p, ob0 + n, s.row0 + m, v);
        }
    }
}

// ---------------------------------------------------------------------------
// Tile kernel: 128 rows x 128 weight rows (SwiGLU: 64 gate and the 64 matching
// up rows; transposed: 128 columns of the weights), 64 contracted inputs a
// tile, four waves of 64 x 64, operands staged through registers into two LDS
// buffers.  The rows lie in LDS as 128-byte rows, chunks XOR-swizzled by
// (row >> 1) & 7; weight fragments as stored, 1 KB each.  Transposed, the
// contracted dimension runs down the weight's rows: ds_read_b64_tr_b16 hands
// each lane four rows of one column.
// ---------------------------------------------------------------------------
template <bool F16, bool SWIGLU, bool TRANS, bool AL>
__global__ __launch_bounds__(256) void grouped_tile_kernel(Grouped p, int slots, int tiles_n) {
    constexpr int TM = 128;
    __shared__ __attribute__((aligned(1024))) uint16_t sA[2][TM * 64], sW[2][16 * 512];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave_m = wave & 1, wave_n = wave >> 1;
    const int tile = xcd_remap(blockIdx.x, slots * tiles_n);
    constexpr int GM = 4;
    const int g = tile / (GM * tiles_n), first = g * GM, gsz = min(GM, slots - first);
    const int tin = tile - g * GM * tiles_n;
    const Slot s = find_slot(p.offsets, p.E, p.R, first + tin % gsz, TM);
    if (s.e < 0) return;
    const int nt = tin / gsz;  // n tile

    // rows this thread loads: (tid >> 3) + 32 i, chunk tid & 7
    int row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = (tid >> 3) + 32 * i;
        row[i] = m < s.nrows ? grouped_row(p.rows, p.kdiv, p.T, s.row0 + m) : -1;
    }
    const uint8_t* W = p.W + (int64_t)s.e * p.w_expert;
    const int kts = (p.kpad + 63) / 64, nkt = p.nseg * kts;
    const int64_t a_bytes = ((int64_t)(p.T - 1) * p.lda + p.kl) * 2;

    u32x4 ra[4], rw[4];
    auto load = [&](int kt) {
        const int seg = kt / kts, k0 = (kt - seg * kts) * 64;
        const uint16_t* base = (const uint16_t*)p.A + seg_offset(p, seg);
        const int k = k0 + 8 * (tid & 7);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (AL)
                ra[i] = load16(buffer(base, a_bytes),
                               row[i] >= 0 && k < p.kl ? (uint32_t)((row[i] * p.lda + k) * 2) : kOutside);
            else
                ra[i] = load8_any(base, row[i], p.lda, k, p.kl);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int f = 4 * i + wave;
            int64_t at;
            bool in = true;
            if constexpr (TRANS) {
                // fragment (block f >> 2 of the tile's four, step f & 3 of its four)
                const int kb = k0 / 16 + (f >> 2), st = nt * 4 + (f & 3);
                in = kb < p.kpad / 16 && st < p.wsteps;
                at = ((int64_t)(seg * (p.kpad / 16) + kb) * p.wsteps + st) * 1024;
            } else {
                // fragment (block f >> 1 of the tile's eight, step f & 1 of its two)
                int ob, half = 0;
                if constexpr (SWIGLU) ob = nt * 4 + (f >> 2), half = (f >> 1) & 1;
                else ob = nt * 8 + (f >> 1);
                const int st = (seg * p.kpad + k0) / 32 + (f & 1);
                at = ((int64_t)weight_block(p, min(ob, p.nout - 1), half) * p.wsteps + st) * 1024;
            }
            rw[i] = in ? *(const u32x4*)(W + at + lane * 16) : u32x4{0, 0, 0, 0};
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = (tid >> 3) + 32 * i;
            *(u32x4*)(sA[buf] + m * 64 + (((tid & 7) ^ ((m >> 1) & 7)) << 3)) = ra[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) *(u32x4*)(sW[buf] + (4 * i + wave) * 512 + lane * 8) = rw[i];
    };

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int c16 = lane >> 4, r16 = lane & 15;
    if (nkt > 0) {
        load(0);
        stage(0);
        __syncthreads();
        for (int t = 0; t < nkt; ++t) {
            const int buf = t & 1;
            if (t + 1 < nkt) load(t + 1);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                u32x4 wf[4], af[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (TRANS) {
                        // columns 16 (4 wave_n + i) .. of the tile; contracted rows 32 kk + 8 c16 ..
                        const int nb = 4 * wave_n + i;
                        const uint16_t* fr = sW[buf] + ((2 * kk + (c16 >> 1)) * 4 + (nb >> 1)) * 512;
                        const int ch = 2 * (nb & 1) + ((r16 & 3) >> 1);
                        const int rr = 8 * (c16 & 1) + (r16 >> 2);
                        const uint16_t* a0 = fr + (rr + 16 * ch) * 8 + 4 * (r16 & 1);
                        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (__attribute__((address_space(3))) s16x4*)a0);
                        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (__attribute__((address_space(3))) s16x4*)(a0 + 4 * 8));
                        const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
                        wf[i] = u32x4{l2[0], l2[1], h2[0], h2[1]};
                    } else {
                        wf[i] = *(const u32x4*)(sW[buf] + ((4 * wave_n + i) * 2 + kk) * 512 + lane * 8);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int m = wave_m * 64 + 16 * j + r16;
                    af[j] = *(const u32x4*)(sA[buf] + m * 64 + (((4 * kk + c16) ^ ((m >> 1) & 7)) << 3));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = mfma16<F16>(wf[i], af[j], acc[i][j]);
            }
            if (t + 1 < nkt) stage(buf ^ 1);
            __syncthreads();
        }
    }

    static_for<0, (SWIGLU ? 2 : 4)>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int ob = SWIGLU ? nt * 4 + wave_n * 2 + i : nt * 8 + wave_n * 4 + i;
        if (ob >= p.nout) return;
        static_for<0, 4>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            const int m = wave_m * 64 + 16 * j + r16;
            if (m >= s.nrows) return;
            f32x4 v;
            if constexpr (SWIGLU) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = silu_f32(acc[2 * i][j][e]) * acc[2 * i + 1][j][e];
            } else {
                v = acc[i][j];
            }
            store_block(p, ob, s.row0 + m, v);
        });
    });
}

// ---- layout -----------------------------------------------------------------
// where stored row n of an expert and stored input q come from (-1: padding)
__device__ __forceinline__ int64_t source_row(const ExpertsLayout& l, int64_t n) {
    const int64_t piece = n / (l.bps * 16), j = n - piece * l.bps * 16;
    if (j >= l.f) return -1;
    if (l.mode == SG_SHARDED_TO_ALL) return n;
    const int64_t r = piece / l.S, s = piece - r * l.S;
    return s * (l.out / l.S) + r * l.f + j;
}
__device__ __forceinline__ int64_t source_col(const ExpertsLayout& l, int64_t q) {
    const int64_t r = q / l.kpad, c = q - r * l.kpad;
    if (c >= l.kl) return -1;
    if (l.mode == SG_ALL_TO_SHARDED) return c;
    const int64_t part = l.in / l.S / l.P, s = c / part;
    return s * (l.in / l.S) + r * part + (c - s * part);
}

__global__ __launch_bounds__(256) void pack_kernel(uint16_t* dst, const uint16_t* src, ExpertsLayout l, int64_t frags) {
    const int64_t fr = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (fr >= frags) return;
    const int lane = threadIdx.x & 63;
    const int64_t st = fr % l.steps, b = (fr / l.steps) % l.blocks, e = fr / (l.steps * l.blocks);
    const int64_t row = source_row(l, b * 16 + (lane & 15)), q = st * 32 + 8 * (lane >> 4);
    const uint16_t* from = src + (e * l.out + row) * l.in;
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t c = row >= 0 ? source_col(l, q + i) : -1;
        h[i] = c >= 0 ? from[c] : 0;
    }
    *(u32x4*)(dst + fr * 512 + lane * 8) =
        u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
}

// (a scale block never straddles two segments' parts: the entry point checks)
__global__ __launch_bounds__(256) void pack_mx4_kernel(uint8_t* codes, uint8_t* scales, const uint8_t* src_codes,
                                                       const uint8_t* src_scales, ExpertsLayout l, int64_t frags) {
    const int64_t fr = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (fr >= frags) return;
    const int lane = threadIdx.x & 63;
    const int64_t st = fr % l.steps, b = (fr / l.steps) % l.blocks, e = fr / (l.steps * l.blocks);
    const int64_t row = source_row(l, b * 16 + (lane & 15));
    const int64_t c = row >= 0 ? source_col(l, st * 128 + 32 * (lane >> 4)) : -1;
    u32x4 v = {0, 0, 0, 0};
    uint8_t s = 127;
    if (c >= 0) {
        const uint8_t* from = src_codes + (e * l.out + row) * (l.in / 2) + c / 2;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = from[4 * i] | (from[4 * i + 1] << 8) | (from[4 * i + 2] << 16) | ((uint32_t)from[4 * i + 3] << 24);
        s = src_scales[(e * l.out + row) * (l.in / 32) + c / 32];
    }
    *(u32x4*)(codes + e * l.blocks * l.steps * 1024 + mx4_offset(b, st, l.steps) + lane * 16) = v;
    uint8_t* se = scales + e * l.blocks * mx4_scale_runs(l.steps) * 256;
    se[mx4_scale_offset(b, st, lane, l.steps)] = s;
    if (st == l.steps - 1)  // the rest of the last run is read and not used
        for (int64_t i = l.steps; i < mx4_scale_runs(l.steps) * 4; ++i) se[mx4_scale_offset(b, i, lane, l.steps)] = 127;
}

template <int MODE, bool SWIGLU, int MB, int NB, int KS, bool AL>
hipError_t stream_launch(const Grouped& p, hipStream_t s) {
    constexpr int per = 4 / KS * NB;
    const int64_t groups = (p.nout + per - 1) / per;
    const int64_t slots = p.R / (16 * MB) + (p.R < p.E ? p.R : p.E);
    if (groups * slots >= kMaxBlocks) return hipErrorInvalidConfiguration;
    launch(grouped_stream_kernel<MODE, SWIGLU, MB, NB, KS, AL>, dim3((unsigned)(groups * slots)), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int MODE, bool SWIGLU, bool AL>
hipError_t stream_mode(const Grouped& p, hipStream_t s) {
    constexpr int NB = SWIGLU ? 2 : 4;
    if (p.R <= (int64_t)16 * p.E) {
        if (p.nout <= 256) return stream_launch<MODE, SWIGLU, 1, NB / 2, 4, AL>(p, s);
        return stream_launch<MODE, SWIGLU, 1, NB, 1, AL>(p, s);
    }
    return stream_launch<MODE, SWIGLU, 2, NB, 1, AL>(p, s);
}

template <bool F16, bool SWIGLU, bool TRANS, bool AL>
hipError_t tile_launch(const Grouped& p, hipStream_t s) {
    const int64_t slots = p.R / 128 + (p.R < p.E ? p.R : p.E);
    const int64_t tiles_n = (p.nout + (SWIGLU ? 3 : 7)) / (SWIGLU ? 4 : 8);
    if (slots * tiles_n >= kMaxBlocks) return hipErrorInvalidConfiguration;
    launch(grouped_tile_kernel<F16, SWIGLU, TRANS, AL>, dim3((unsigned)(slots * tiles_n)), dim3(256), 0, s, p,
           (int)slots, (int)tiles_n);
    return hipGetLastError();
}

template <int MODE, bool AL>
hipError_t by_mode(const Grouped& p, hipStream_t s) {
    if constexpr (MODE < G_MX4) {
        constexpr bool F = MODE == G_F16;
        if (p.transposed) return tile_launch<F, false, true, AL>(p, s);
        if (p.R > (int64_t)32 * p.E)
            return p.swiglu ? tile_launch<F, true, false, AL>(p, s) : tile_launch<F, false, false, AL>(p, s);
    }
    return p.swiglu ? stream_mode<MODE, true, AL>(p, s) : stream_mode<MODE, false, AL>(p, s);
}

}  // namespace

hipError_t launch_grouped(const Grouped& p, hipStream_t s) {
    // 16-byte loads of eight inputs need aligned rows that end on eight
    const bool al = (uintptr_t)p.A % 16 == 0 && p.lda % 8 == 0 && p.a_rank % 8 == 0 && p.kl % 8 == 0;
    switch (p.mode) {
    case G_BF16: return al ? by_mode<G_BF16, true>(p, s) : by_mode<G_BF16, false>(p, s);
    case G_F16: return al ? by_mode<G_F16, true>(p, s) : by_mode<G_F16, false>(p, s);
    case G_MX4: return al ? by_mode<G_MX4, true>(p, s) : by_mode<G_MX4, false>(p, s);
    default: return by_mode<G_MX4A4, true>(p, s);
    }
}

hipError_t experts_pack(void* dst, const void* src, const ExpertsLayout& l, hipStream_t s) {
    const int64_t frags = l.E * l.blocks * l.steps;
    launch(pack_kernel, dim3((unsigned)((frags + 3) / 4)), dim3(256), 0, s, (uint16_t*)dst, (const uint16_t*)src, l,
           frags);
    return hipGetLastError();
}

hipError_t experts_pack_mx4(uint8_t* codes, uint8_t* scales, const uint8_t* src_codes, const uint8_t* src_scales,
                            const ExpertsLayout& l, hipStream_t s) {
    const int64_t frags = l.E * l.blocks * l.steps;
    launch(pack_mx4_kernel, dim3((unsigned)((frags + 3) / 4)), dim3(256), 0, s, codes, scales, src_codes, src_scales, l,
           frags);
    return hipGetLastError();
}

}  // namespace sg
