// The grouped tile kernel (experts.h, Grouped): its code, and the choice of a tile.
// experts.hip has the products that store their sums, experts_gated.hip those of the
// gated block, adapters_tile.hip those with low-rank adapters beside them.
#pragma once

#include "adapters.h"
#include "gated.h"

namespace sg {

typedef int i32x8 __attribute__((ext_vector_type(8)));

namespace {

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

// silu(g) u.  For 16-bit results (NEAR) on the hardware's exponential and
// reciprocal: e^-z = 2^t 2^r with t = -z log2 e rounded and r what the rounding
// left.  r knows log2 e to 1.93e-8 (its own fp32 rounding), so e^-z is off by
// 1.93e-8 ln 2 |z|, at most 1.2e-6 = 20 half steps of fp32 where it is finite, and
// a few half steps of the instructions: below 2^-19, where half a step of a
// 16-bit result is 2^-11 or more.  Beyond |t| = 126 r is left out: 2^t then tells z
// from 0 (t < 0), or silu is below 90 * 2^-126 (t > 0), where 2^t may be infinite,
// silu 0, and an r of 0 times it a NaN.
template <bool NEAR>
__device__ __forceinline__ f32x4 swiglu4(f32x4 g, f32x4 u) {
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (NEAR) {
            const float z = g[i], t = -1.44269504f * z;
            float e = __builtin_amdgcn_exp2f(t);
            if (fabsf(t) < 126.f) e = fmaf(e * fmaf(-1.44269504f, z, -t), 0.693147181f, e);
            v[i] = z * __builtin_amdgcn_rcpf(1.0f + e) * u[i];
        } else {
            v[i] = silu_f32(g[i]) * u[i];
        }
    }
    return v;
}

// Stores a wave's N x M result blocks: value(i, j) is this lane's four columns
// 4 (lane >> 4) .. + 3 of output block ob0 + i, row row0 + 16 j + (lane & 15).
// PAD: columns behind the piece's own may be asked for (p.pad; only SwiGLU has them).
// to_row(j): the output row of this lane's row of row block j.
template <int DT, bool PAD, int N, int M, typename F, typename R>
__device__ __forceinline__ void store_typed(const Grouped& p, int ob0, int row0, int nrows, F&& value, R&& to_row) {
    const int lane = threadIdx.x & 63;
    static_for<0, N>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int ob = ob0 + i;
        if (ob >= p.nout) return;
        const int piece = ob / p.bps, blk = ob - piece * p.bps;
        const int r = p.swiglu ? piece : piece / p.S, s = p.swiglu ? 0 : piece - r * p.S;
        const int c = 16 * blk + 4 * (lane >> 4);
        if (c >= p.f) return;
        const int64_t base = (int64_t)r * p.o_rank + s * p.f + c;
        const int live = p.f - p.pad - c;
        static_for<0, M>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            const int m = 16 * j + (lane & 15);
            if (m >= nrows) return;
            const f32x4 q = value(ic, jc, std::bool_constant<DT != SG_F32>{});
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = !PAD || e < live ? q[e] : 0.f;
            store_cols<DT>(p.out, base + (int64_t)to_row(jc) * p.ldo, v, p.f - c);
        });
    });
}
template <bool PAD, int N, int M, typename F, typename R>
__device__ __forceinline__ void store_blocks(const Grouped& p, int ob0, int row0, int nrows, F&& value, R&& to_row) {
    if (p.out_dtype == SG_BF16) store_typed<SG_BF16, PAD, N, M>(p, ob0, row0, nrows, value, to_row);
    else if (p.out_dtype == SG_F16) store_typed<SG_F16, PAD, N, M>(p, ob0, row0, nrows, value, to_row);
    else store_typed<SG_F32, PAD, N, M>(p, ob0, row0, nrows, value, to_row);
}
template <bool PAD, int N, int M, typename F>
__device__ __forceinline__ void store_blocks(const Grouped& p, int ob0, int row0, int nrows, F&& value) {
    store_blocks<PAD, N, M>(p, ob0, row0, nrows, value,
                            [&](auto jc) { return row0 + 16 * decltype(jc)::value + (int)(threadIdx.x & 15); });
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
// Tile kernel: TM rows x BN weight rows (SwiGLU: BN / 2 gate and the BN / 2
// matching up rows; transposed: BN columns of the weights), 2 x 4 waves, two to
// four LDS stages.  Bound by the matrix unit for many rows of an expert.
//
// A k tile is 64 inputs (MXFP4 weights: 128; MXFP4 x MXFP4: 256, the same 128
// bytes a row).  Its operands go from memory straight into the stage that the
// k tile before left (with three or four stages, two or three k tiles ahead): one
// barrier a k tile, behind which every wave's loads of it have landed; the next
// loads are issued between the two halves' operand reads and MFMAs.  With two
// waves a SIMD the reads of one run beside the MFMAs of the other; a raised wave
// priority around the MFMAs keeps them back to back (256 x 256, 8192 x 28672 x
// 4096: 1.08 -> 1.28 PFLOP/s, where the vendor library's product of that size
// reaches 1.37).  Each stage is an array of its own, so that the compiler sees that reads
// of one do not wait for the loads into the other.
//
// LDS: rows of A as 128 bytes (MXFP4 weights: 256), 16-byte chunks
// XOR-swizzled by (row >> 1) & 7 (row & 15), so that the sixteen rows of an
// operand read spread over all banks; weight fragments as stored, 1 KB each.
// Transposed, the contracted dimension runs down the weight's rows:
// ds_read_b64_tr_b16 hands each lane four rows of one column, and the odd
// chunks of a fragment are stored four rows on, so that the two chunks of a
// read lie in different banks.
// ---------------------------------------------------------------------------
template <int MODE, int TM, int BN>
struct TileShape {
    static constexpr int ROWB = MODE == G_MX4 ? 256 : 128;  // bytes of a row of A in LDS
    static constexpr int FPB = MODE == G_MX4 ? 1 : 2;       // fragments of a weight block
    static constexpr int A = TM * ROWB, W = BN * FPB * 64;  // bytes of a stage
    // scales of a stage, in words: four a weight row and step, four a row of A and step
    static constexpr int SW = MODE >= G_MX4 ? BN * FPB : 1, SA = MODE == G_MX4A4 ? TM * 2 : 1;
};

template <int NS>
struct Stages {
    uint8_t *A[NS], *W[NS];
    uint32_t *SW[NS], *SA[NS];
    uint8_t* M;  // adapt_blocks'
};

// ---- the gated block's epilogues (gated.h) ------------------------------------
// Stores the kept gate and up rows of a wave's output blocks ob0 .. (of a rank's f
// columns each) in MX FP8, and h.  A scale block is two output blocks.  NO == 2: one
// wave has both, a lane eight adjacent columns of them (grouped_tile, PERM).  NO == 1:
// two adjacent waves have them, which exchange their rows' maxima through `lds`, and h
// is left to store_blocks.  (bps is even, or there is one rank: a pair never straddles
// two.)  Bound by the product in front of it: 4096 tokens of 4096 inputs, 28672 gate|up
// rows, 814 us with it, 763 with SwiGLU and nothing kept, 901 for storing the sums.
template <bool F16, int NO, int NBM, int WN, typename Acc>
__device__ __forceinline__ void keep_blocks(const Grouped& p, const Gated& g, int ob0, int row0, int nrows, Acc& acc,
                                            uint32_t* lds) {
    static_assert(NO == 1 || NO == 2, "output blocks of a wave");
    constexpr int W = 4 * NO;  // columns of a lane
    const int lane = threadIdx.x & 63, r16 = lane & 15, c16 = lane >> 4, wave = threadIdx.x >> 6;
    const int r = ob0 / p.bps, blk0 = ob0 - r * p.bps, c = 16 * blk0 + W * c16;
    const int left = ob0 < p.nout ? g.f - c : 0;  // this lane's columns in the row
    const int nb = (int)mx8_blocks(g.f);
    uint32_t top[2][NBM];
    static_for<0, 2>([&](auto hc) ALWAYS_INLINE {
        constexpr int h = decltype(hc)::value;
        static_for<0, NBM>([&](auto jc) ALWAYS_INLINE {
            constexpr int j = decltype(jc)::value;
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < W; ++e) m = e < left ? max(m, mx8_bits(acc[2 * (e >> 2) + h][j][e & 3])) : m;
            m = max(m, (uint32_t)__shfl_xor((int)m, 16));
            top[h][j] = max(m, (uint32_t)__shfl_xor((int)m, 32));
        });
    });
    if constexpr (NO == 1) {
        static_assert(WN % 2 == 0, "wave ^ 1 is the neighbour in the tile's columns");
        __syncthreads();  // every wave has read its last operands
        auto at = [&](int w, int h, int j) { return ((w * NBM + j) * 2 + h) * 16 + r16; };
#pragma unroll
        for (int j = 0; j < NBM; ++j)
            if (c16 < 2) lds[at(wave, c16, j)] = c16 ? top[1][j] : top[0][j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NBM; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) top[h][j] = max(top[h][j], lds[at(wave ^ 1, h, j)]);
    }
    static_for<0, NBM>([&](auto jc) ALWAYS_INLINE {
        constexpr int j = decltype(jc)::value;
        const int m = 16 * j + r16;
        if (m >= nrows || ob0 >= p.nout) return;
        const int64_t row = (int64_t)r * p.R + row0 + m;
        static_for<0, 2>([&](auto hc) ALWAYS_INLINE {
            constexpr int h = decltype(hc)::value;
            const uint32_t t = top[h][j];
            const int e = mx8_exponent(t);
            uint32_t w[NO];
#pragma unroll
            for (int i = 0; i < NO; ++i) {
                const f32x4 v = acc[2 * i + h][j];
                w[i] = mx8_bad(t) ? 0u : mx8_codes(v[0], v[1], v[2], v[3], e);
            }
            put_bytes(g.codes + (row * 2 + h) * g.f + c, w, left);
            if (c16 == h && (NO == 2 || (blk0 & 1) == 0)) g.scales[(row * 2 + h) * nb + blk0 / 2] = mx8_scale(t);
        });
        if constexpr (NO == 2) {
            if (c >= p.f) return;
            const f32x4 a = swiglu4<true>(acc[0][j], acc[1][j]), b = swiglu4<true>(acc[2][j], acc[3][j]);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < left ? (e < 4 ? a[e] : b[e - 4]) : 0.f;
            store_cols<F16 ? SG_F16 : SG_BF16>(p.out, r * p.o_rank + (int64_t)(row0 + m) * p.ldo + c, v, p.f - c);
        }
    });
}

// The sums are dh: with the kept gate and up rows, the gradient of those (out, rows of
// two pieces of p.f columns, of which those behind g.f are zeros) and h.  A lane has 4 N
// adjacent columns (grouped_tile, PERM), all of one scale block, so that codes move in
// accesses of 8 or 16 bytes: with four-byte ones (columns in the sums' own order) product
// and end took 752 us, the product and a kernel of its own 626, this 592 (4096 rows of
// 4096 x 14336).
template <bool F16, int N, int NBM, typename Acc>
__device__ __forceinline__ void grad_blocks(const Grouped& p, const Gated& g, int ob0, int row0, int nrows, Acc& acc) {
    constexpr int DT = F16 ? SG_F16 : SG_BF16, W = 4 * N;
    if (nrows <= 0 || ob0 >= p.nout) return;
    const int lane = threadIdx.x & 63;
    const int nb = (int)mx8_blocks(g.f);
    const int r = ob0 / p.bps, c = 16 * (ob0 - r * p.bps) + W * (lane >> 4);
    if (c >= p.f) return;
    const int live = g.f - c;
    constexpr int JB = NBM < 4 ? NBM : 4;  // row blocks whose codes are out at once
    static_for<0, NBM / JB>([&](auto bc) ALWAYS_INLINE {
        constexpr int j0 = decltype(bc)::value * JB;
        uint32_t gw[JB][N], uw[JB][N];
        int gs[JB], us[JB];
        static_for<0, JB>([&](auto jc) ALWAYS_INLINE {
            constexpr int j = decltype(jc)::value;
            const int m = 16 * (j0 + j) + (lane & 15);
            const int64_t row = ((int64_t)r * p.R + row0 + (m < nrows ? m : 0)) * 2;
            const int b = min(c / 32, nb - 1);
            get_bytes(g.codes + row * g.f + c, gw[j], live);
            get_bytes(g.codes + (row + 1) * g.f + c, uw[j], live);
            gs[j] = g.scales[row * nb + b];
            us[j] = g.scales[(row + 1) * nb + b];
        });
        static_for<0, JB>([&](auto jc) ALWAYS_INLINE {
            constexpr int j = decltype(jc)::value;
            const int m = 16 * (j0 + j) + (lane & 15);
            if (m >= nrows) return;
            const int64_t row = (int64_t)r * p.R + row0 + m;
            static_for<0, N / 2>([&](auto ic) ALWAYS_INLINE {  // eight columns
                constexpr int i = 2 * decltype(ic)::value;
                float gv[8], uv[8], dg[8], du[8], h[8];
                mx8_values(gw[j][i], gs[j], gv[0], gv[1], gv[2], gv[3]);
                mx8_values(gw[j][i + 1], gs[j], gv[4], gv[5], gv[6], gv[7]);
                mx8_values(uw[j][i], us[j], uv[0], uv[1], uv[2], uv[3]);
                mx8_values(uw[j][i + 1], us[j], uv[4], uv[5], uv[6], uv[7]);
                const int left = p.f - c - 4 * i;
                if (left <= 0) return;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    swiglu_grad(gv[e], uv[e], acc[i + (e >> 2)][j0 + j][e & 3], dg[e], du[e], h[e]);
                    if (4 * i + e >= live) dg[e] = du[e] = h[e] = 0.f;
                }
                store_cols<DT>(p.out, row * 2 * p.f + c + 4 * i, dg, left);
                store_cols<DT>(p.out, row * 2 * p.f + p.f + c + 4 * i, du, left);
                if (g.h) store_cols<DT>(g.h, row * p.f + c + 4 * i, h, left);
            });
        });
    });
}

// ---- adapters beside the product (adapters.h, Adapted) ------------------------
// Adds U's rows through their adapters' matrices to the sums: after the inputs' steps,
// one more for every sixteen ranks of every adapter that has rows here, which keeps the
// sums of its own rows.  Rows are grouped by adapter, so a tile of many
// rows has few of them; of few rows, the matrices of several are loaded at once.
// fp16: a row's operand is scaled by a power of two, and so are its sums here.
// Adapted calls, with the plain product's time and, in it, what x A^T and its operands take
// by the trace: 4096 tokens of 4096 inputs, 12288 outputs, 8 adapters of rank 32: 364 us,
// 323 and 28; sixteen tokens of 4096, 28672, SwiGLU, 32 adapters: 48 us, 34 and 9.
template <bool F16, bool SWIGLU, bool TRANS, int N, int NBM, typename Acc>
__device__ __forceinline__ void adapt_blocks(const Grouped& p, const Adapted& d, int ob0, int row0, int nrows, Acc& acc,
                                             uint8_t* lds) {
    constexpr int BA = N == 4 ? 1 : TRANS ? 2 : 4;  // adapters whose matrices are out at once
    constexpr int JB = NBM < 4 ? NBM : 4;           // row blocks at a time (a lane a row)
    [[maybe_unused]] uint8_t* mine_lds = lds + (threadIdx.x >> 6) * (BA * N * 512);
    const int lane = threadIdx.x & 63, r16 = lane & 15, c16 = lane >> 4;
    const uint16_t* M = (const uint16_t*)d.M;
    const int chunks = (d.rank + 15) / 16;
    // TRANS: the first of this lane's eight unsharded columns of block 2 i + lane / 32, -1
    // where there is none
    [[maybe_unused]] int col8[N / 2], base8[N / 2];  // (base8: the part's first)
    [[maybe_unused]] const bool whole = (uintptr_t)M % 16 == 0 && (TRANS ? d.width % 8 == 0 && p.f % 8 == 0 : d.rank % 8 == 0);
    if constexpr (TRANS)
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const int ob = ob0 + 2 * i + (lane >> 5), piece = ob / p.bps, c = 16 * (ob - piece * p.bps) + 8 * (lane & 1);
            const int r = piece / p.S, s = piece - r * p.S;
            base8[i] = (s * d.P + r) * p.f;
            col8[i] = ob < p.nout && c < p.f ? base8[i] + c : -1;
        }
    static_for<0, NBM / JB>([&](auto bc) ALWAYS_INLINE {
        constexpr int j0 = decltype(bc)::value * JB;
        const int first = row0 + 16 * j0, rows = min(nrows - 16 * j0, 16 * JB);
        // the rows' adapters: of row `lane`, and of this lane's of each block
        const int id = lane < rows ? d.plan.ids[first + lane] : -1;
        const uint64_t all = __ballot(id >= 0 && id < d.plan.n);
        if (!all) return;
        int mine[JB];
#pragma unroll
        for (int j = 0; j < JB; ++j) mine[j] = __shfl(id, 16 * j + r16);
        // (the operands of 16 rows and 16 ranks are 1 KB, a lane's 16 bytes)
        auto load_u = [&](int j, int ch) ALWAYS_INLINE {
            const bool in = mine[j] >= 0 && mine[j] < d.plan.n;
            const u32x4 v = d.operands[in ? ((int64_t)(first / 16 + j) * chunks + ch) * 64 + lane : 0];
            return in ? v : u32x4{0, 0, 0, 0};
        };
        [[maybe_unused]] int ex[JB];
        if constexpr (F16) {
#pragma unroll
            for (int j = 0; j < JB; ++j)
                ex[j] = mine[j] >= 0 && mine[j] < d.plan.n ? d.exponents[first + 16 * j + r16] : 0;
            static_for<0, JB>([&](auto jc) ALWAYS_INLINE {
                constexpr int j = decltype(jc)::value;
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j0 + j][e] = ldexpf(acc[i][j0 + j][e], -ex[j]);
            });
        }
        for (int ch = 0; ch < chunks; ++ch) {
            uint64_t rem = all;
            int a[BA];
            u32x4 mf[BA][N];
            auto load_matrices = [&]() ALWAYS_INLINE {
                static_for<0, BA>([&](auto bc) ALWAYS_INLINE {
                    constexpr int b = decltype(bc)::value;
                    a[b] = -1;
                    if (!rem) return;
                    a[b] = __builtin_amdgcn_readlane(id, __builtin_ctzll(rem));
                    rem &= ~__ballot(id == a[b]);
                    const uint16_t* Ma = M + (int64_t)a[b] * d.rank * d.width;
                    [[maybe_unused]] const int k = ch * 16 + 8 * (c16 & 1);
                    if constexpr (TRANS) {  // sixteen ranks of 16 columns, 32 bytes each, through LDS
                        static_for<0, N / 2>([&](auto ic) ALWAYS_INLINE {
                            constexpr int i = decltype(ic)::value;
                            const int j = ch * 16 + (lane >> 1 & 15);
                            const bool in = col8[i] >= 0 && j < d.rank;
                            if (whole) {
                                const u32x4 v = *(const u32x4*)(in ? Ma + (int64_t)j * d.width + col8[i] : M);
                                mf[b][i] = in ? v : u32x4{0, 0, 0, 0};
                            } else {
                                mf[b][i] = row8<false>(Ma + (in ? (int64_t)j * d.width + base8[i] : 0), M, in, col8[i] - base8[i], p.f);
                            }
                        });
                    } else {
                        static_for<0, N>([&](auto ic) ALWAYS_INLINE {
                            constexpr int i = decltype(ic)::value;
                            const int ob = ob0 + (SWIGLU ? i / 2 : i), piece = ob / p.bps, blk = ob - piece * p.bps;
                            const int r = SWIGLU ? piece : piece / p.S, s = SWIGLU ? i & 1 : piece - r * p.S;
                            const bool in = ob < p.nout && 16 * blk + r16 < p.f;
                            const int64_t col = in ? (int64_t)(s * d.P + r) * p.f + 16 * blk + r16 : 0;  // unsharded
                            if (whole) {
                                const u32x4 v = *(const u32x4*)(in && k < d.rank ? Ma + col * d.rank + k : M);
                                mf[b][i] = in && k < d.rank ? v : u32x4{0, 0, 0, 0};
                            } else {
                                mf[b][i] = row8<false>(Ma + col * d.rank, M, in && k < d.rank, k, d.rank);
                            }
                        });
                    }
                });
                if constexpr (TRANS) {
                    lds_order();
#pragma unroll
                    for (int b = 0; b < BA; ++b)
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) *(u32x4*)(mine_lds + (b * N / 2 + i) * 1024 + lane * 16) = mf[b][i];
                    lds_order();
#pragma unroll
                    for (int b = 0; b < BA; ++b)
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            mf[b][i] = read_columns(mine_lds + (b * N + i) * 512, 8 * (c16 & 1) + (r16 >> 2), 32, 8 * (r16 & 3));
                }
            };
            load_matrices();
            u32x4 uf[JB];
#pragma unroll
            for (int j = 0; j < JB; ++j) uf[j] = load_u(j, ch);
            while (true) {
                static_for<0, BA>([&](auto bc) ALWAYS_INLINE {
                    constexpr int b = decltype(bc)::value;
                    if (a[b] < 0) return;
                    static_for<0, JB>([&](auto jc) ALWAYS_INLINE {
                        constexpr int j = decltype(jc)::value;
                        const bool own = mine[j] == a[b];
                        const uint64_t owners = __ballot(own);
                        if (!owners) return;
                        const u32x4 u = own ? uf[j] : u32x4{0, 0, 0, 0};
                        if (owners == ~0ull) {
#pragma unroll
                            for (int i = 0; i < N; ++i) acc[i][j0 + j] = mfma16<F16>(mf[b][i], u, acc[i][j0 + j]);
                        } else {  // (an infinite matrix times the other rows' zeros is NaN)
#pragma unroll
                            for (int i = 0; i < N; ++i) {
                                const f32x4 v = mfma16<F16>(mf[b][i], u, acc[i][j0 + j]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[i][j0 + j][e] = own ? v[e] : acc[i][j0 + j][e];
                            }
                        }
                    });
                });
                if (!rem) break;
                load_matrices();
            }
        }
        if constexpr (F16)
            static_for<0, JB>([&](auto jc) ALWAYS_INLINE {
                constexpr int j = decltype(jc)::value;
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j0 + j][e] = ldexpf(acc[i][j0 + j][e], ex[j]);
            });
        asm volatile("" ::: "memory");  // (no load of the next row blocks' before)
    });
}

// What becomes of a tile's sums (E_KEEP and E_GRAD: the gated block, gated.h; E_ADAPT:
// adapters.h)
enum Epilogue { E_STORE = 0, E_KEEP = 1, E_GRAD = 2, E_SPLIT = 3, E_ADAPT = 4 };
template <int EPI>
using Extra = std::conditional_t<EPI == E_ADAPT, Adapted, Gated>;

// n tile nt of the rows of one slot; the stages may be larger than needed.  E_SPLIT:
// part blockIdx.y of gridDim.y of the k tiles, stored in a slab of its own.
template <int MODE, bool SWIGLU, bool TRANS, int TM, int BN, int NS, bool AL, int EPI>
__device__ __forceinline__ void grouped_tile(const Grouped& p, const Slot s, const int nt, const Stages<NS>& stage,
                                             const Extra<EPI>& extra) {
    using Shape = TileShape<MODE, TM, BN>;
    constexpr int WM = 2, WN = 4, NWV = WM * WN;
    constexpr int NBM = TM / WM / 16, NBN = BN / WN / 16;
    constexpr bool MX = MODE >= G_MX4, A4 = MODE == G_MX4A4;
    constexpr int KT = A4 ? 256 : MX ? 128 : 64;
    constexpr int KST = MX ? 128 : 32;  // inputs of a stored weight step
    constexpr int ROWB = Shape::ROWB, FPB = Shape::FPB;
    constexpr int CPR = ROWB / 16;                // chunks of a row
    constexpr int RPI = 64 / CPR;                 // rows of a 1 KB load
    constexpr int LA = TM * ROWB / 1024 / NWV;    // loads of a wave
    constexpr int LW = BN / 16 * FPB / NWV;
    constexpr int KK = MODE == G_MX4 ? 4 : 2;     // MFMA steps of a k tile
    static_assert(LA * NWV * 1024 == TM * ROWB && LW * NWV * 16 == BN * FPB, "loads divide over the waves");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // (the WM waves of one column stand on one SIMD: where the tile has rows for
    // one of them only, it has the SIMD for itself)
    const int wave_m = wave / WN, wave_n = wave % WN;

    // load i of a wave: rows (i NWV + wave) RPI .. of A, chunk lane % CPR of them
    uint32_t aoff[LA];
    [[maybe_unused]] int arow[LA];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int m = (i * NWV + wave) * RPI + lane / CPR;
        const int row = m < s.nrows ? grouped_row(p.rows, p.kdiv, p.T, s.row0 + m) : -1;
        const int sw = ROWB == 128 ? (m >> 1) & 7 : m & 15;
        const int ch = (lane % CPR) ^ sw;
        arow[i] = row;
        aoff[i] = row < 0 ? kOutside : (uint32_t)((A4 ? row * (p.lda / 2) : row * p.lda * 2) + ch * 16);
    }
    auto chunk_of = [&](int i) {
        const int m = (i * NWV + wave) * RPI + lane / CPR;
        return (lane % CPR) ^ (ROWB == 128 ? (m >> 1) & 7 : m & 15);
    };
    constexpr int KPC = A4 ? 32 : 8;  // inputs of a chunk
    const uint8_t* W = p.W + (int64_t)s.e * p.w_expert;
    // PERM: columns (weight rows) are dealt to the MFMAs so that a lane ends up with 4
    // NBN (8) adjacent ones, for the epilogue's wide accesses; the fragments' rows are
    // then stored apart so that the four pieces of a read lie in different banks
    constexpr bool PERM = EPI == E_GRAD || (EPI == E_KEEP && NBN == 4);
    const uint32_t wlane = (uint32_t)(TRANS ? lane ^ (((lane >> 4) & 1) << 2) : lane) * 16;
    uint32_t wbase[LW];  // fragment's byte offset at k tile 0 (wave-uniform)
#pragma unroll
    for (int i = 0; i < LW; ++i) {
        const int f = i * NWV + wave;
        if constexpr (TRANS) {
            wbase[i] = 0;
        } else {
            const int b = f / FPB;
            const int ob = SWIGLU ? nt * (BN / 32) + b / 2 : nt * (BN / 16) + b;
            wbase[i] = ((uint32_t)weight_block(p, min(ob, p.nout - 1), SWIGLU ? b & 1 : 0) * p.wsteps + f % FPB) * 1024u;
        }
    }
    const int kts = (p.kpad + KT - 1) / KT;
    int nkt = p.nseg * kts, first = 0;
    if constexpr (EPI == E_SPLIT) {
        first = (int)((int64_t)nkt * blockIdx.y / gridDim.y);
        nkt = (int)((int64_t)nkt * (blockIdx.y + 1) / gridDim.y) - first;
    }
    const int64_t a_bytes = A4 ? (int64_t)p.T * (p.lda / 2) : ((int64_t)(p.T - 1) * p.lda + p.kl) * 2;

    // the k tile that is loaded next: its segment, first input, and the
    // segment's first element of A
    int iseg = 0, ik = 0, ipiece = 0;
    int64_t irank = 0, ia = 0;
    if constexpr (EPI == E_SPLIT) {
        iseg = first / kts;
        ik = (first - iseg * kts) * KT;
        ipiece = iseg % p.a_pieces;
        irank = (int64_t)(iseg / p.a_pieces) * p.a_rank;
        ia = seg_offset(p, iseg);
    }
    // (past the last k tile every load reads zeros, into a stage never read)
    auto bytes = [&](int64_t n) ALWAYS_INLINE { return iseg < p.nseg ? n : 0; };
    auto load_a = [&](uint8_t* sA, int i) ALWAYS_INLINE {
        const int k = ik + chunk_of(i) * KPC;
        uint8_t* to = sA + (i * NWV + wave) * 1024;
        const uint8_t* base = (const uint8_t*)p.A + (A4 ? ia / 2 : ia * 2);
        uint32_t off = aoff[i];
        if (ik + KT > p.kl && k >= p.kl) off = kOutside;
        dma16(buffer(base, bytes(a_bytes)), off, (uint32_t)(A4 ? ik / 2 : ik * 2), to);
    };
    // rows of any alignment: through registers, into LDS a k tile later (of two
    // stages: when the k tile at hand is done)
    constexpr bool LATE = !AL && NS > 2;
    [[maybe_unused]] u32x4 av[LA];
    auto fetch_a = [&]() ALWAYS_INLINE {
#pragma unroll
        for (int i = 0; i < LA; ++i)
            av[i] = load8_any((const uint16_t*)p.A + (iseg < p.nseg ? ia : 0), iseg < p.nseg ? arow[i] : -1, p.lda,
                              ik + chunk_of(i) * KPC, p.kl);
    };
    auto put_a = [&](uint8_t* sA) ALWAYS_INLINE {
#pragma unroll
        for (int i = 0; i < LA; ++i) *(u32x4*)(sA + (i * NWV + wave) * 1024 + lane * 16) = av[i];
    };
    auto load_w = [&](uint8_t* sW, int i) ALWAYS_INLINE {
        const int f = i * NWV + wave;
        uint32_t off = wlane, at;
        if constexpr (TRANS) {
            const int kb = ik / 16 + f / (BN / 32), st = nt * (BN / 32) + f % (BN / 32);
            at = ((uint32_t)(iseg * (p.kpad / 16) + kb) * p.wsteps + st) * 1024u;
            if constexpr (EPI == E_ADAPT) {  // (ranks' columns may be matrices of their own)
                const int q = st / p.wsteps;
                at = (uint32_t)q * extra.wrank + ((uint32_t)(iseg * (p.kpad / 16) + kb) * p.wsteps + st - q * p.wsteps) * 1024u;
            }
            if constexpr (PERM) off = (uint32_t)(lane ^ (NBN == 4 ? (((f & 1) << 1) | (lane >> 5)) << 2 : (lane >> 4) << 2)) * 16;
            if (kb >= p.kpad / 16 || (EPI == E_ADAPT ? 2 * st >= p.nout : st >= p.wsteps)) off = kOutside, at = 0;
        } else {
            if constexpr (PERM) off = (uint32_t)(lane ^ ((f / FPB & 2) << 1)) * 16;
            at = wbase[i] + (uint32_t)(iseg * p.kpad + ik) / KST * 1024u;
            if constexpr (EPI == E_ADAPT) at = wbase[i] + (uint32_t)iseg * extra.wseg + (uint32_t)ik / KST * 1024u;
            if (FPB * KST > KST && MX && ik + (f % FPB) * KST >= p.kpad) off = kOutside, at = 0;
        }
        dma16(buffer(W, bytes(p.w_expert)), off, at, sW + f * 1024);
    };
    // MXFP4: this lane's scales of a k tile, one load each: weight row lane & 15
    // of (block, step) number wave * 4 + lane / 16, and row wave * 32 + lane / 2
    // of A, step lane & 1
    constexpr int SW = BN * FPB / 64;  // loads of a k tile's weight scales
    static_assert(!MX || SW <= NWV, "one load a wave");
    constexpr int SA = TM * 2 / 64;    // and of the rows' scales
    static_assert(!A4 || SA <= NWV, "one load a wave");
    [[maybe_unused]] uint32_t swoff = 0, saoff = kOutside;
    [[maybe_unused]] const int ssub = (wave * 4 + (lane >> 4)) % FPB;
    if constexpr (MX) {
        const int b = (wave * 4 + (lane >> 4)) / FPB;
        const int ob = SWIGLU ? nt * (BN / 32) + b / 2 : nt * (BN / 16) + b;
        const int wb = weight_block(p, min(ob, p.nout - 1), SWIGLU ? b & 1 : 0);
        swoff = (uint32_t)mx4_scale_offset(wb, 0, lane & 15, p.wsteps);
    }
    if constexpr (A4) {
        const int m = wave * 32 + (lane >> 1);
        const int row = m < s.nrows ? grouped_row(p.rows, p.kdiv, p.T, s.row0 + m) : -1;
        if (row >= 0) saoff = (uint32_t)(row * (p.kl / 32)) + (lane & 1) * 4;
    }
    auto load_scales = [&](uint32_t* sSW, uint32_t* sSA) ALWAYS_INLINE {
        if constexpr (MX) {
            if (wave < SW) {
                const int st = (iseg * p.kpad + ik) / 128 + ssub;
                const uint32_t off = swoff + (st >> 2) * 256 + (st & 3) * 4;
                dma4(buffer(p.wsc + (int64_t)s.e * p.wsc_expert, bytes(p.wsc_expert)),
                     ik + ssub * 128 < p.kpad ? off : kOutside, 0, (uint8_t*)(sSW + wave * 64));
            }
        }
        if constexpr (A4) {
            if (wave < SA)
                dma4(buffer(p.a_scales + (int64_t)iseg * p.T * (p.kl / 32), bytes((int64_t)p.T * (p.kl / 32))),
                     saoff != kOutside && ik + (lane & 1) * 128 < p.kl ? saoff + ik / 32 : kOutside, 0,
                     (uint8_t*)(sSA + wave * 64));
        }
    };
    auto advance = [&]() ALWAYS_INLINE {
        ik += KT;
        if (ik < p.kpad) return;
        ik = 0;
        ++iseg;
        ia += p.kl;
        if (++ipiece == p.a_pieces) ipiece = 0, irank += p.a_rank, ia = irank;
        if constexpr (EPI == E_ADAPT)
            if (iseg == extra.again) ia = irank = 0;
    };

    f32x4 acc[NBN][NBM];
#pragma unroll
    for (int i = 0; i < NBN; ++i)
#pragma unroll
        for (int j = 0; j < NBM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int c16 = lane >> 4, r16 = lane & 15;
    const int amine = (wave_m * NBM * 16 + r16) * ROWB, asw = ROWB == 128 ? (r16 >> 1) & 7 : r16;
    auto read = [&](const uint8_t* sA, const uint8_t* sW, const u32x4(&codes)[NBN], const float(&scale)[NBN], int kk,
                    u32x4(&wf)[NBN], u32x4(&af)[NBM]) ALWAYS_INLINE {
#pragma unroll
        for (int i = 0; i < NBN; ++i) {
            const int nb = wave_n * NBN + i;
            if constexpr (PERM && TRANS) {
                // D row 4 c + e of block i: column 4 NBN c + 4 i + e of the wave's
                const int c = r16 & 3, col = 4 * NBN * c + 4 * i;
                const uint8_t* fr = sW + ((2 * kk + (c16 >> 1)) * (BN / 32) + wave_n * (NBN / 2) + (col >> 5)) * 1024;
                const int rr = (8 * (c16 & 1) + (r16 >> 2)) ^ (c << 2);
                const uint8_t* a0 = fr + (rr + 16 * ((col >> 3) & 3)) * 16 + 8 * (i & 1);
                const uint8_t* a1 = fr + ((rr ^ 4) + 16 * ((col >> 3) & 3)) * 16 + 8 * (i & 1);
                const u32x2 lo = read_tr(a0), hi = read_tr(a1);
                wf[i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            } else if constexpr (PERM) {
                // D row 4 c + e of the wave's output block k = i / 2: its column 8 c + 4 k + e
                const int k = i >> 1, b = wave_n * NBN + 2 * (r16 >> 3) + (i & 1);
                const int row = ((8 * (r16 >> 2) + 4 * k + (r16 & 3)) & 15) ^ ((r16 >> 3) << 2);
                wf[i] = *(const u32x4*)(sW + (b * FPB + kk) * 1024 + (row + 16 * c16) * 16);
            } else if constexpr (TRANS) {
                // columns 16 nb .. of the tile, contracted rows 32 kk + 8 c16 ..
                const uint8_t* fr = sW + ((2 * kk + (c16 >> 1)) * (BN / 32) + (nb >> 1)) * 1024;
                const int ch = 2 * (nb & 1) + ((r16 & 3) >> 1);
                const int rr = (8 * (c16 & 1) + (r16 >> 2)) ^ ((ch & 1) << 2);
                const uint8_t* a0 = fr + (rr + 16 * ch) * 16 + 8 * (r16 & 1);
                const uint8_t* a1 = fr + ((rr ^ 4) + 16 * ch) * 16 + 8 * (r16 & 1);
                const u32x2 lo = read_tr(a0), hi = read_tr(a1);
                wf[i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            } else if constexpr (MODE == G_MX4) {
                wf[i] = mx4_to_bf16(codes[i][kk], scale[i]);
            } else {
                wf[i] = *(const u32x4*)(sW + (nb * FPB + kk) * 1024 + lane * 16);
            }
        }
#pragma unroll
        for (int j = 0; j < NBM; ++j) {
            const int ch = MODE == G_MX4 ? 4 * c16 + kk : 4 * kk + c16;
            af[j] = *(const u32x4*)(sA + amine + j * 16 * ROWB + ((ch ^ asw) << 4));
        }
    };
    auto multiply = [&](const uint32_t* sSW, const uint32_t* sSA, int kk, u32x4(&wf)[NBN], u32x4(&af)[NBM]) ALWAYS_INLINE {
        uint32_t ws[NBN], as[NBM];
        if constexpr (A4) {
#pragma unroll
            for (int i = 0; i < NBN; ++i) ws[i] = sSW[((wave_n * NBN + i) * 2 + kk) * 16 + r16] >> (8 * c16);
#pragma unroll
            for (int j = 0; j < NBM; ++j) as[j] = sSA[(wave_m * NBM * 16 + j * 16 + r16) * 2 + kk] >> (8 * c16);
        }
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int j = 0; j < NBM; ++j)
#pragma unroll
            for (int i = 0; i < NBN; ++i) {
                if constexpr (A4) acc[i][j] = mfma_mx4(wf[i], ws[i], af[j], as[j], acc[i][j]);
                else acc[i][j] = mfma16<MODE == G_F16>(wf[i], af[j], acc[i][j]);
            }
        __builtin_amdgcn_s_setprio(0);
    };
    auto issue = [&](uint8_t* nA, uint8_t* nW, uint32_t* nSW, uint32_t* nSA) ALWAYS_INLINE {
        load_scales(nSW, nSA);
        if constexpr (AL) {
#pragma unroll
            for (int i = 0; i < LA; ++i) load_a(nA, i);
        } else {
            fetch_a();
            if constexpr (!LATE) put_a(nA);
        }
#pragma unroll
        for (int i = 0; i < LW; ++i) load_w(nW, i);
        advance();
    };
    // (of the loads that may stay in flight, a wave's scales are not counted, nor
    // rows that go into LDS behind the barrier)
    constexpr int LATER = (NS - 2) * (LATE ? LW : LA + LW);
    auto arrived = [&](auto uc) ALWAYS_INLINE {
        stage_barrier<LATER>();
        if constexpr (LATE) put_a(stage.A[(decltype(uc)::value + NS - 2) % NS]);
    };
    auto step = [&](auto uc) ALWAYS_INLINE {
        constexpr int u = decltype(uc)::value, next = (u + NS - 1) % NS;
        const uint8_t *sA = stage.A[u], *sW = stage.W[u];
        const uint32_t *sSW = stage.SW[u], *sSA = stage.SA[u];
        uint8_t *nA = stage.A[next], *nW = stage.W[next];
        uint32_t *nSW = stage.SW[next], *nSA = stage.SA[next];
        // this wave's loads of the k tile have landed; behind the barrier every
        // wave's have, and every wave has read the k tile before
        arrived(uc);
        u32x4 wf[NBN], af[NBM];
        // MXFP4 weights: a lane's 32 codes and their scale serve the k tile's four steps
        [[maybe_unused]] u32x4 codes[NBN];
        [[maybe_unused]] float scale[NBN];
        if constexpr (MODE == G_MX4) {
#pragma unroll
            for (int i = 0; i < NBN; ++i) {
                codes[i] = *(const u32x4*)(sW + (wave_n * NBN + i) * 1024 + lane * 16);
                scale[i] = e8m0_to_f32((sSW[(wave_n * NBN + i) * 16 + r16] >> (8 * c16)) & 255u);
            }
        }
        if constexpr (A4) issue(nA, nW, nSW, nSA);
        static_for<0, KK>([&](auto kc) ALWAYS_INLINE {
            constexpr int kk = decltype(kc)::value;
            read(sA, sW, codes, scale, kk, wf, af);
            if constexpr (!A4 && kk == 0) {
                load_scales(nSW, nSA);
                if constexpr (AL) {
#pragma unroll
                    for (int i = 0; i < LA; ++i) load_a(nA, i);
                } else {
                    fetch_a();
                }
            } else if constexpr (!A4 && kk == 1) {
#pragma unroll
                for (int i = 0; i < LW; ++i) load_w(nW, i);
                advance();
            }
            multiply(sSW, sSA, kk, wf, af);
        });
        if constexpr (!AL && !LATE) put_a(nA);
    };
    static_for<0, NS - 1>([&](auto uc) ALWAYS_INLINE {
        constexpr int u = decltype(uc)::value;
        issue(stage.A[u], stage.W[u], stage.SW[u], stage.SA[u]);
        if constexpr (LATE && u < NS - 2) put_a(stage.A[u]);
    });
    if (wave_m * NBM * 16 < s.nrows) {
        for (int t = 0; t < nkt; t += NS)
            static_for<0, NS>([&](auto uc) ALWAYS_INLINE {
                if (decltype(uc)::value == 0 || t + decltype(uc)::value < nkt) step(uc);
            });
    } else {  // none of the wave's rows is there: its share of the loads is all
        for (int t = 0; t < nkt; t += NS)
            static_for<0, NS>([&](auto uc) ALWAYS_INLINE {
                constexpr int u = decltype(uc)::value, next = (u + NS - 1) % NS;
                if (u > 0 && t + u >= nkt) return;
                arrived(uc);
                issue(stage.A[next], stage.W[next], stage.SW[next], stage.SA[next]);
            });
    }
    wait_loads();  // none may still be writing this workgroup's LDS when it ends

    constexpr int NO = SWIGLU ? NBN / 2 : NBN;  // output blocks of a wave
    const int m0 = wave_m * NBM * 16;
    [[maybe_unused]] int rows_to[NBM];
    if constexpr (EPI == E_KEEP) {
        keep_blocks<MODE == G_F16, NO, NBM, WN>(p, extra, nt * NO * WN + wave_n * NO, s.row0 + m0, s.nrows - m0, acc,
                                                (uint32_t*)stage.A[0]);
        if constexpr (NO == 2) return;
    } else if constexpr (EPI == E_GRAD) {
        grad_blocks<MODE == G_F16, NO, NBM>(p, extra, nt * NO * WN + wave_n * NO, s.row0 + m0, s.nrows - m0, acc);
        return;
    } else if constexpr (EPI == E_ADAPT) {
#pragma unroll
        for (int j = 0; j < NBM; ++j)  // (all at once, before the stores)
            rows_to[j] = m0 + 16 * j + r16 < s.nrows ? token(extra.plan, s.row0 + m0 + 16 * j + r16) : 0;
        adapt_blocks<MODE == G_F16, SWIGLU, TRANS, NBN, NBM>(p, extra, nt * NO * WN + wave_n * NO, s.row0 + m0, s.nrows - m0,
                                                             acc, stage.M);
    }
    const Grouped* to = &p;
    [[maybe_unused]] Grouped part;
    if constexpr (EPI == E_SPLIT) {
        part = p;
        part.out = (float*)p.out + blockIdx.y * extra.slab;
        to = &part;
    }
    auto value = [&](auto ic, auto jc, auto near) {
        constexpr int i = decltype(ic)::value, j = decltype(jc)::value;
        if constexpr (!SWIGLU) return acc[i][j];
        else return swiglu4<decltype(near)::value>(acc[2 * i][j], acc[2 * i + 1][j]);
    };
    const int ob0 = nt * NO * WN + wave_n * NO;
    if constexpr (EPI == E_ADAPT)
        store_blocks<SWIGLU, NO, NBM>(*to, ob0, s.row0 + m0, s.nrows - m0, value,
                                      [&](auto jc) { return rows_to[decltype(jc)::value]; });
    else
        store_blocks<SWIGLU, NO, NBM>(*to, ob0, s.row0 + m0, s.nrows - m0, value);
}

template <int MODE, bool SWIGLU, bool TRANS, int TM, int BN, int NS, bool AL, int EPI>
__global__ __launch_bounds__(512) void grouped_tile_kernel(Grouped p, int slots, int tiles_n, int cus, Extra<EPI> extra) {
    using Shape = TileShape<MODE, TM, BN>;
    constexpr bool R = NS >= 3, Q = NS == 4;  // (a ring of two, three or four)
    static_assert(NS >= 2 && NS <= 4, "stages");
    __shared__ __attribute__((aligned(1024))) uint8_t sA0[Shape::A], sA1[Shape::A], sW0[Shape::W], sW1[Shape::W],
        sA2[R ? Shape::A : 4], sA3[Q ? Shape::A : 4], sW2[R ? Shape::W : 4], sW3[Q ? Shape::W : 4];
    __shared__ uint32_t sSW0[Shape::SW], sSW1[Shape::SW], sSA0[Shape::SA], sSA1[Shape::SA], sSW2[R ? Shape::SW : 1],
        sSW3[Q ? Shape::SW : 1], sSA2[R ? Shape::SA : 1], sSA3[Q ? Shape::SA : 1];
    // (an array of its own, too: as part of a stage, it made the stages' reads wait for each
    // other's loads)
    __shared__ __attribute__((aligned(16))) uint8_t sM[EPI == E_ADAPT && TRANS ? 16384 : 4];
    Stages<NS> stage;
    stage.M = sM;
    stage.A[0] = sA0, stage.W[0] = sW0, stage.SW[0] = sSW0, stage.SA[0] = sSA0;
    stage.A[1] = sA1, stage.W[1] = sW1, stage.SW[1] = sSW1, stage.SA[1] = sSA1;
    if constexpr (R) {
        stage.A[2] = sA2, stage.W[2] = sW2, stage.SW[2] = sSW2, stage.SA[2] = sSA2;
    }
    if constexpr (Q) {
        stage.A[3] = sA3, stage.W[3] = sW3, stage.SW[3] = sSW3, stage.SA[3] = sSA3;
    }
    // The launch has room for every way the rows may fall on the experts; the
    // tiles that there are, not that room, are dealt out to the XCDs.  (Falling
    // offsets could count more: those are left out.)
    SlotMap map(p.offsets, p.E, p.R, TM);
    slots = min(slots, map.count());
    int tiles = slots * tiles_n, rest = 0;
    // 256 x 256 tiles take a compute unit each.  Where the last time round the
    // chip would leave half of it idle or more, its tiles are cut into quarters
    // (down projection of 4096 tokens, 2.25 times round: 1168 -> 1024 us).
    if constexpr (TM == 256) {
        rest = tiles % cus;
        if (rest * 2 > cus) rest = 0;
        tiles -= rest;
    }
    auto slot_of = [&](int tile, int& nt) {
        constexpr int GM = 4;
        const int g = tile / (GM * tiles_n), first = g * GM, gsz = min(GM, slots - first);
        const int tin = tile - g * GM * tiles_n;
        nt = tin / gsz;
        return map.find(first + tin % gsz);
    };
    int nt;
    if ((int)blockIdx.x < tiles) {
        const Slot s = slot_of(xcd_remap(blockIdx.x, tiles), nt);
        if (s.e < 0) return;
        grouped_tile<MODE, SWIGLU, TRANS, TM, BN, NS, AL, EPI>(p, s, nt, stage, extra);
    } else if constexpr (TM == 256) {
        if ((int)blockIdx.x >= tiles + 4 * rest) return;
        const int q = xcd_remap(blockIdx.x - tiles, 4 * rest);
        Slot s = slot_of(tiles + q / 4, nt);
        s.row0 += (q & 1) * 128;
        s.nrows = min(s.nrows - (q & 1) * 128, 128);
        if (s.e < 0 || s.nrows <= 0) return;
        grouped_tile<MODE, SWIGLU, TRANS, 128, BN / 2, NS, AL, EPI>(p, s, 2 * nt + ((q >> 1) & 1), stage, extra);
    }
}

template <int MODE, bool SWIGLU, bool TRANS, int TM, int BN, int NS, bool AL, int EPI = E_STORE>
hipError_t tile_launch(const Grouped& p, hipStream_t s, const Extra<EPI>& extra = Extra<EPI>{}) {
    constexpr int NB = SWIGLU ? BN / 32 : BN / 16;
    const int64_t slots = p.R / TM + (p.R < p.E ? p.R : p.E);
    const int64_t tiles_n = (p.nout + NB - 1) / NB;
    const int cus = device_cus();
    const int64_t blocks = slots * tiles_n + (TM == 256 ? 3 * (cus / 2) : 0);
    if (blocks >= kMaxBlocks / 2) return hipErrorInvalidConfiguration;
    int parts = 1;
    if constexpr (EPI == E_SPLIT) parts = extra.splits;
    launch(grouped_tile_kernel<MODE, SWIGLU, TRANS, TM, BN, NS, AL, EPI>, dim3((unsigned)blocks, parts), dim3(512), 0, s, p,
           (int)slots, (int)tiles_n, cus, extra);
    return hipGetLastError();
}

// Tiles of TM rows and 128 weight rows; a quarter more rows than the average
// expert's are reckoned with.
template <bool SWIGLU, int TM>
int64_t tiles_of(const Grouped& p) {
    const int64_t experts = p.R < p.E ? p.R : p.E;
    const int64_t slots = experts * ((p.R * (int64_t)5 / (4 * experts) + TM - 1) / TM);
    return slots * ((p.nout + (SWIGLU ? 3 : 7)) / (SWIGLU ? 4 : 8));
}

// Whether these hardly fill the chip once: they then take four stages, which
// leave a compute unit room for one workgroup instead of two or three.  us with
// two / four stages, 8 x (4096 x 14336), 256 tiles: m = 32: 200 / 156, 96: 238 /
// 180; MXFP4 m = 32: 113 / 87; 8 x (28672 x 4096, SwiGLU), 1792 tiles: m = 32: 332
// / 324, 128: 471 / 503; 32 x (2048 x 2048, SwiGLU), 512 tiles: m = 64: 58 / 69.
template <bool SWIGLU, int TM>
bool few_tiles(const Grouped& p) {
    return tiles_of<SWIGLU, TM>(p) * 5 <= (int64_t)device_cus() * 6;
}

// Tile by the rows of an expert, m = R / E on average, and by whether the tiles
// fill the chip (experts differ: half a tile more for each is reckoned with where
// wide tiles are asked about, a quarter more rows in tiles_of).  Times
// in us on bf16 experts, 64 x 128 / 128 x 128 / 256 x 256 tiles:
//   8 x (28672 x 4096, SwiGLU)  m = 32: 339 335 407   96: 440 378 434  128: 604 471 464   256: 1010 765 717
//   8 x (4096 x 14336)          m = 32: 200 204 318   96: 229 237 323  192: 434 271 360   256: 476 498 385
//   32 x (2048 x 2048, SwiGLU)  m = 32:  55  55  62   48:  66  57  64  128:  88  84  72   256: 146 118 125
template <int MODE, bool SWIGLU, bool TRANS, bool AL, int EPI = E_STORE>
hipError_t tile_mode(const Grouped& p, hipStream_t s, const Extra<EPI>& extra = Extra<EPI>{}) {
    if constexpr (!AL && MODE == G_MX4) {
        return tile_launch<MODE, SWIGLU, TRANS, 128, 128, 2, false, EPI>(p, s, extra);
    } else if constexpr (!AL) {
        // Rows through registers: times round the chip, of two or three workgroups
        // a compute unit.  us, 128 x 128 / 64 x 128 / the latter in three stages:
        // 8 x (2046 x 4094) m = 125: 100 76 73   gate|up of 8 x (8188 x 2046): 131 115 123
        // 8 x (4094 x 4094) m = 500: 354 318 390   32 x (1022 x 2046) m = 188: 66 79 75
        const int64_t cus = device_cus();
        if (few_tiles<SWIGLU, 64>(p)) return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 3, false, EPI>(p, s, extra);
        const int64_t wide = (tiles_of<SWIGLU, 128>(p) + 2 * cus - 1) / (2 * cus);
        const int64_t narrow = (tiles_of<SWIGLU, 64>(p) + 3 * cus - 1) / (3 * cus);
        if (3 * narrow <= 4 * wide) return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 2, false, EPI>(p, s, extra);
        return tile_launch<MODE, SWIGLU, TRANS, 128, 128, 2, false, EPI>(p, s, extra);
    } else if constexpr (MODE == G_MX4) {
        // (turning codes into operands costs the narrow tile as much as its few
        // rows' products; gate|up, 64 x 128 / 128 x 256:  m = 64: 185 222  256: 552 531  1024: 1987 1742,
        // down  64: 126 174  256: 280 364  1024: 960 938)
        const int64_t tiles = (p.R / 128 + p.E / 2) * ((p.nout + 15) / 16) * (SWIGLU ? 2 : 1);
        if (p.R >= (int64_t)192 * p.E && tiles >= (int64_t)device_cus() * 6)
            return tile_launch<MODE, SWIGLU, TRANS, 128, 256, 2, true, EPI>(p, s, extra);
        if (few_tiles<SWIGLU, 64>(p)) return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 4, true, EPI>(p, s, extra);
        return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 2, true, EPI>(p, s, extra);
    } else {
        // (MXFP4 products are so short that a wave of tiles more costs them a
        // wider tile's gain: 512 rows of 8 experts, gate|up 461 429, down 221 256)
        const int64_t tiles = (p.R / 256 + p.E / 2) * ((p.nout + 15) / 16) * (SWIGLU ? 2 : 1);
        if (p.R >= (int64_t)128 * p.E && tiles * 10 >= (int64_t)device_cus() * (MODE == G_MX4A4 ? 40 : 7))
            return tile_launch<MODE, SWIGLU, TRANS, 256, 256, 2, true, EPI>(p, s, extra);
        // (few narrow tiles go before few wide ones: 256 rows of 4096 x 4096 27 32, 500 rows
        // of 2 x (2048 x 2048) 15 19)
        if (few_tiles<SWIGLU, 64>(p)) return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 4, true, EPI>(p, s, extra);
        if (p.R > (int64_t)40 * p.E) {
            if (few_tiles<SWIGLU, 128>(p)) return tile_launch<MODE, SWIGLU, TRANS, 128, 128, 4, true, EPI>(p, s, extra);
            return tile_launch<MODE, SWIGLU, TRANS, 128, 128, 2, true, EPI>(p, s, extra);
        }
        return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 2, true, EPI>(p, s, extra);
    }
}

}  // namespace

}  // namespace sg
