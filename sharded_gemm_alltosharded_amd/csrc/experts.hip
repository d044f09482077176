// Grouped products of a mixture of experts (experts.h, Grouped), and the
// layout of an expert layer's weights.
#include "experts.h"

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
template <int DT, bool PAD, int N, int M, typename F>
__device__ __forceinline__ void store_typed(const Grouped& p, int ob0, int row0, int nrows, F&& value) {
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
            store_cols<DT>(p.out, base + (int64_t)(row0 + m) * p.ldo, v, p.f - c);
        });
    });
}
template <bool PAD, int N, int M, typename F>
__device__ __forceinline__ void store_blocks(const Grouped& p, int ob0, int row0, int nrows, F&& value) {
    if (p.out_dtype == SG_BF16) store_typed<SG_BF16, PAD, N, M>(p, ob0, row0, nrows, value);
    else if (p.out_dtype == SG_F16) store_typed<SG_F16, PAD, N, M>(p, ob0, row0, nrows, value);
    else store_typed<SG_F32, PAD, N, M>(p, ob0, row0, nrows, value);
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
// other operand.  KS of the NWV waves split the inputs of one group of NB output
// blocks (their sums are added in wave order through LDS), NWV / KS groups stand
// side by side.  Steps come in runs of four, a run of loads ahead.
// ---------------------------------------------------------------------------
template <int MODE, bool SWIGLU, int MB, int NB, int KS, int NWV, bool AL>
__global__ __launch_bounds__(64 * NWV) void grouped_stream_kernel(Grouped p) {
    constexpr int NG = NWV / KS, NW = SWIGLU ? 2 * NB : NB;
    constexpr bool MX = MODE >= G_MX4;
    constexpr int KST = MX ? 128 : 32;               // inputs of a step
    constexpr int AF = MODE == G_MX4 ? 4 : 1;        // 16-byte operands of a step and 16 rows
    __shared__ f32x4 red[KS > 1 ? (KS - 1) * NG * NW * MB * 64 : 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kw = wave % KS, ng = wave / KS;
    const int groups = (p.nout + NG * NB - 1) / (NG * NB);
    const int si = blockIdx.x / groups;
    const Slot s = SlotMap(p.offsets, p.E, p.R, 16 * MB).find(si);
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
            ws[i] = p.wsc + (int64_t)s.e * p.wsc_expert + mx4_scale_offset(wb, 0, lane & 15, p.wsteps);
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
    uint32_t as[4][MB];
    u32x4 wsc[NW], wsn[NW];  // a run's scales of a weight row: a word a step, a byte a block
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
            for (int i = 0; i < NW; ++i) wsn[i] = *(const u32x4*)(ws[i] + (int64_t)c * 256);
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
                        const float sc = e8m0_to_f32((wsc[i][u] >> (8 * (lane >> 4))) & 255u);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const u32x4 wv = mx4_to_bf16(wf[u][i][j], sc);
#pragma unroll
                            for (int b = 0; b < MB; ++b) acc[i][b] = mfma16<false>(wv, af[u][b][j], acc[i][b]);
                        }
                    } else if constexpr (MODE == G_MX4A4) {
#pragma unroll
                        for (int b = 0; b < MB; ++b)
                            acc[i][b] = mfma_mx4(wf[u][i], wsc[i][u] >> (8 * (lane >> 4)), af[u][b][0], as[u][b], acc[i][b]);
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
    store_blocks<SWIGLU, NB, MB>(p, ob0, s.row0, s.nrows, [&](auto ic, auto jc, auto near) {
        constexpr int n = decltype(ic)::value, b = decltype(jc)::value;
        if constexpr (!SWIGLU) return acc[n][b];
        else return swiglu4<decltype(near)::value>(acc[2 * n][b], acc[2 * n + 1][b]);
    });
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
};

// n tile nt of the rows of one slot; the stages may be larger than needed
template <int MODE, bool SWIGLU, bool TRANS, int TM, int BN, int NS, bool AL>
__device__ __forceinline__ void grouped_tile(const Grouped& p, const Slot s, const int nt, const Stages<NS>& stage) {
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
    const int kts = (p.kpad + KT - 1) / KT, nkt = p.nseg * kts;
    const int64_t a_bytes = A4 ? (int64_t)p.T * (p.lda / 2) : ((int64_t)(p.T - 1) * p.lda + p.kl) * 2;

    // the k tile that is loaded next: its segment, first input, and the
    // segment's first element of A
    int iseg = 0, ik = 0, ipiece = 0;
    int64_t irank = 0, ia = 0;
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
            if (kb >= p.kpad / 16 || st >= p.wsteps) off = kOutside, at = 0;
        } else {
            at = wbase[i] + (uint32_t)(iseg * p.kpad + ik) / KST * 1024u;
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
            if constexpr (TRANS) {
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
    store_blocks<SWIGLU, NO, NBM>(p, nt * NO * WN + wave_n * NO, s.row0 + m0, s.nrows - m0, [&](auto ic, auto jc, auto near) {
        constexpr int i = decltype(ic)::value, j = decltype(jc)::value;
        if constexpr (!SWIGLU) return acc[i][j];
        else return swiglu4<decltype(near)::value>(acc[2 * i][j], acc[2 * i + 1][j]);
    });
}

template <int MODE, bool SWIGLU, bool TRANS, int TM, int BN, int NS, bool AL>
__global__ __launch_bounds__(512) void grouped_tile_kernel(Grouped p, int slots, int tiles_n, int cus) {
    using Shape = TileShape<MODE, TM, BN>;
    constexpr bool R = NS >= 3, Q = NS == 4;  // (a ring of two, three or four)
    static_assert(NS >= 2 && NS <= 4, "stages");
    __shared__ __attribute__((aligned(1024))) uint8_t sA0[Shape::A], sA1[Shape::A], sW0[Shape::W], sW1[Shape::W],
        sA2[R ? Shape::A : 4], sA3[Q ? Shape::A : 4], sW2[R ? Shape::W : 4], sW3[Q ? Shape::W : 4];
    __shared__ uint32_t sSW0[Shape::SW], sSW1[Shape::SW], sSA0[Shape::SA], sSA1[Shape::SA], sSW2[R ? Shape::SW : 1],
        sSW3[Q ? Shape::SW : 1], sSA2[R ? Shape::SA : 1], sSA3[Q ? Shape::SA : 1];
    Stages<NS> stage;
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
        grouped_tile<MODE, SWIGLU, TRANS, TM, BN, NS, AL>(p, s, nt, stage);
    } else if constexpr (TM == 256) {
        if ((int)blockIdx.x >= tiles + 4 * rest) return;
        const int q = xcd_remap(blockIdx.x - tiles, 4 * rest);
        Slot s = slot_of(tiles + q / 4, nt);
        s.row0 += (q & 1) * 128;
        s.nrows = min(s.nrows - (q & 1) * 128, 128);
        if (s.e < 0 || s.nrows <= 0) return;
        grouped_tile<MODE, SWIGLU, TRANS, 128, BN / 2, NS, AL>(p, s, 2 * nt + ((q >> 1) & 1), stage);
    }
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

__global__ __launch_bounds__(256) void pack_kernel(uint16_t* dst, const uint16_t* src, ExpertsLayout l, int64_t frags,
                                                   bool whole) {
    const int64_t fr = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (fr >= frags) return;
    const int lane = threadIdx.x & 63;
    const int64_t st = fr % l.steps, b = (fr / l.steps) % l.blocks, e = fr / (l.steps * l.blocks);
    const int64_t row = source_row(l, b * 16 + (lane & 15)), q = st * 32 + 8 * (lane >> 4);
    const uint16_t* from = src + (e * l.out + row) * l.in;
    if (whole) {  // eight inputs lie together, 16-byte aligned
        const int64_t c = row >= 0 ? source_col(l, q) : -1;
        *(u32x4*)(dst + fr * 512 + lane * 8) = c >= 0 ? *(const u32x4*)(from + c) : u32x4{0, 0, 0, 0};
        return;
    }
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
    se[mx4_scale_offset(b, st, lane & 15, l.steps) + (lane >> 4)] = s;
    if (st == l.steps - 1)  // the rest of the last run is read and not used
        for (int64_t i = l.steps; i < mx4_scale_runs(l.steps) * 4; ++i)
            se[mx4_scale_offset(b, i, lane & 15, l.steps) + (lane >> 4)] = 127;
}

template <int MODE, bool SWIGLU, int MB, int NB, int KS, int NWV, bool AL>
hipError_t stream_launch(const Grouped& p, hipStream_t s) {
    constexpr int per = NWV / KS * NB;
    const int64_t groups = (p.nout + per - 1) / per;
    const int64_t slots = p.R / (16 * MB) + (p.R < p.E ? p.R : p.E);
    if (groups * slots >= kMaxBlocks * 4 / NWV) return hipErrorInvalidConfiguration;
    launch(grouped_stream_kernel<MODE, SWIGLU, MB, NB, KS, NWV, AL>, dim3((unsigned)(groups * slots)), dim3(64 * NWV),
           0, s, p);
    return hipGetLastError();
}

// How many output blocks a wave takes, and how many waves share their inputs.
// 16-bit weights: few blocks and many waves (us, two rows and 32 rows of 8
// experts of the decode MLP, then 32 rows of 64 experts of 2048 x 1024):
//   gate|up  eight waves a pair of blocks   72 201 37   one wave for two pairs  108 211 52
//   down     eight waves for two blocks     44 108 22   four waves              69 107 22
//            four waves for four blocks     87 115 22
// MXFP4 weights spend more on turning codes into operands, which a wider group
// shares out over no more rows but which fewer waves repeat less often: the
// widest group, and the fewest waves that give every compute unit seven (gate|up
// of 32 rows, two pairs a wave: 83 us, one pair and eight waves: 158 us; down,
// four waves for four blocks 49 us, eight for two 67 us).
// Sixteen waves where compute units get one workgroup of eight at most, and each
// wave still has a run of steps, of one block where that is enough for all (us,
// eight / sixteen waves, one row of an expert; MXFP4 weights for two blocks have
// no registers for sixteen, 22 / 30 us on the first):
//                      16-bit     MXFP4     MXFP4 x MXFP4
//   2 x (4096 x 14336)  48 / 40    22         18 / 16
//   1 x (4096 x 14336)  44 / 29    19 / 15    15 / 12
//   1 x (2048 x 8192)   23 / 16    11 / 9     8.5 / 7.1
// and with half as many workgroups again as compute units 63 / 71.
// (None of this looks at alignment: how many waves share the inputs decides the
// order of the sums, and so the result's bits.)
template <int MODE, bool SWIGLU, bool AL>
hipError_t stream_mode(const Grouped& p, hipStream_t s) {
    constexpr int NB = SWIGLU ? 2 : 4;
    const int64_t blocks = (int64_t)p.nout * (p.R < p.E ? p.R : p.E), want = 7 * (int64_t)device_cus();
    // (MXFP4 activations whose scales the tiles cannot take come here with any rows:
    // the weights are read once for every 32 of them.  us of K = 1984 / the same on
    // tiles, K = 2048 / with bf16 activations: 4096 rows of 8192 weight rows 151 / 71
    // / 159, of 8 x 4096 79 / 39 / 78, 256 rows of those 14 / 10 / 15)
    if constexpr (MODE == G_MX4A4)
        if (p.R > (int64_t)8 * p.E) return stream_launch<MODE, SWIGLU, 2, NB, 1, 4, AL>(p, s);
    if constexpr (MODE < G_MX4) {
        if constexpr (!SWIGLU)
            if (blocks * 2 > want) return stream_launch<MODE, SWIGLU, 1, NB / 2, 4, 4, AL>(p, s);
    } else {
        if (blocks / NB >= want) return stream_launch<MODE, SWIGLU, 1, NB, 1, 4, AL>(p, s);
        if (blocks / NB * 2 >= want) return stream_launch<MODE, SWIGLU, 1, NB, 2, 4, AL>(p, s);
        if (blocks / NB * 4 >= want) return stream_launch<MODE, SWIGLU, 1, NB, 4, 4, AL>(p, s);
        if (blocks / NB * 8 >= want) return stream_launch<MODE, SWIGLU, 1, NB, 8, 8, AL>(p, s);
    }
    if (blocks <= NB / 2 * (int64_t)device_cus() && p.wsteps >= 64) {
        if constexpr (!SWIGLU)
            if (blocks <= (int64_t)device_cus()) return stream_launch<MODE, SWIGLU, 1, 1, 16, 16, AL>(p, s);
        if constexpr (MODE != G_MX4) return stream_launch<MODE, SWIGLU, 1, NB / 2, 16, 16, AL>(p, s);
    }
    return stream_launch<MODE, SWIGLU, 1, NB / 2, 8, 8, AL>(p, s);
}

template <int MODE, bool SWIGLU, bool TRANS, int TM, int BN, int NS, bool AL>
hipError_t tile_launch(const Grouped& p, hipStream_t s) {
    constexpr int NB = SWIGLU ? BN / 32 : BN / 16;
    const int64_t slots = p.R / TM + (p.R < p.E ? p.R : p.E);
    const int64_t tiles_n = (p.nout + NB - 1) / NB;
    const int cus = device_cus();
    const int64_t blocks = slots * tiles_n + (TM == 256 ? 3 * (cus / 2) : 0);
    if (blocks >= kMaxBlocks / 2) return hipErrorInvalidConfiguration;
    launch(grouped_tile_kernel<MODE, SWIGLU, TRANS, TM, BN, NS, AL>, dim3((unsigned)blocks), dim3(512), 0, s, p, (int)slots,
           (int)tiles_n, cus);
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
template <int MODE, bool SWIGLU, bool TRANS, bool AL>
hipError_t tile_mode(const Grouped& p, hipStream_t s) {
    if constexpr (!AL && MODE == G_MX4) {
        return tile_launch<MODE, SWIGLU, TRANS, 128, 128, 2, false>(p, s);
    } else if constexpr (!AL) {
        // Rows through registers: times round the chip, of two or three workgroups
        // a compute unit.  us, 128 x 128 / 64 x 128 / the latter in three stages:
        // 8 x (2046 x 4094) m = 125: 100 76 73   gate|up of 8 x (8188 x 2046): 131 115 123
        // 8 x (4094 x 4094) m = 500: 354 318 390   32 x (1022 x 2046) m = 188: 66 79 75
        const int64_t cus = device_cus();
        if (few_tiles<SWIGLU, 64>(p)) return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 3, false>(p, s);
        const int64_t wide = (tiles_of<SWIGLU, 128>(p) + 2 * cus - 1) / (2 * cus);
        const int64_t narrow = (tiles_of<SWIGLU, 64>(p) + 3 * cus - 1) / (3 * cus);
        if (3 * narrow <= 4 * wide) return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 2, false>(p, s);
        return tile_launch<MODE, SWIGLU, TRANS, 128, 128, 2, false>(p, s);
    } else if constexpr (MODE == G_MX4) {
        // (turning codes into operands costs the narrow tile as much as its few
        // rows' products; gate|up, 64 x 128 / 128 x 256:  m = 64: 185 222  256: 552 531  1024: 1987 1742,
        // down  64: 126 174  256: 280 364  1024: 960 938)
        const int64_t tiles = (p.R / 128 + p.E / 2) * ((p.nout + 15) / 16) * (SWIGLU ? 2 : 1);
        if (p.R >= (int64_t)192 * p.E && tiles >= (int64_t)device_cus() * 6)
            return tile_launch<MODE, SWIGLU, TRANS, 128, 256, 2, true>(p, s);
        if (few_tiles<SWIGLU, 64>(p)) return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 4, true>(p, s);
        return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 2, true>(p, s);
    } else {
        // (MXFP4 products are so short that a wave of tiles more costs them a
        // wider tile's gain: 512 rows of 8 experts, gate|up 461 429, down 221 256)
        const int64_t tiles = (p.R / 256 + p.E / 2) * ((p.nout + 15) / 16) * (SWIGLU ? 2 : 1);
        if (p.R >= (int64_t)128 * p.E && tiles * 10 >= (int64_t)device_cus() * (MODE == G_MX4A4 ? 40 : 7))
            return tile_launch<MODE, SWIGLU, TRANS, 256, 256, 2, true>(p, s);
        // (few narrow tiles go before few wide ones: 256 rows of 4096 x 4096 27 32, 500 rows
        // of 2 x (2048 x 2048) 15 19)
        if (few_tiles<SWIGLU, 64>(p)) return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 4, true>(p, s);
        if (p.R > (int64_t)40 * p.E) {
            if (few_tiles<SWIGLU, 128>(p)) return tile_launch<MODE, SWIGLU, TRANS, 128, 128, 4, true>(p, s);
            return tile_launch<MODE, SWIGLU, TRANS, 128, 128, 2, true>(p, s);
        }
        return tile_launch<MODE, SWIGLU, TRANS, 64, 128, 2, true>(p, s);
    }
}

template <int MODE, bool AL>
hipError_t by_mode(const Grouped& p, hipStream_t s) {
    if constexpr (MODE < G_MX4)
        if (p.transposed) return tile_mode<MODE, false, true, AL>(p, s);
    // (an MXFP4 row's scales are staged four at a time, by aligned 4-byte loads: rows
    // of no multiple of 128 inputs go to the streaming kernel however many they are)
    const bool tiles = p.R > (int64_t)8 * p.E && (MODE != G_MX4A4 || (p.kl % 128 == 0 && (uintptr_t)p.a_scales % 4 == 0));
    if (tiles) return p.swiglu ? tile_mode<MODE, true, false, AL>(p, s) : tile_mode<MODE, false, false, AL>(p, s);
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
    const int64_t part = l.mode == SG_ALL_TO_SHARDED ? l.in : l.in / l.S / l.P;
    launch(pack_kernel, dim3((unsigned)((frags + 3) / 4)), dim3(256), 0, s, (uint16_t*)dst, (const uint16_t*)src, l,
           frags, part % 8 == 0 && (uintptr_t)src % 16 == 0);
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
