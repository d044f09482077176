// Grouped products of a mixture of experts (experts.h, Grouped), and the
// layout of an expert layer's weights.
#include "grouped_tile.h"

namespace sg {
namespace {

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
