// Weight gradients of a grouped layer (experts.h, GroupedDw):
//
//   dW[e][r][o][i] = sum over expert e's rows m of G_r[m][o] X_r[row(m)][i]
//
// The contracted dimension is the rows, so both operands lie in memory across
// it: their tiles are staged in LDS as rows, and ds_read_b64_tr_b16 hands each
// lane four rows of one column, two of them the eight contracted values of an
// MFMA operand.
#include "experts.h"

namespace sg {


namespace {

// A tile row's 32-byte pieces are XOR-swizzled in LDS so that the sixteen rows
// one transposed read touches (8 c + 0 .. 3 for c = 0 .. 3) spread over all
// banks.
__device__ __forceinline__ int swz(int row) { return (row & 3) | (((row >> 3) & 1) << 2); }

// TO x TI outputs, WO x WI waves, 64 contracted rows a tile, two LDS stages
// filled straight from memory as in the grouped tile kernel (experts.hip).  The
// gather map's entries are read two tiles ahead, so that no load waits for its
// own address (4096 tokens, 8 experts, 28672 x 4096: 12.3 ms when it did).
// Experts without rows get zeros.
template <bool F16, int TO, int TI, int WO, int WI, bool AL>
__global__ __launch_bounds__(64 * WO * WI) void grouped_dw_kernel(GroupedDw p, int tiles_o, int tiles_i) {
    constexpr int NWV = WO * WI, NBO = TO / WO / 16, NBI = TI / WI / 16;
    constexpr int LG = 64 * TO * 2 / 1024 / NWV, LX = 64 * TI * 2 / 1024 / NWV;  // 1 KB loads of a wave
    constexpr int CG = TO / 8, CX = TI / 8;                                    // 16-byte chunks of a row
    __shared__ __attribute__((aligned(1024))) uint8_t sG0[64 * TO * 2], sG1[64 * TO * 2], sX0[64 * TI * 2],
        sX1[64 * TI * 2];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // every XCD takes a run of tiles of every expert: experts differ in rows
    // (whole experts to an XCD: 4.5 ms where this takes 2.4)
    const int per = tiles_o * tiles_i, run = (per + 7) / 8;
    const int er = (blockIdx.x / 8) / run, tin = (blockIdx.x % 8) * run + (blockIdx.x / 8) % run;
    if (tin >= per) return;
    const int e = er / p.P, r = er - e * p.P;
    constexpr int GM = 4;
    const int g = tin / (GM * tiles_i), first = g * GM, gsz = min(GM, tiles_o - first);
    const int tt = tin - g * GM * tiles_i;
    const int o0 = (first + tt % gsz) * TO, i0 = tt / gsz * TI;
    int m0 = 0, m1 = p.R;
    if (p.offsets) {
        m0 = min(max(p.offsets[e], 0), p.R);
        m1 = max(min(p.offsets[e + 1], p.R), m0);
    }
    const uint16_t* G = (const uint16_t*)p.G + r * p.g_rank;
    const uint16_t* X = (const uint16_t*)p.X + r * p.x_rank;
    const __amdgpu_buffer_rsrc_t bg = buffer(G, ((int64_t)(p.R - 1) * p.ldg + p.O) * 2);
    const __amdgpu_buffer_rsrc_t bx = buffer(X, ((int64_t)(p.T - 1) * p.ldx + p.I) * 2);

    // load i of a wave: tile row (i NWV + wave) 64 / C + lane / C, LDS chunk lane
    // % C.  Byte offsets within a tile stay in registers; the tile's own is a
    // scalar, or with a gather map its row's product.
    int gcol[LG], xcol[LX], raw[LX];
    uint32_t goff[LG], xoff[LX];
#pragma unroll
    for (int i = 0; i < LG; ++i) {
        const int m = (i * NWV + wave) * (64 / CG) + lane / CG;
        gcol[i] = o0 + 8 * ((lane % CG) ^ (swz(m) << 1));
        goff[i] = gcol[i] < p.O ? (uint32_t)((m * p.ldg + gcol[i]) * 2) : kOutside;
    }
#pragma unroll
    for (int i = 0; i < LX; ++i) {
        const int m = (i * NWV + wave) * (64 / CX) + lane / CX;
        xcol[i] = i0 + 8 * ((lane % CX) ^ (swz(m) << 1));
        xoff[i] = xcol[i] < p.I ? (uint32_t)(((p.rows ? 0 : m * p.ldx) + xcol[i]) * 2) : kOutside;
    }
    auto fetch_rows = [&](int mt) ALWAYS_INLINE {  // the gather map of tile mt
        if (!p.rows) return;
#pragma unroll
        for (int i = 0; i < LX; ++i) {
            const int m = mt + (i * NWV + wave) * (64 / CX) + lane / CX;
            raw[i] = p.rows[min(m, p.R - 1)];
        }
    };
    // (rows of any alignment go through registers, into LDS when the tile at hand is done)
    [[maybe_unused]] u32x4 gv[LG], xv[LX];
    auto put_rows = [&](uint8_t* g, uint8_t* x) ALWAYS_INLINE {
        if constexpr (!AL) {
#pragma unroll
            for (int i = 0; i < LG; ++i) *(u32x4*)(g + (i * NWV + wave) * 1024 + lane * 16) = gv[i];
#pragma unroll
            for (int i = 0; i < LX; ++i) *(u32x4*)(x + (i * NWV + wave) * 1024 + lane * 16) = xv[i];
        }
    };
    auto load_g = [&](int mt, uint8_t* s) ALWAYS_INLINE {
        const uint32_t at = mt < m1 ? (uint32_t)(mt * p.ldg * 2) : 0;
#pragma unroll
        for (int i = 0; i < LG; ++i) {
            const int m = mt + (i * NWV + wave) * (64 / CG) + lane / CG;
            if constexpr (AL) dma16(bg, m < m1 ? goff[i] : kOutside, at, s + (i * NWV + wave) * 1024);
            else gv[i] = load8_any(G, m < m1 ? m : -1, p.ldg, gcol[i], p.O);
        }
    };
    auto load_x = [&](int mt, uint8_t* s) ALWAYS_INLINE {
        const uint32_t at = p.rows || mt >= m1 ? 0 : (uint32_t)(mt * p.ldx * 2);
#pragma unroll
        for (int i = 0; i < LX; ++i) {
            const int m = mt + (i * NWV + wave) * (64 / CX) + lane / CX;
            int row = m;
            if (p.rows) row = raw[i] < 0 ? -1 : p.kmul ? (int)(__umulhi((uint32_t)raw[i], p.kmul) >> p.kshift) : raw[i];
            const bool in = m < m1 && row >= 0 && row < p.T;
            if constexpr (AL) {
                uint32_t off = xoff[i];
                if (p.rows) off = xcol[i] < p.I ? off + (uint32_t)row * (uint32_t)(p.ldx * 2) : kOutside;
                dma16(bx, in ? off : kOutside, at, s + (i * NWV + wave) * 1024);
            } else {
                xv[i] = load8_any(X, in ? row : -1, p.ldx, xcol[i], p.I);
            }
        }
    };

    f32x4 acc[NBI][NBO];
#pragma unroll
    for (int i = 0; i < NBI; ++i)
#pragma unroll
        for (int j = 0; j < NBO; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int c16 = lane >> 4, r16 = lane & 15;
    const int wo = (wave % WO) * (TO / WO), wi = (wave / WO) * (TI / WI);
    // contracted rows 32 kk + 8 c16 + 0 .. 7 of columns col .. col + 15
    auto operand = [&](const uint8_t* s, int col, int kk) ALWAYS_INLINE -> u32x4 {
        constexpr int rowb = TO * 2;
        const int row = 32 * kk + 8 * c16 + (r16 >> 2);  // (row + 4 has the same swizzle)
        const int c = (col >> 3) + ((r16 & 3) >> 1);
        const uint8_t* a = s + row * rowb + ((c ^ (swz(row) << 1)) << 4) + 8 * (r16 & 1);
        const u32x2 lo = read_tr(a), hi = read_tr(a + 4 * rowb);
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    // X's columns are dealt to the MFMA's rows so that a lane ends up with eight
    // adjacent ones of two blocks: block i, row 4 c + e is column 32 (i / 2) + 8 c
    // + 4 (i % 2) + e of the wave's (16-byte stores in place of 8-byte ones)
    auto operand_x = [&](const uint8_t* s, int i, int kk) ALWAYS_INLINE -> u32x4 {
        constexpr int rowb = TI * 2;
        const int row = 32 * kk + 8 * c16 + (r16 >> 2);
        const int c = (wi >> 3) + 4 * (i >> 1) + (r16 & 3);
        const uint8_t* a = s + row * rowb + ((c ^ (swz(row) << 1)) << 4) + 8 * (i & 1);
        const u32x2 lo = read_tr(a), hi = read_tr(a + 4 * rowb);
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    auto step = [&](int mt, const uint8_t* sG, const uint8_t* sX, uint8_t* nG, uint8_t* nX) ALWAYS_INLINE {
        stage_barrier();
        static_for<0, 2>([&](auto kc) ALWAYS_INLINE {
            constexpr int kk = decltype(kc)::value;
            u32x4 gf[NBO], xf[NBI];
#pragma unroll
            for (int i = 0; i < NBI; ++i) xf[i] = operand_x(sX, i, kk);
#pragma unroll
            for (int j = 0; j < NBO; ++j) gf[j] = operand(sG, wo + 16 * j, kk);
            // (past the last tile: zeros, into a stage never read)
            if constexpr (kk == 0) load_x(mt + 64, nX);
            else {
                load_g(mt + 64, nG);
                fetch_rows(mt + 128);
            }
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int j = 0; j < NBO; ++j)
#pragma unroll
                for (int i = 0; i < NBI; ++i) acc[i][j] = mfma16<F16>(xf[i], gf[j], acc[i][j]);
            __builtin_amdgcn_s_setprio(0);
        });
        put_rows(nG, nX);
    };
    if (m0 < m1) {
        fetch_rows(m0);
        load_x(m0, sX0);
        load_g(m0, sG0);
        put_rows(sG0, sX0);
        fetch_rows(m0 + 64);
        for (int mt = m0; mt < m1; mt += 128) {
            step(mt, sG0, sX0, sG1, sX1);
            if (mt + 64 < m1) step(mt + 64, sG1, sX1, sG0, sX0);
        }
        wait_loads();  // none may still be writing this workgroup's LDS when it ends
    }

    const int64_t base = (int64_t)er * p.O * p.I;
    auto put = [&](auto dt) ALWAYS_INLINE {
        constexpr int DT = decltype(dt)::value;
        static_for<0, NBO>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            const int o = o0 + wo + 16 * j + r16;
            if (o >= p.O) return;
            static_for<0, NBI / 2>([&](auto ic) {
                constexpr int i = 2 * decltype(ic)::value;
                const int c = i0 + wi + 16 * i + 8 * c16;
                if (c >= p.I) return;
                const f32x4 a = acc[i][j], b = acc[i + 1][j];
                const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                store_cols<DT>(p.out, base + (int64_t)o * p.I + c, v, p.I - c);
            });
        });
    };
    if (p.out_dtype == SG_BF16) put(std::integral_constant<int, SG_BF16>{});
    else if (p.out_dtype == SG_F16) put(std::integral_constant<int, SG_F16>{});
    else put(std::integral_constant<int, SG_F32>{});
}

template <bool F16, int TO, int TI, int WO, int WI, bool AL>
hipError_t dw_launch(const GroupedDw& p, hipStream_t s) {
    const int64_t to = (p.O + TO - 1) / TO, ti = (p.I + TI - 1) / TI;
    const int64_t blocks = (int64_t)p.E * p.P * ((to * ti + 7) / 8 * 8);
    if (blocks >= kMaxBlocks / 2) return hipErrorInvalidConfiguration;
    launch(grouped_dw_kernel<F16, TO, TI, WO, WI, AL>, dim3((unsigned)blocks), dim3(64 * WO * WI), 0, s, p, (int)to,
           (int)ti);
    return hipGetLastError();
}

template <bool F16>
hipError_t dw_type(const GroupedDw& p, hipStream_t s) {
    const bool al = (uintptr_t)p.G % 16 == 0 && (uintptr_t)p.X % 16 == 0 && p.ldg % 8 == 0 && p.ldx % 8 == 0 &&
                    p.g_rank % 8 == 0 && p.x_rank % 8 == 0 && p.O % 8 == 0 && p.I % 8 == 0;
    if (!al) return dw_launch<F16, 128, 128, 2, 4, false>(p, s);
    // the wide tile where its tiles go round the chip several times (8 experts
    // of 28672 x 4096: 2.30 ms, 2.72 on the narrow one; 32 of 1024 x 704 over
    // 1500 x 4 rows, twice round: 35 us, 28 on the narrow one)
    const int64_t big = (int64_t)p.E * p.P * ((p.O + 255) / 256) * ((p.I + 255) / 256);
    if (big >= 4 * device_cus()) return dw_launch<F16, 256, 256, 2, 4, true>(p, s);
    return dw_launch<F16, 128, 128, 2, 4, true>(p, s);
}

}  // namespace

hipError_t launch_grouped_dw(const GroupedDw& call, hipStream_t s) {
    GroupedDw p = call;
    // slot / kdiv as a multiplication: exact for slots below 2^31 (the error of
    // kmul, at most kdiv, times a slot stays below 2^(32 + kshift))
    if (p.kdiv > 1) {
        int log = 31 - __builtin_clz((unsigned)p.kdiv);
        if ((p.kdiv & (p.kdiv - 1)) == 0) --log;
        p.kshift = log;
        p.kmul = (uint32_t)((1ull << (32 + log)) / (unsigned)p.kdiv + 1);
    }
    return p.f16 ? dw_type<true>(p, s) : dw_type<false>(p, s);
}

}  // namespace sg
