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

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

namespace {

template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 w, u32x4 a, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, a), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, a),
                                                       c, 0, 0, 0);
}

// A tile row is 256 bytes (128 columns) in LDS; its 32-byte pieces are
// XOR-swizzled so that the sixteen rows one transposed read touches
// (8 c + 0 .. 3 for c = 0 .. 3) spread over all eight.
__device__ __forceinline__ int swz(int row) { return (row & 3) | (((row >> 3) & 1) << 2); }

__device__ __forceinline__ u32x2 read_tr(const uint16_t* p) {
    return __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// 128 x 128 outputs, four waves of 64 x 64, 64 rows a tile, staged through
// registers into two LDS buffers.
template <bool F16, bool AL>
__global__ __launch_bounds__(256) void grouped_dw_kernel(GroupedDw p, int tiles_o, int tiles_i) {
    __shared__ __attribute__((aligned(1024))) uint16_t sG[2][64 * 128], sX[2][64 * 128];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tile = xcd_remap(blockIdx.x, gridDim.x);
    const int per = tiles_o * tiles_i;
    const int er = tile / per, tin = tile - er * per;
    const int e = er / p.P, r = er - e * p.P;
    constexpr int GM = 8;
    const int g = tin / (GM * tiles_i), first = g * GM, gsz = min(GM, tiles_o - first);
    const int tt = tin - g * GM * tiles_i;
    const int o0 = (first + tt % gsz) * 128, i0 = tt / gsz * 128;
    int m0 = 0, m1 = p.R;
    if (p.offsets) {
        m0 = min(max(p.offsets[e], 0), p.R);
        m1 = max(min(p.offsets[e + 1], p.R), m0);
    }
    const uint16_t* G = (const uint16_t*)p.G + r * p.g_rank;
    const uint16_t* X = (const uint16_t*)p.X + r * p.x_rank;

    // thread: chunk tid & 15 (8 columns) of rows (tid >> 4) + 16 i
    const int ch = tid & 15;
    u32x4 rg[4], rx[4];
    auto load8 = [&](const uint16_t* a, int64_t row, int64_t ld, int c, int n) -> u32x4 {
        if constexpr (AL) {
            if (row < 0 || c >= n) return u32x4{0, 0, 0, 0};
            return *(const u32x4*)(a + row * ld + c);
        } else {
            uint32_t h[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) h[q] = row >= 0 && c + q < n ? a[row * ld + c + q] : 0;
            return u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
        }
    };
    auto load = [&](int mt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = mt + (tid >> 4) + 16 * i;
            rg[i] = load8(G, m < m1 ? m : -1, p.ldg, o0 + 8 * ch, p.O);
            rx[i] = load8(X, m < m1 ? grouped_row(p.rows, p.kdiv, p.T, m) : -1, p.ldx, i0 + 8 * ch, p.I);
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = (tid >> 4) + 16 * i;
            const int at = m * 128 + ((ch ^ (swz(m) << 1)) << 3);
            *(u32x4*)(sG[buf] + at) = rg[i];
            *(u32x4*)(sX[buf] + at) = rx[i];
        }
    };

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int c16 = lane >> 4, r16 = lane & 15;
    const int wo = (wave & 1) * 64, wi = (wave >> 1) * 64;
    // operand of columns col .. col + 15: contracted rows 32 kk + 8 c16 + 0 .. 7
    auto operand = [&](const uint16_t* s, int col, int kk) -> u32x4 {
        const int row = 32 * kk + 8 * c16 + (r16 >> 2);
        const int c = (col >> 3) + ((r16 & 3) >> 1);  // 16-byte chunk
        const uint16_t* a = s + 4 * (r16 & 1);
        const u32x2 lo = read_tr(a + row * 128 + ((c ^ (swz(row) << 1)) << 3));
        const u32x2 hi = read_tr(a + (row + 4) * 128 + ((c ^ (swz(row + 4) << 1)) << 3));
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };

    if (m0 < m1) {
        load(m0);
        stage(0);
        __syncthreads();
        int buf = 0;
        for (int mt = m0; mt < m1; mt += 64, buf ^= 1) {
            if (mt + 64 < m1) load(mt + 64);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                u32x4 gf[4], xf[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    xf[i] = operand(sX[buf], wi + 16 * i, kk);
                    gf[i] = operand(sG[buf], wo + 16 * i, kk);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = mfma16<F16>(xf[i], gf[j], acc[i][j]);
            }
            if (mt + 64 < m1) stage(buf ^ 1);
            __syncthreads();
        }
    }

    // lane: output row o = .. + r16, columns 4 c16 .. + 3 of each block
    const int64_t base = (int64_t)er * p.O * p.I;
    static_for<0, 4>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        const int o = o0 + wo + 16 * j + r16;
        if (o >= p.O) return;
        static_for<0, 4>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            const int c = i0 + wi + 16 * i + 4 * c16;
            if (c >= p.I) return;
            const int64_t at = base + (int64_t)o * p.I + c;
            const f32x4 v = acc[i][j];
            if (p.vec) {
                if (p.out_dtype == SG_F32) {
                    *(f32x4*)((float*)p.out + at) = v;
                } else {
                    u32x2 w;
                    if (p.out_dtype == SG_BF16) {
                        w[0] = f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16);
                        w[1] = f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16);
                    } else {
                        w[0] = f32_to_f16(v[0]) | ((uint32_t)f32_to_f16(v[1]) << 16);
                        w[1] = f32_to_f16(v[2]) | ((uint32_t)f32_to_f16(v[3]) << 16);
                    }
                    *(u32x2*)((uint16_t*)p.out + at) = w;
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < p.I) store_from_f32(p.out, p.out_dtype, at + q, v[q]);
            }
        });
    });
}

}  // namespace

hipError_t launch_grouped_dw(const GroupedDw& p, hipStream_t s) {
    const int64_t to = (p.O + 127) / 128, ti = (p.I + 127) / 128;
    const int64_t blocks = (int64_t)p.E * p.P * to * ti;
    if (blocks >= kMaxBlocks) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks);
    const bool al = (uintptr_t)p.G % 16 == 0 && (uintptr_t)p.X % 16 == 0 && p.ldg % 8 == 0 && p.ldx % 8 == 0 &&
                    p.g_rank % 8 == 0 && p.x_rank % 8 == 0 && p.O % 8 == 0 && p.I % 8 == 0;
    auto go = [&](auto f16, auto a) {
        launch(grouped_dw_kernel<decltype(f16)::value, decltype(a)::value>, grid, dim3(256), 0, s, p, (int)to, (int)ti);
    };
    using T = std::true_type;
    using F = std::false_type;
    if (p.f16) al ? go(T{}, T{}) : go(T{}, F{});
    else al ? go(F{}, T{}) : go(F{}, F{});
    return hipGetLastError();
}

}  // namespace sg
