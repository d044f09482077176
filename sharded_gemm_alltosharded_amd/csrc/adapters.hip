// Low-rank adapters of many requests beside a sharded projection (adapters.h):
//
//   u = x A_a^T,   y += scale_a u B_a^T,   a the token's adapter
//
// and the gradients.  Tokens are grouped by adapter once a step (the plan); a tile
// is up to 16 or 64 grouped rows of one adapter.  With ranks of 8 to 64 every
// product here is bound by reading and writing the activations and the adapters'
// matrices, not by the matrix unit.
//
// u is held in fp32.  As an operand of a 16-bit matrix instruction it is split in
// two, hi + lo, side by side along the contracted dimension: 16 ranks fill the 32
// of a v_mfma_f32_16x16x32, so the second half costs nothing, and u keeps 16 bits
// (bf16) or 22 (fp16).  For fp16 a row is scaled by a power of two first, so that
// neither half leaves fp16's range.
#include "adapters.h"

namespace sg {
namespace {

// lanes of the wave whose value equals this lane's (values below 2^bits)
__device__ __forceinline__ uint64_t equal_lanes(int v, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((v >> b) & 1);
        m &= ((v >> b) & 1) ? set : ~set;
    }
    return m;
}

// ---- plan -------------------------------------------------------------------
// A stable counting sort by one workgroup (once a step, for all layers): each wave
// counts a run of tokens, the counts become first rows, each wave places its run.  More
// workgroups would want a launch each for counts and places; a step has few thousands.
__global__ __launch_bounds__(1024) void adapter_plan_kernel(const int32_t* which, int T, int n, int tile_rows,
                                                            int ntiles, int32_t* offsets, int32_t* rows,
                                                            int32_t* ids, int32_t* tiles) {
    __shared__ int first[16][kMaxAdapters + 1];  // counts, then the first row, of a wave's run and a group
    __shared__ int total[kMaxAdapters + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, groups = n + 1;
    int bits = 1;
    while ((1 << bits) <= groups) ++bits;
    for (int i = tid; i < 16 * groups; i += 1024) first[i / groups][i % groups] = 0;
    __syncthreads();
    const int run = ((T + 1023) / 1024) * 64, s0 = wave * run;
    auto group = [&](int t) {
        if (t >= T) return -1;
        const int a = which[t];
        return a >= 0 && a < n ? a : n;
    };
    for (int i = 0; i < run; i += 64) {
        const int g = group(s0 + i + lane);
        const uint64_t same = equal_lanes(g + 1, bits);
        if (g >= 0 && lane == __builtin_ctzll(same)) first[wave][g] += __builtin_popcountll(same);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    for (int g = tid; g < groups; g += 1024) {
        int sum = 0;
        for (int w = 0; w < 16; ++w) {
            const int c = first[w][g];
            first[w][g] = sum;
            sum += c;
        }
        total[g] = sum;
    }
    __syncthreads();
    if (wave == 0) {  // first rows of the groups, and their tiles
        int before = 0, tile = 0;
        for (int g0 = 0; g0 < groups; g0 += 64) {
            const int g = g0 + lane, c = g < groups ? total[g] : 0, tc = (c + tile_rows - 1) / tile_rows;
            int sum = c, tsum = tc;
            for (int d = 1; d < 64; d *= 2) {
                const int v = __shfl_up(sum, d), w = __shfl_up(tsum, d);
                if (lane >= d) sum += v, tsum += w;
            }
            const int at = before + sum - c;
            if (g < groups) {
                total[g] = at;
                offsets[g] = at;
                for (int i = 0; i < tc; ++i) {
                    int32_t* e = tiles + 4 * (int64_t)(tile + tsum - tc + i);
                    e[0] = g, e[1] = at + i * tile_rows, e[2] = min(tile_rows, c - i * tile_rows), e[3] = 0;
                }
            }
            before += __shfl(sum, 63);
            tile += __shfl(tsum, 63);
        }
        if (lane == 0) offsets[groups] = before;
        for (int i = tile + lane; i < ntiles; i += 64) tiles[4 * (int64_t)i] = -1;
    }
    __syncthreads();
    for (int i = 0; i < run; i += 64) {
        const int t = s0 + i + lane, g = group(t);
        const uint64_t same = equal_lanes(g + 1, bits);
        if (g >= 0) {
            const int at = total[g] + first[wave][g] + __builtin_popcountll(same & ((1ull << lane) - 1));
            rows[at] = t;
            ids[at] = g;
        }
        // the wave's reads of `first` are done before its update (one wave, in order)
        __builtin_amdgcn_wave_barrier();
        if (g >= 0 && lane == __builtin_ctzll(same)) first[wave][g] += __builtin_popcountll(same);
        __builtin_amdgcn_wave_barrier();
    }
}

// ---- shrink -----------------------------------------------------------------
// U[slab][m][j] = scale_a sum over the slab's columns of X[t(m)][k] M[j][k].  Bound by
// reading X (many rows of an adapter) or M (few).  Columns go in steps of 32, one MFMA;
// slabs (blockIdx.y) and the NW waves split them, a wave's steps adjacent.  TR: M is
// (width, rank): a step's 32 rows pass through LDS and are read transposed.  4096 rows of 28672
// (235 MB) in sixteen slabs 64 us, in eight 75; of 4096 columns 18 us; sixteen tokens of
// 4096 4.8 us.
template <bool F16, bool TR, int NR, int MB, bool AL>
__global__ __launch_bounds__(256) void shrink_kernel(LowRank p) {
    constexpr int NW = 4, U = NR + MB <= 6 ? 4 : 2;  // waves; steps whose loads are out at once
    // (the waves' sums go where their steps of M went)
    constexpr int RED = (NW - 1) * NR * MB * 1024, ST = TR ? NW * U * NR * 1024 : 0;
    __shared__ __attribute__((aligned(16))) uint8_t lds[RED > ST ? RED : ST];
    f32x4* red = (f32x4*)lds;
    uint8_t* stage = lds;
    const Tile tile = tile_of(p.plan, blockIdx.x);
    if (tile.a < 0 || tile.a >= p.plan.n) return;
    const int lane = threadIdx.x & 63, r16 = lane & 15, c16 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j0 = blockIdx.z * NR * 16;
    const int spp = (p.x.part + 31) / 32, steps = p.x.S * p.x.P * spp, parts = NW * p.slabs;
    const int w = blockIdx.y * NW + wave;
    const int st0 = (int)((int64_t)steps * w / parts), st1 = (int)((int64_t)steps * (w + 1) / parts);

    const uint16_t* X = (const uint16_t*)p.X;
    const uint16_t* M = (const uint16_t*)p.M + (int64_t)tile.a * p.rank * p.width;
    const uint16_t* xrow[MB];
    bool live[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        live[b] = 16 * b + r16 < tile.nrows;
        xrow[b] = X + (int64_t)(live[b] ? token(p.plan, tile.row0 + 16 * b + r16) : 0) * p.x.ld;
    }
    f32x4 acc[NR][MB];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    int q = st0 / spp, k0 = (st0 - q * spp) * 32;
    int64_t at = piece_at(p.x, q);
    for (int st = st0; st < st1; st += U) {
        u32x4 xf[U][MB], mf[U][NR];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = st + u < st1;
#pragma unroll
            for (int b = 0; b < MB; ++b) xf[u][b] = row8<AL>(xrow[b] + at, X, on && live[b], k0 + 8 * c16, p.x.part);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                if constexpr (TR) {
                    // chunk (lane + 64 i) of the step's 32 rows of 2 NR chunks of eight ranks
                    const int ch = lane + 64 * i, k = k0 + ch / (2 * NR), j = j0 + ch % (2 * NR) * 8;
                    const bool in = on && k < p.x.part && j < p.rank;
                    mf[u][i] = row8<AL>(M + ((int64_t)q * p.x.part + (in ? k : 0)) * p.rank, M, in, j, p.rank);
                } else {
                    const int j = j0 + 16 * i + r16;
                    const bool in = on && j < p.rank;
                    mf[u][i] = row8<AL>(M + (int64_t)(in ? j : 0) * p.width + (int64_t)q * p.x.part, M, in,
                                         k0 + 8 * c16, p.x.part);
                }
            }
            if (on && (k0 += 32) >= p.x.part) {
                k0 = 0;
                if (st + u + 1 < steps) at = piece_at(p.x, ++q);
            }
        }
        if constexpr (TR) {
            uint8_t* mine = stage + wave * (U * 1024 * NR);
            lds_order();
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < NR; ++i) *(u32x4*)(mine + (u * NR + i) * 1024 + lane * 16) = mf[u][i];
            lds_order();
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < NR; ++i)
                    mf[u][i] = read_columns(mine + u * NR * 1024, 8 * c16 + (r16 >> 2), 32 * NR, 32 * i + 8 * (r16 & 3));
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int b = 0; b < MB; ++b) acc[i][b] = mfma16<F16>(mf[u][i], xf[u][b], acc[i][b]);
    }
    if constexpr (TR) __syncthreads();
    if (wave > 0)
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int b = 0; b < MB; ++b) red[((wave - 1) * NR * MB + i * MB + b) * 64 + lane] = acc[i][b];
    __syncthreads();
    if (wave > 0) return;
    float* out = p.U + blockIdx.y * p.slab;
    const float scale = p.scale ? p.scale[tile.a] : 1.0f;
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            f32x4 v = acc[i][b];
#pragma unroll
            for (int o = 0; o < NW - 1; ++o) v += red[(o * NR * MB + i * MB + b) * 64 + lane];
            const int j = j0 + 16 * i + 4 * c16;
            if (live[b] && j < p.rp) *(f32x4*)(out + (int64_t)(tile.row0 + 16 * b + r16) * p.rp + j) = v * scale;
        }
}

// A wave takes 16 rows: the slabs' sum, back into the first where there are several, and
// the operands (adapters.h).  Lane l holds row l & 15, ranks 8 (l >> 4 & 1) .. + 7 of each
// sixteen; lanes 32 apart hold the same.
template <bool F16>
__global__ __launch_bounds__(256) void finish_kernel(LowRank p, u32x4* operands, int32_t* exponents) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, c16 = lane >> 4;
    const int64_t block = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), m = block * 16 + r16;
    if (block * 16 >= p.plan.T) return;
    const int chunks = p.rp / 16;
    // (rows without an adapter hold nothing)
    const bool in = m < p.plan.T && p.plan.ids[m] >= 0 && p.plan.ids[m] < p.plan.n;
    auto sum = [&](int ch, f32x4 (&v)[2]) {
        v[0] = v[1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (!in) return;
        const float* u = p.U + m * p.rp + ch * 16 + 8 * (c16 & 1);
#pragma unroll 4
        for (int q = 0; q < p.slabs; ++q) v[0] += *(const f32x4*)(u + q * p.slab), v[1] += *(const f32x4*)(u + q * p.slab + 4);
    };
    int ex = 0;
    if (F16 && operands) {
        float top = 0.f;
        for (int ch = 0; ch < chunks; ++ch) {
            f32x4 v[2];
            sum(ch, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (ch * 16 + 8 * (c16 & 1) + e < p.rank) top = fmaxf(top, fabsf(v[e >> 2][e & 3]));
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        // (products of fp16 values are 2^-48 at least; the sums scaled with it must not overflow)
        ex = max(range_exponent(top), -80);
        if (in && lane < 16) exponents[m] = ex;
    }
    for (int ch = 0; ch < chunks; ++ch) {
        f32x4 v[2];
        sum(ch, v);
        if (operands) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                uint16_t h0, l0, h1, l1;
                const int j = ch * 16 + 8 * (c16 & 1) + e;
                // (ranks behind the last hold nothing: an infinite x times zeros)
                const float a = j < p.rank ? v[e >> 2][e & 3] : 0.f, b = j + 1 < p.rank ? v[e >> 2][(e & 3) + 1] : 0.f;
                split16<F16>(F16 ? ldexpf(a, -ex) : a, h0, l0);
                split16<F16>(F16 ? ldexpf(b, -ex) : b, h1, l1);
                w[e / 2] = c16 < 2 ? h0 | ((uint32_t)h1 << 16) : l0 | ((uint32_t)l1 << 16);
            }
            operands[(block * chunks + ch) * 64 + lane] = w;
        }
        if (p.slabs > 1 && in && c16 < 2) {
            float* u = p.U + m * p.rp + ch * 16 + 8 * c16;
            *(f32x4*)u = v[0];
            *(f32x4*)(u + 4) = v[1];
        }
    }
}

// ---- quantized weights for the tiles ----------------------------------------
// 4-bit: w = scale q + bias in fp32, split in hi + lo (scale and bias are multiples of
// fp16's smallest step, 2^-24, so that fp16's two halves lose nothing of small weights
// either).  MX FP8: w = 2^s code, exact in bf16 alone, from its smallest value, 2^-133, on.
// A wave writes a 16-row block's step of 32 inputs, a lane its eight.
template <bool F16, bool MX>
__global__ __launch_bounds__(256) void code_tiles_kernel(LayerCodes q, int64_t frags, int64_t blocks, int64_t steps,
                                                       int64_t rows, int64_t part, int64_t cols, u32x4* hi, u32x4* lo) {
    const int64_t fr = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (fr >= frags) return;
    const int lane = threadIdx.x & 63;
    const int64_t st = fr % steps, b = fr / steps % blocks, m = fr / (steps * blocks);
    const int64_t bps = (part + 15) / 16, j = b % bps * 16 + (lane & 15), k = st * 32 + 8 * (lane >> 4);
    u32x4 h = {0, 0, 0, 0}, l = h;
    if (j < part && k < cols) {
        const int64_t row = m * rows + b / bps * part + j;
        if constexpr (MX) {
            const uint2 w = *(const uint2*)(q.codes8 + row * cols + k);
            const float scale = e8m0_to_f32(q.scales8[row * (cols / 32) + k / 32]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[e / 2] |= (uint32_t)to16<false>(scale * e4m3_to_f32((uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))))) << (16 * (e & 1));
            hi[fr * 64 + lane] = h;
            return;
        }
        const uint32_t w = q.codes[row * (cols / 8) + k / 8];
        const float scale = f16_to_f32(q.scales[row * (cols / 64) + k / 64]), bias = f16_to_f32(q.biases[row * (cols / 64) + k / 64]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint16_t a, c;
            split16<F16>(fmaf(scale, (float)((w >> (4 * q4_nibble_pos(e))) & 15u), bias), a, c);
            h[e / 2] |= (uint32_t)a << (16 * (e & 1));
            l[e / 2] |= (uint32_t)c << (16 * (e & 1));
        }
    }
    hi[fr * 64 + lane] = h;
    if constexpr (!MX) lo[fr * 64 + lane] = l;
}

// ---- grad -------------------------------------------------------------------
// G_a[j][c] = sum over a's rows m of U[m][j] X[t(m)][c].  Bound by reading X.
// A workgroup takes 64 columns of one adapter, its waves every eighth 32 rows: X and
// the two halves of U go through LDS, a wave's own part of it, and are read
// transposed.  For fp16 U's 32 rows are scaled by one power of two.  4096 rows of 28672
// columns: 64 us (3.7 TB/s); of 4096 columns 22 us, with four waves 38.
template <bool F16, bool TR, int NR, bool AL>
__global__ __launch_bounds__(512) void grad_kernel(LowRank p) {
    constexpr int NW = 8;
    constexpr int XB = 4096, UB = 32 * 32 * NR, WAVE = XB + 2 * UB;  // bytes of X, of a half of U
    constexpr int RED = (NW - 1) * 4 * NR * 64 * 16;
    __shared__ __attribute__((aligned(16))) uint8_t lds[NW * WAVE > RED ? NW * WAVE : RED];
    const int a = blockIdx.y, lane = threadIdx.x & 63, r16 = lane & 15, c16 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int gpp = (p.x.part + 63) / 64, q = blockIdx.x / gpp, c0 = (blockIdx.x - q * gpp) * 64, j0 = blockIdx.z * NR * 16;
    const int m0 = min(max(p.plan.offsets[a], 0), p.plan.T), m1 = max(min(p.plan.offsets[a + 1], p.plan.T), m0);
    const uint16_t* X = (const uint16_t*)p.X;
    const int64_t at = piece_at(p.x, q);
    uint8_t *sx = lds + wave * WAVE, *sh = sx + XB, *sl = sh + UB;

    f32x4 acc[4][NR];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 xv[4];
    f32x4 uv[NR][2];
    auto fetch = [&](int m) ALWAYS_INLINE {  // 32 rows from m on
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = m + 8 * i + lane / 8;
            const bool in = row < m1;
            xv[i] = row8<AL>(X + (int64_t)(in ? token(p.plan, row) : 0) * p.x.ld + at, X, in, c0 + 8 * (lane % 8), p.x.part);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int ch = lane + 64 * i, row = m + ch / (2 * NR), j = j0 + ch % (2 * NR) * 8;
            const bool in = row < m1 && j < p.rp;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                uv[i][h] = in ? *(const f32x4*)(p.U + (int64_t)row * p.rp + j + 4 * h) : f32x4{0.f, 0.f, 0.f, 0.f};
        }
    };
    int m = m0 + 32 * wave;
    if (m < m1) fetch(m);
    for (; m < m1; m += 32 * NW) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int j = j0 + (lane + 64 * i) % (2 * NR) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = j + e < p.rank ? uv[i][e >> 2][e & 3] : 0.f;
                uv[i][e >> 2][e & 3] = v;
                top = fmaxf(top, fabsf(v));
            }
        }
        [[maybe_unused]] int ex = 0;
        if constexpr (F16) {
#pragma unroll
            for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
            ex = range_exponent(top);
        }
        lds_order();
#pragma unroll
        for (int i = 0; i < 4; ++i) *(u32x4*)(sx + i * 1024 + lane * 16) = xv[i];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            u32x4 h, l;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint16_t h0, l0, h1, l1;
                const float v0 = uv[i][e >> 1][2 * (e & 1)], v1 = uv[i][e >> 1][2 * (e & 1) + 1];
                split16<F16>(F16 ? ldexpf(v0, -ex) : v0, h0, l0);
                split16<F16>(F16 ? ldexpf(v1, -ex) : v1, h1, l1);
                h[e] = h0 | ((uint32_t)h1 << 16);
                l[e] = l0 | ((uint32_t)l1 << 16);
            }
            *(u32x4*)(sh + i * 1024 + lane * 16) = h;
            *(u32x4*)(sl + i * 1024 + lane * 16) = l;
        }
        lds_order();
        if (m + 32 * NW < m1) fetch(m + 32 * NW);
        const int row = 8 * c16 + (r16 >> 2);
        u32x4 xf[4], hf[NR], lf[NR];
        // (TR, results along the ranks: plain columns; else eight adjacent columns a lane)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            xf[i] = read_columns(sx, row, 128, TR ? 32 * i + 8 * (r16 & 3) : 64 * (i >> 1) + 16 * (r16 & 3) + 8 * (i & 1));
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            hf[j] = read_columns(sh, row, 32 * NR, 32 * j + 8 * (r16 & 3));
            lf[j] = read_columns(sl, row, 32 * NR, 32 * j + 8 * (r16 & 3));
        }
        [[maybe_unused]] const float back = ldexpf(1.0f, ex);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                f32x4 v = F16 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[i][j];
                v = TR ? mfma16<F16>(lf[j], xf[i], v) : mfma16<F16>(xf[i], lf[j], v);
                v = TR ? mfma16<F16>(hf[j], xf[i], v) : mfma16<F16>(xf[i], hf[j], v);
                if constexpr (F16) acc[i][j] += v * back;
                else acc[i][j] = v;
            }
        lds_order();
    }
    __syncthreads();
    f32x4* red = (f32x4*)lds;
    if (wave > 0)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NR; ++j) red[(((wave - 1) * 4 + i) * NR + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int o = 0; o < NW - 1; ++o) acc[i][j] += red[((o * 4 + i) * NR + j) * 64 + lane];
    const int64_t base = (int64_t)a * p.rank * p.width, col0 = (int64_t)q * p.x.part;
    by_out_type(p.out_dtype, [&](auto dt) {
        constexpr int OT = decltype(dt)::value;
        static_for<0, NR>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            if constexpr (TR) {  // (width, rank): four adjacent ranks of column r16
                const int k = j0 + 16 * j + 4 * c16;
                static_for<0, 4>([&](auto ic) {
                    constexpr int i = decltype(ic)::value;
                    const int c = c0 + 16 * i + r16;
                    if (c >= p.x.part || k >= p.rank) return;
                    const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                    store_cols<OT>(p.out, base + (col0 + c) * p.rank + k, v, p.rank - k);
                });
            } else {  // (rank, width): eight adjacent columns of rank r16
                const int k = j0 + 16 * j + r16;
                if (k >= p.rank) return;
                static_for<0, 2>([&](auto ic) {
                    constexpr int i = 2 * decltype(ic)::value;
                    const int c = c0 + 16 * i + 8 * c16;
                    if (c >= p.x.part) return;
                    const f32x4 a0 = acc[i][j], a1 = acc[i + 1][j];
                    const float v[8] = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
                    store_cols<OT>(p.out, base + (int64_t)k * p.width + col0 + c, v, p.x.part - c);
                });
            }
        });
    });
}

}  // namespace

hipError_t launch_adapter_plan(const int32_t* which, int64_t T, int n, int32_t* plan, hipStream_t s) {
    const PlanLayout l = plan_layout(T, n);
    launch(adapter_plan_kernel, dim3(1), dim3(1024), 0, s, which, (int)T, n, adapter_tile_rows(T, n),
           (int)adapter_tiles(T, n), plan + l.offsets, plan + l.rows, plan + l.ids, plan + l.tiles);
    return hipGetLastError();
}

// As many slabs as give every compute unit four workgroups, of four steps a wave at
// least.  With few tokens that is what counts: a compute unit takes about 75 GB/s, so few
// of them are slow whatever their waves (16 tokens of 16 adapters, 4096 inputs: 5 us, 9 in
// one slab of sixteen waves).  At most sixteen: somebody adds them up.
int shrink_slabs(const Plan& p, int64_t width, int rank) {
    const int64_t blocks = (int64_t)p.ntiles * ((rank + 63) / 64), want = (4 * device_cus() + blocks - 1) / blocks;
    const int64_t most = width / 512 < 16 ? width / 512 : 16;
    return (int)(want < most ? want : most > 1 ? most : 1);
}

hipError_t launch_shrink(const LowRank& p, hipStream_t s) {
    const bool al = pieces8(p.X, p.x);
    const bool alm = (uintptr_t)p.M % 16 == 0 && (p.transposed ? p.rank % 8 == 0 : p.width % 8 == 0 && p.x.part % 8 == 0);
    return by_rank(p.rank, [&](auto nr) {
        constexpr int NR = decltype(nr)::value;
        const dim3 grid(p.plan.ntiles, p.slabs, (p.rank + 16 * NR - 1) / (16 * NR));
        return by_bool(p.f16, [&](auto f16) {
            return by_bool(p.transposed, [&](auto tr) {
                return by_bool(p.plan.tile_rows == 16, [&](auto few) {
                    return by_bool(al && alm, [&](auto a) {
                        launch(shrink_kernel<decltype(f16)::value, decltype(tr)::value, NR, decltype(few)::value ? 1 : 4,
                                             decltype(a)::value>, grid, dim3(256), 0, s, p);
                        return hipGetLastError();
                    });
                });
            });
        });
    });
}

hipError_t launch_finish(const LowRank& p, void* operands, int32_t* exponents, hipStream_t s) {
    if (p.slabs == 1 && !operands) return hipSuccess;
    const dim3 grid((unsigned)(((p.plan.T + 15) / 16 + 3) / 4));
    if (p.f16) launch(finish_kernel<true>, grid, dim3(256), 0, s, p, (u32x4*)operands, exponents);
    else launch(finish_kernel<false>, grid, dim3(256), 0, s, p, (u32x4*)operands, exponents);
    return hipGetLastError();
}

hipError_t launch_code_tiles(const LayerCodes& q, int f16, int64_t matrices, int64_t rows, int64_t part, int64_t cols,
                           void* out, hipStream_t s) {
    const int64_t blocks = rows / part * ((part + 15) / 16), steps = (cols + 63) / 64 * 2, frags = matrices * blocks * steps;
    u32x4 *hi = (u32x4*)out, *lo = hi + frags * 64;
    const dim3 grid((unsigned)((frags + 3) / 4));
    if (q.codes8) launch(code_tiles_kernel<false, true>, grid, dim3(256), 0, s, q, frags, blocks, steps, rows, part, cols, hi, lo);
    else if (f16) launch(code_tiles_kernel<true, false>, grid, dim3(256), 0, s, q, frags, blocks, steps, rows, part, cols, hi, lo);
    else launch(code_tiles_kernel<false, false>, grid, dim3(256), 0, s, q, frags, blocks, steps, rows, part, cols, hi, lo);
    return hipGetLastError();
}

hipError_t launch_grad(const LowRank& p, hipStream_t s) {
    const bool al = pieces8(p.X, p.x);
    return by_rank(p.rank, [&](auto nr) {
        constexpr int NR = decltype(nr)::value;
        const dim3 grid((unsigned)((p.x.part + 63) / 64 * p.x.P * p.x.S), p.plan.n, (p.rank + 16 * NR - 1) / (16 * NR));
        return by_bool(p.f16, [&](auto f16) {
            return by_bool(p.transposed, [&](auto tr) {
                return by_bool(al, [&](auto a) {
                    launch(grad_kernel<decltype(f16)::value, decltype(tr)::value, NR, decltype(a)::value>, grid, dim3(512), 0,
                           s, p);
                    return hipGetLastError();
                });
            });
        });
    });
}

}  // namespace sg
