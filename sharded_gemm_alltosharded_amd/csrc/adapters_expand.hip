// The second half of a low-rank adapter's product (adapters.h): U's rows through an
// adapter's matrix, added to the shared projection's result.
#include "adapters.h"

namespace sg {
namespace {

// ---- expand -----------------------------------------------------------------
// out[t(m)][c] = base[t(m)][c] + sum_j U[m][j] M[c][j].  Bound by reading
// base and writing out.  A wave takes groups of 32 adjacent columns of one piece for
// all rows of the tile; M's columns are dealt to the MFMA's rows so that a lane ends
// up with eight adjacent ones (block i, row 4 c + e: column 8 c + 4 i + e).  TR: M is
// (rank, width), read transposed through LDS.  Eight tokens of 4096 outputs, rank 32:
// 7 us, the launch and two dependent loads.
template <bool F16, bool TR, int NR, int MB, bool SWIGLU, bool ALM>
__global__ __launch_bounds__(256) void expand_kernel(LowRank p, int groups, int per, int subs) {
    constexpr int H = SWIGLU ? 2 : 1;  // gate and up
    __shared__ __attribute__((aligned(16))) uint8_t stage[TR ? 4 * NR * 1024 : 16];
    // (a tile of more than 16 MB rows is several workgroups')
    Tile tile = tile_of(p.plan, blockIdx.x / subs);
    tile.row0 += blockIdx.x % subs * 16 * MB;
    tile.nrows = min(tile.nrows - (int)(blockIdx.x % subs) * 16 * MB, 16 * MB);
    if (tile.a < 0 || tile.nrows <= 0) return;
    const bool adapted = tile.a < p.plan.n;
    if (!adapted && p.base == p.out) return;  // there already
    const int lane = threadIdx.x & 63, r16 = lane & 15, c16 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = p.x.part, gpp = (part + 31) / 32, chunks = (p.rank + NR * 16 - 1) / (NR * 16);
    const uint16_t* M = (const uint16_t*)p.M + (adapted ? (int64_t)tile.a * p.rank * p.width : 0);

    int64_t t[MB];
    bool live[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        live[b] = 16 * b + r16 < tile.nrows;
        t[b] = live[b] ? token(p.plan, tile.row0 + 16 * b + r16) : 0;
    }
    // this lane's operands of the rows: ranks 8 (c16 & 1) .. + 7 of each sixteen, hi
    // (c16 < 2) or lo, for fp16 times 2^-ex
    u32x4 uf[NR][MB];
    [[maybe_unused]] float back[MB];
    auto load_u = [&](int ch) ALWAYS_INLINE {
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            float v[NR][8];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int j = (ch * NR + i) * 16 + 8 * (c16 & 1);
                f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
                if (live[b] && j < p.rp) {
                    const float* u = p.U + (int64_t)(tile.row0 + 16 * b + r16) * p.rp + j;
#pragma unroll 4
                    for (int q = 0; q < p.slabs; ++q) lo += *(const f32x4*)(u + q * p.slab), hi += *(const f32x4*)(u + q * p.slab + 4);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // (ranks behind the last hold nothing: an infinite x times zeros)
                    v[i][e] = j + e < p.rank ? (e < 4 ? lo[e] : hi[e - 4]) : 0.f;
                    top = fmaxf(top, fabsf(v[i][e]));
                }
            }
            int ex = 0;
            if constexpr (F16) {
                top = fmaxf(top, __shfl_xor(top, 16));
                ex = range_exponent(top);
                back[b] = ldexpf(1.0f, ex);
            }
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    uint16_t h0, l0, h1, l1;
                    split16<F16>(F16 ? ldexpf(v[i][e], -ex) : v[i][e], h0, l0);
                    split16<F16>(F16 ? ldexpf(v[i][e + 1], -ex) : v[i][e + 1], h1, l1);
                    uf[i][b][e / 2] = c16 < 2 ? h0 | ((uint32_t)h1 << 16) : l0 | ((uint32_t)l1 << 16);
                }
        }
    };
    if (adapted && chunks == 1) load_u(0);

    const int g1 = min((int)(blockIdx.y + 1) * per, groups);
    for (int g = blockIdx.y * per + wave; g < g1; g += 4) {
        // (with swiglu the groups count rank r's gate columns)
        const int q = g / gpp, c0 = (g - q * gpp) * 32;
        const int s = SWIGLU ? 0 : q / p.x.P, r = SWIGLU ? q : q - s * p.x.P;
        f32x4 sum[H][2][MB];
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int b = 0; b < MB; ++b) sum[h][i][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (adapted)
            for (int ch = 0; ch < chunks; ++ch) {
                if (chunks > 1) load_u(ch);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int64_t col0 = (int64_t)((SWIGLU ? h : s) * p.x.P + r) * part;  // unsharded
                    u32x4 mf[NR][2];
                    if constexpr (TR) {
                        uint8_t* mine = stage + wave * NR * 1024;
#pragma unroll
                        for (int i = 0; i < NR; ++i) {
                            const int j = (ch * NR + i) * 16 + lane / 4;
                            const bool in = j < p.rank;
                            mf[i][0] = row8<ALM>(M + (int64_t)(in ? j : 0) * p.width + col0, M, in, c0 + 8 * (lane % 4), part);
                        }
                        lds_order();
#pragma unroll
                        for (int i = 0; i < NR; ++i) *(u32x4*)(mine + i * 1024 + lane * 16) = mf[i][0];
                        lds_order();
#pragma unroll
                        for (int i = 0; i < NR; ++i)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                mf[i][k] = read_columns(mine + i * 1024, 8 * (c16 & 1) + (r16 >> 2), 64,
                                                        16 * (r16 & 3) + 8 * k);
                    } else {
#pragma unroll
                        for (int i = 0; i < NR; ++i)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int c = c0 + 8 * (r16 >> 2) + 4 * k + (r16 & 3), j = (ch * NR + i) * 16 + 8 * (c16 & 1);
                                const bool in = c < part && j < p.rank;
                                mf[i][k] = row8<ALM>(M + (in ? col0 + c : 0) * p.rank, M, in, j, p.rank);
                            }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int b = 0; b < MB; ++b) {
                            f32x4 a = F16 ? f32x4{0.f, 0.f, 0.f, 0.f} : sum[h][k][b];
#pragma unroll
                            for (int i = 0; i < NR; ++i) a = mfma16<F16>(mf[i][k], uf[i][b], a);
                            if constexpr (F16) sum[h][k][b] += a * back[b];
                            else sum[h][k][b] = a;
                        }
                }
            }
        const int c = c0 + 8 * c16, left = min(part - c, 8);
        if (left <= 0) continue;
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            if (!live[b]) continue;
            float v[8], w[8];
            const int64_t at = r * p.x.rank + t[b] * p.x.ld + (int64_t)s * part + c;
            load_cols<SG_F32>(p.base, at, v, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += sum[0][e >> 2][b][e & 3];
            if constexpr (SWIGLU) {
                load_cols<SG_F32>(p.base, at + part, w, left);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = silu_f32(v[e]) * (w[e] + sum[H - 1][e >> 2][b][e & 3]);
            }
            by_out_type(p.out_dtype, [&](auto ot) {
                store_cols<decltype(ot)::value>(p.out, r * p.out_rank + t[b] * p.out_ld + (int64_t)s * part + c, v, left);
            });
        }
    }
}

}  // namespace

hipError_t launch_expand(const LowRank& p, hipStream_t s) {
    const bool alm = (uintptr_t)p.M % 16 == 0 && (p.transposed ? p.width % 8 == 0 && p.x.part % 8 == 0 : p.rank % 8 == 0);
    const int groups = (int)((p.x.part + 31) / 32) * p.x.P * (p.swiglu ? 1 : p.x.S);
    // sixteen groups a workgroup where the chip is filled all the same, else four
    const int per = (int64_t)p.plan.ntiles * groups >= (int64_t)64 * device_cus() ? 16 : 4;
    return by_rank(p.rank, [&](auto nr) {
        constexpr int NR = decltype(nr)::value;
        return by_bool(p.f16, [&](auto f16) {
            return by_bool(p.plan.tile_rows == 16, [&](auto few) {
                // (four blocks of ranks and of rows have more operands than registers)
                constexpr int MB = decltype(few)::value ? 1 : NR == 4 ? 2 : 4;
                const int subs = p.plan.tile_rows / (16 * MB);
                const dim3 grid(p.plan.ntiles * subs, (groups + per - 1) / per);
                return by_bool(alm, [&](auto al) {
                    auto go = [&](auto tr, auto sw) {
                        launch(expand_kernel<decltype(f16)::value, decltype(tr)::value, NR, MB, decltype(sw)::value,
                                             decltype(al)::value>, grid, dim3(256), 0, s, p, groups, per, subs);
                        return hipGetLastError();
                    };
                    if (p.transposed) return go(std::true_type{}, std::false_type{});
                    return p.swiglu ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
                });
            });
        });
    });
}

}  // namespace sg
