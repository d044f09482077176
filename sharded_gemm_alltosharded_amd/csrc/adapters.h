// Low-rank adapters beside a sharded projection: what the entry points
// (adapters_api.hip) hand to the kernels (adapters.hip).
#pragma once

#include "experts.h"

namespace sg {

// A (tokens, width) activation in the layout of P ranks and S segments: unsharded
// column (s P + r) part + c of token t at r rank + t ld + s part + c.
struct Pieces {
    int64_t rank, ld;
    int S, P, part;
};

// The plan of a step (ints): the tokens grouped by adapter (group n: those without
// one), and the groups cut into tiles of adapter_tile_rows rows.
//   offsets (n + 2), rows (T): the token of each grouped row, in token order for each
//   group, ids (T): its adapter (n: none), tiles (adapter_tiles, 4): adapter, first row,
//   rows; adapter -1 behind the last.
constexpr int kMaxAdapters = 1024, kMaxRank = 256;
// 16 rows where an adapter has few, else 64 (a tile reads its adapter's matrices once)
inline int adapter_tile_rows(int64_t T, int n) { return T >= 32 * ((int64_t)n + 1) ? 64 : 16; }
inline int64_t adapter_tiles(int64_t T, int n) {
    return T / adapter_tile_rows(T, n) + (T < n + 1 ? T : n + 1);
}
struct PlanLayout {
    int64_t offsets, rows, ids, tiles, ints;
};
inline PlanLayout plan_layout(int64_t T, int n) {
    const int64_t tiles = (n + 2 + 2 * T + 3) / 4 * 4;
    return {0, n + 2, n + 2 + T, tiles, tiles + 4 * adapter_tiles(T, n)};
}
struct Plan {
    const int32_t *offsets, *rows, *ids, *tiles;
    int T, n, ntiles, tile_rows;
};
hipError_t launch_adapter_plan(const int32_t* which, int64_t T, int n, int32_t* plan, hipStream_t s);

// Low-rank products, U (rows, rp) fp32 in `slabs` parts that are added in order, rp =
// rank rounded up to 16.  M: an adapter's matrix, (rank, width) row-major, or
// transposed (width, rank).
//
//   shrink: U[m][j] = scale_a sum over the columns k of X[t(m)][k] M[j][k]
//   expand: out[t(m)][c] = base[t(m)][c] + sum_j U[m][j] M[j][c]; tokens without an
//           adapter: base.  swiglu: column c of each rank is silu(gate) up of its
//           columns c and f + c.
//   grad:   G_a[j][c] = sum over the rows m of a of U[m][j] X[t(m)][c], laid out as M
struct LowRank {
    Plan plan;
    int f16, rank, rp, slabs;
    float* U;
    int64_t slab;  // floats
    const void* M;
    int transposed;
    int64_t width;
    const float* scale;
    const void* X;   // shrink, grad: 16 bits
    Pieces x;        // shrink, grad: of X; expand: of base (without swiglu, of out too)
    const float* base;
    int swiglu;
    void* out;       // expand: out; grad: G
    int out_dtype;
    int64_t out_rank, out_ld;  // expand
};
int shrink_slabs(const Plan& p, int64_t width, int rank);

// expand in the epilogue of the product itself (grouped_tile.h): the projection's rows
// are the plan's, and its sums never leave the registers before U's part is in.
struct Adapted {
    Plan plan;
    const uint32_t __attribute__((ext_vector_type(4)))* operands;  // finish's
    const int32_t* exponents;
    int rank;
    const void* M;    // (width, rank); of a transposed product (rank, width)
    int64_t width;
    int P;            // ranks of the output's columns: rank r's part s is the unsharded (s P + r)
    // a layer's weights, fragment-major: bytes from one input segment's, and (transposed)
    // from one rank's output columns, to the next
    uint32_t wseg, wrank;
    int again;        // segment from which on the inputs are the first ones' again (none: 0)
};
// Quantized weights (`matrices` of rows x cols, in parts of `part` rows each) as 16-bit
// tiles: 4-bit ones as two, hi and behind it lo, MX FP8 ones as one.
hipError_t launch_code_tiles(const LayerCodes& q, int f16, int64_t matrices, int64_t rows, int64_t part, int64_t cols,
                           void* out, hipStream_t s);
// transposed or not, p.rows the plan's
hipError_t launch_adapted(const Grouped& p, const Adapted& d, hipStream_t s);
// whether that beats the product's own kernel and expand behind it
bool adapted_fills(const Grouped& p);
hipError_t launch_shrink(const LowRank& p, hipStream_t s);
// The slabs added into the first; and, where operands is given, U split for the tiles'
// matrix instructions: for every 16 grouped rows and 16 ranks a lane's 16 bytes (row l &
// 15, ranks 8 (l >> 4 & 1) .. + 7, hi or from lane 32 on lo), of fp16 layers times
// 2^-exponents[row].
hipError_t launch_finish(const LowRank& p, void* operands, int32_t* exponents, hipStream_t s);
inline size_t operand_bytes(int64_t T, int rank) { return (size_t)((T + 15) / 16 * ((rank + 15) / 16) * 1024); }
hipError_t launch_expand(const LowRank& p, hipStream_t s);
hipError_t launch_grad(const LowRank& p, hipStream_t s);

#ifdef __HIPCC__
// ---- what the kernels share -------------------------------------------------
struct Tile {
    int a, row0, nrows;
};
__device__ __forceinline__ Tile tile_of(const Plan& p, int i) {
    const int32_t* e = p.tiles + 4 * (int64_t)i;
    Tile t = {__builtin_amdgcn_readfirstlane(e[0]), __builtin_amdgcn_readfirstlane(e[1]),
              __builtin_amdgcn_readfirstlane(e[2])};
    t.row0 = min(max(t.row0, 0), p.T);  // whatever a plan holds, nothing leaves the arrays
    t.nrows = min(min(t.nrows, p.T - t.row0), p.tile_rows);
    if (t.a > p.n || t.nrows <= 0) t.a = -1;
    return t;
}
__device__ __forceinline__ int token(const Plan& p, int m) { return min(max(p.rows[m], 0), p.T - 1); }

// piece q of a row, in unsharded order
__device__ __forceinline__ int64_t piece_at(const Pieces& x, int q) {
    const int s = q / x.P, r = q - s * x.P;
    return r * x.rank + (int64_t)s * x.part;
}

// eight inputs k .. k + 7 of a row whose `n` inputs start at a; zeros behind them and
// where !in.  AL: k and n are multiples of 8, the row 16-byte aligned.
template <bool AL>
__device__ __forceinline__ u32x4 row8(const uint16_t* a, const uint16_t* safe, bool in, int k, int n) {
    if constexpr (AL) {
        in = in && k < n;
        const u32x4 v = *(const u32x4*)(in ? a + k : safe);
        return in ? v : u32x4{0, 0, 0, 0};
    } else {
        return load8_any(a, in ? 0 : -1, 0, k, n);
    }
}

template <bool F16>
__device__ __forceinline__ uint16_t to16(float v) {
    if constexpr (F16) return f32_to_f16(v);
    else return f32_to_bf16(v);
}
template <bool F16>
__device__ __forceinline__ float from16(uint16_t v) {
    if constexpr (F16) return f16_to_f32(v);
    else return bf16_to_f32(v);
}
// v = hi + lo + what 16 bits more cannot hold; an infinite hi has no lo
template <bool F16>
__device__ __forceinline__ void split16(float v, uint16_t& hi, uint16_t& lo) {
    hi = to16<F16>(v);
    const float h = from16<F16>(hi);
    lo = fabsf(h) < __builtin_inff() ? to16<F16>(v - h) : 0;
}
// exponent by which fp16 operands of this largest magnitude are scaled: to 2^14 at most
__device__ __forceinline__ int range_exponent(float m) {
    return m > 0.f && m < __builtin_inff() ? (int)(__float_as_uint(m) >> 23) - 127 - 13 : 0;
}

// 32-byte pieces of an LDS row read transposed: lane (r16, c16) gets column r16 of
// rows 8 c16 .. 8 c16 + 7 (`row` = 8 c16 + (r16 >> 2)), columns from byte `col` on
__device__ __forceinline__ u32x4 read_columns(const uint8_t* s, int row, int rowb, int col) {
    const u32x2 lo = read_tr(s + row * rowb + col), hi = read_tr(s + (row + 4) * rowb + col);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
}
__device__ __forceinline__ void lds_order() { asm volatile("" ::: "memory"); }


template <typename F>
__device__ __forceinline__ void by_out_type(int dt, F&& f) {
    if (dt == SG_F32) f(std::integral_constant<int, SG_F32>{});
    else if (dt == SG_BF16) f(std::integral_constant<int, SG_BF16>{});
    else f(std::integral_constant<int, SG_F16>{});
}

// ---- launches ---------------------------------------------------------------
inline bool whole8(const void* a, int64_t ld) { return (uintptr_t)a % 16 == 0 && ld % 8 == 0; }
inline bool pieces8(const void* a, const Pieces& x) { return whole8(a, x.ld) && x.rank % 8 == 0 && x.part % 8 == 0; }

template <typename F>
hipError_t by_bool(bool b, F&& f) {
    return b ? f(std::true_type{}) : f(std::false_type{});
}
template <typename F>
hipError_t by_rank(int rank, F&& f) {
    if (rank <= 16) return f(std::integral_constant<int, 1>{});
    if (rank <= 32) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 4>{});
}
#endif

}  // namespace sg
