// Activation checkpoints in MX FP8: blocks of 32 adjacent values of a row share
// one E8M0 scale 2^(s - 127), each value an E4M3 code (sign, 4 exponent bits with
// bias 7, 3 mantissa bits; at most 448).  The last block of a row may be short.
//
//   e = the smallest integer, -127 at least, with max|x| <= 448 2^e
//   code = round to nearest even of x 2^-e  (never above 448: nothing saturates)
//   a block that holds an infinity or a NaN: scale 255 (NaN), codes 0
//
// and SwiGLU of gate|up rows that are then kept, where the product's epilogue does not
// do it (grouped_tile.h).  All of it is bound by HBM: 4096 x 28672 bf16 quantized in 67 us
// (356 MB, 5.3 TB/s; eight values a thread are one 16-byte load and one 8-byte store),
// back in 81 us (4.4 TB/s, the writes).
#include "experts.h"

namespace sg {
namespace {

// A thread takes 8 adjacent values, four threads a block: thread i of a row's
// 4 ceil(cols / 32); those behind the row's end hold zeros and store nothing.
struct Place {
    int64_t row, c;
    int left;  // values of this thread in the row
};
__device__ __forceinline__ Place place(int64_t i, int64_t blocks, int64_t cols) {
    const int64_t row = i / (4 * blocks), c = (i - row * 4 * blocks) * 8;
    return {row, c, (int)max(min(cols - c, (int64_t)8), (int64_t)0)};
}

__device__ __forceinline__ uint32_t block_max(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, mx8_bits(v[e]));
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    return max(m, (uint32_t)__shfl_xor((int)m, 2));
}

template <bool WHOLE>
__device__ __forceinline__ void put_codes(uint8_t* codes, int64_t at, const float (&v)[8], uint32_t m, int left) {
    const int e = mx8_exponent(m);
    const bool bad = mx8_bad(m);
    uint32_t w[2] = {bad ? 0u : mx8_codes(v[0], v[1], v[2], v[3], e), bad ? 0u : mx8_codes(v[4], v[5], v[6], v[7], e)};
    if (WHOLE || left == 8) {
        __builtin_memcpy(codes + at, w, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) codes[at + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

template <bool WHOLE>
__device__ __forceinline__ void get_codes(const uint8_t* codes, int64_t at, int s, int left, float (&v)[8]) {
    uint32_t w[2] = {0, 0};
    if (WHOLE || left == 8) {
        __builtin_memcpy(w, codes + at, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) w[i >> 2] |= (uint32_t)codes[at + i] << (8 * (i & 3));
    }
    mx8_values(w[0], s, v[0], v[1], v[2], v[3]);
    mx8_values(w[1], s, v[4], v[5], v[6], v[7]);
}

// WHOLE: rows of whole blocks
template <int DT, bool WHOLE>
__global__ __launch_bounds__(256) void quantize8_kernel(const void* x, int64_t n, int64_t blocks, int64_t cols,
                                                        int64_t ld, uint8_t* codes, uint8_t* scales) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const Place p = place(i, blocks, cols);
    float v[8];
    load_cols<DT>(x, p.row * ld + p.c, v, WHOLE ? 8 : p.left);
    const uint32_t m = block_max(v);
    put_codes<WHOLE>(codes, p.row * cols + p.c, v, m, p.left);
    if ((i & 3) == 0) scales[i >> 2] = mx8_scale(m);
}

// kept16: the values were kept from DT's own.  E4M3 rounds fp16's largest ones, from 63488
// on, to 65536; they come back as 65504, half a step of fp16 away, not as infinities.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(256) void dequantize8_kernel(const uint8_t* codes, const uint8_t* scales, int64_t n,
                                                          int64_t blocks, int64_t cols, int64_t ld, void* x, bool kept16) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const Place p = place(i, blocks, cols);
    float v[8];
    get_codes<WHOLE>(codes, p.row * cols + p.c, scales[i >> 2], p.left, v);
    if (DT == SG_F16 && kept16)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fabsf(v[e]) == 65536.f ? copysignf(65504.f, v[e]) : v[e];
    store_cols<DT>(x, p.row * ld + p.c, v, WHOLE ? 8 : p.left);
}

// rows outside the experts' are left alone
__device__ __forceinline__ bool in_groups(const int32_t* offsets, int E, int64_t m) {
    return !offsets || (m >= offsets[0] && m < offsets[E]);
}

// gu (P, R, 2 f) fp32 rows [gate; up] -> h (P, R, f) = silu(gate) up and the kept
// codes (P, R, 2, f), scales
template <int DT>
__global__ __launch_bounds__(256) void gated_keep_kernel(const float* gu, int64_t n, int64_t blocks, int64_t f,
                                                         int64_t fp, int64_t R, const int32_t* offsets, int E, void* h,
                                                         uint8_t* codes, uint8_t* scales) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const Place p = place(i, blocks, f);
    if (!in_groups(offsets, E, p.row % R)) return;
    float g[8], u[8], v[8];
    load_cols<SG_F32>(gu, p.row * 2 * f + p.c, g, p.left);
    load_cols<SG_F32>(gu, p.row * 2 * f + f + p.c, u, p.left);
    const uint32_t mg = block_max(g), mu = block_max(u);
    put_codes<false>(codes, p.row * 2 * f + p.c, g, mg, p.left);
    put_codes<false>(codes, p.row * 2 * f + f + p.c, u, mu, p.left);
    if ((i & 3) == 0) {
        const int64_t b = p.c / 32;
        scales[p.row * 2 * blocks + b] = mx8_scale(mg);
        scales[p.row * 2 * blocks + blocks + b] = mx8_scale(mu);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = silu_f32(g[e]) * u[e];  // (zeros behind the row's end)
    store_cols<DT>(h, p.row * fp + p.c, v, (int)max(min(fp - p.c, (int64_t)8), (int64_t)0));
}

dim3 grid_of(int64_t n) { return dim3((unsigned)((n + 255) / 256)); }

template <typename F>
void by_type(int dtype, bool whole, F&& go) {
    auto with = [&](auto dt) {
        if (whole) go(dt, std::true_type{});
        else go(dt, std::false_type{});
    };
    if (dtype == SG_F32) with(std::integral_constant<int, SG_F32>{});
    else if (dtype == SG_BF16) with(std::integral_constant<int, SG_BF16>{});
    else with(std::integral_constant<int, SG_F16>{});
}

}  // namespace

hipError_t launch_quantize_mxfp8(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s) {
    const int64_t blocks = mx8_blocks(cols), n = rows * blocks * 4;
    by_type(dtype, cols % 32 == 0, [&](auto dt, auto whole) {
        launch(quantize8_kernel<decltype(dt)::value, decltype(whole)::value>, grid_of(n), dim3(256), 0, s, x, n, blocks,
               cols, ld, codes, scales);
    });
    return hipGetLastError();
}

hipError_t launch_dequantize_mxfp8(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* x,
                                   int64_t ld, int dtype, bool kept16, hipStream_t s) {
    const int64_t blocks = mx8_blocks(cols), n = rows * blocks * 4;
    by_type(dtype, cols % 32 == 0, [&](auto dt, auto whole) {
        launch(dequantize8_kernel<decltype(dt)::value, decltype(whole)::value>, grid_of(n), dim3(256), 0, s, codes,
               scales, n, blocks, cols, ld, x, kept16);
    });
    return hipGetLastError();
}

hipError_t launch_gated_keep(const float* gu, int64_t P, int64_t R, int64_t f, int64_t fp, const int32_t* offsets,
                             int E, void* h, int f16, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    const int64_t blocks = mx8_blocks(f), n = P * R * blocks * 4;
    if (f16)
        launch(gated_keep_kernel<SG_F16>, grid_of(n), dim3(256), 0, s, gu, n, blocks, f, fp, R, offsets, E, h, codes, scales);
    else
        launch(gated_keep_kernel<SG_BF16>, grid_of(n), dim3(256), 0, s, gu, n, blocks, f, fp, R, offsets, E, h, codes, scales);
    return hipGetLastError();
}

}  // namespace sg
