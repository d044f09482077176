// MXFP4 quantisation: blocks of 32 values share one E8M0 scale 2^(s - 127),
// each value an E2M1 code (sign, 2 exponent bits with bias 1, 1 mantissa bit:
// 0, 0.5, 1, 1.5, 2, 3, 4, 6).
//
//   e = floor(log2 max|x|) - 2, clamped to -127 .. 127 (a block of zeros: -127)
//   code = round to nearest even of x 2^-e, magnitudes above 6 to 6
//   a block that holds an infinity or a NaN: scale 255 (NaN), codes 0
//
// Bound by HBM: the input read once, 17/32 byte written per value.  A thread
// takes 8 adjacent values (one 16-byte load of 16-bit inputs, two of fp32),
// four threads share a block's maximum through two lane exchanges.
#include "experts.h"

namespace sg {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int DT>
__global__ __launch_bounds__(256) void quantize_kernel(const void* x, int64_t n8, int64_t cols8, int64_t ld,
                                                       uint8_t* codes, uint8_t* scales) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // which 8 values; n8 is a multiple of 4
    if (i >= n8) return;
    const int64_t row = i / cols8, c = i - row * cols8;
    float v[8];
    load_cols<DT>(x, row * ld + c * 8, v, 8);
    // magnitudes compare like their bit patterns; infinities and NaNs are the largest
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2));
    const bool bad = m >= 0x7f800000u;
    // floor(log2 m): the exponent field, or for subnormal m the highest set bit
    const int top = m >= 0x00800000u ? (int)(m >> 23) - 127 : m ? (31 - __builtin_clz(m)) - 149 : -200;
    const int ex = max(top - 2, -127);
    uint32_t w = 0;
    if (!bad) {
        // x 2^-ex is exact (a power of two) unless it falls below 2^-149, where the code is 0 anyway
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = ldexpf(v[e], -ex);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[0], q[1], 1.0f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[2], q[3], 1.0f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[4], q[5], 1.0f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[6], q[7], 1.0f, 3);
    }
    *(uint32_t*)(codes + i * 4) = w;
    if ((i & 3) == 0) scales[i >> 2] = bad ? 255 : (uint8_t)(ex + 127);
}

template <int DT>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int64_t n8,
                                                         void* x) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    const uint32_t w = *(const uint32_t*)(codes + i * 4);
    const int s = scales[i >> 2];
    float v[8];
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s == 255 ? __builtin_nanf("") : ldexpf(v[e], s - 127);
    store_cols<DT>(x, i * 8, v, 8);
}

template <int DT>
void quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    const int64_t n8 = rows * (cols / 8);
    const dim3 grid((unsigned)((n8 + 255) / 256));
    launch(quantize_kernel<DT>, grid, dim3(256), 0, s, x, n8, cols / 8, ld, codes, scales);
}

}  // namespace

hipError_t launch_quantize_mxfp4(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s) {
    if (dtype == SG_F32) quantize<SG_F32>(x, rows, cols, ld, codes, scales, s);
    else if (dtype == SG_BF16) quantize<SG_BF16>(x, rows, cols, ld, codes, scales, s);
    else quantize<SG_F16>(x, rows, cols, ld, codes, scales, s);
    return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* x,
                                   int dtype, hipStream_t s) {
    const int64_t n8 = rows * (cols / 8);
    const dim3 grid((unsigned)((n8 + 255) / 256));
    if (dtype == SG_F32) launch(dequantize_kernel<SG_F32>, grid, dim3(256), 0, s, codes, scales, n8, x);
    else if (dtype == SG_BF16) launch(dequantize_kernel<SG_BF16>, grid, dim3(256), 0, s, codes, scales, n8, x);
    else launch(dequantize_kernel<SG_F16>, grid, dim3(256), 0, s, codes, scales, n8, x);
    return hipGetLastError();
}

}  // namespace sg
