// The gated block on activations kept in MX FP8: what the entry points hand to the
// grouped tile kernel beside its Grouped (grouped_tile.h, experts_gated.hip).
#pragma once

#include "experts.h"

namespace sg {

// codes (P, R, 2, f) and scales (P, R, 2, mx8_blocks(f)): the kept gate and up rows.
struct Gated {
    uint8_t* codes;   // written forward, read backward
    uint8_t* scales;
    int f;            // columns of a rank
    void* h;          // backward: h again, rows of Grouped.f columns; may be null
    int splits;       // parts of a split product's inputs
    int64_t slab;     // fp32 values of a part
};

// Whether the products' epilogues do it: a scale block's two 16-column blocks must
// not belong to two ranks.
inline bool gated_fits(int64_t P, int64_t bps) { return P == 1 || bps % 2 == 0; }
// forward: p as for the SwiGLU product
hipError_t launch_gated(const Grouped& p, const Gated& g, hipStream_t s);
// backward: p as for the product dh, p.out and g.h 16-bit rows
hipError_t launch_gated_backward(const Grouped& p, const Gated& g, hipStream_t s);

// A product of few tiles, its inputs split over more workgroups: parts of fp32 sums in
// slabs of R ldo values for each rank of the output, added in order.  1: not worth it.
int grouped_splits(const Grouped& p);
int64_t grouped_outputs(const Grouped& p);  // values of a slab
hipError_t launch_grouped_split(const Grouped& p, int splits, float* ws, hipStream_t s);

#ifdef __HIPCC__
// 4 N adjacent codes of which `left` are the row's; any alignment
template <int N>
__device__ __forceinline__ void put_bytes(uint8_t* to, const uint32_t (&w)[N], int left) {
    if (left >= 4 * N) {
        __builtin_memcpy(to, w, 4 * N);
    } else {
#pragma unroll
        for (int e = 0; e < 4 * N; ++e)
            if (e < left) to[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
}
template <int N>
__device__ __forceinline__ void get_bytes(const uint8_t* from, uint32_t (&w)[N], int left) {
    if (left >= 4 * N) {
        __builtin_memcpy(w, from, 4 * N);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 0;
#pragma unroll
        for (int e = 0; e < 4 * N; ++e)
            if (e < left) w[e >> 2] |= (uint32_t)from[e] << (8 * (e & 3));
    }
}
#endif

}  // namespace sg
