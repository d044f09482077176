// The gated block's products, with their halves of the block in the epilogue
// (grouped_tile.h: keep_blocks, grad_blocks), and products of few tiles split over
// their inputs.
#include "grouped_tile.h"

namespace sg {
namespace {

bool rows16(const Grouped& p) {  // as in launch_grouped
    return (uintptr_t)p.A % 16 == 0 && p.lda % 8 == 0 && p.a_rank % 8 == 0 && p.kl % 8 == 0;
}

template <bool SWIGLU, bool TRANS, int EPI>
hipError_t by_type(const Grouped& p, const Gated& g, hipStream_t s) {
    if (p.mode == G_F16)
        return rows16(p) ? tile_mode<G_F16, SWIGLU, TRANS, true, EPI>(p, s, g) : tile_mode<G_F16, SWIGLU, TRANS, false, EPI>(p, s, g);
    return rows16(p) ? tile_mode<G_BF16, SWIGLU, TRANS, true, EPI>(p, s, g) : tile_mode<G_BF16, SWIGLU, TRANS, false, EPI>(p, s, g);
}

template <int MODE, bool TRANS>
hipError_t split_mode(const Grouped& p, const Gated& g, hipStream_t s) {
    if (rows16(p)) return tile_launch<MODE, false, TRANS, 64, 128, 4, true, E_SPLIT>(p, s, g);
    return tile_launch<MODE, false, TRANS, 64, 128, 3, false, E_SPLIT>(p, s, g);
}

// the parts' sums, eight columns a thread (48 rows of 4096 x 14336: 27 us for the parts
// and 5 for this, 114 unsplit)
template <int OT>
__global__ __launch_bounds__(256) void split_sum_kernel(const float* ws, int splits, int64_t slab, int64_t N,
                                                        const int32_t* offsets, int E, int64_t R, void* out) {
    const int64_t per = (N + 7) / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= slab / N * per) return;
    const int64_t m = i / per, c = (i - m * per) * 8;
    if (offsets && (m % R < offsets[0] || m % R >= offsets[E])) return;
    const int left = (int)min(N - c, (int64_t)8);
    float v[8], w[8];
    load_cols<SG_F32>(ws, m * N + c, v, left);
    for (int q = 1; q < splits; ++q) {
        load_cols<SG_F32>(ws + q * slab, m * N + c, w, left);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
    store_cols<OT>(out, m * N + c, v, left);
}

}  // namespace

hipError_t launch_gated(const Grouped& p, const Gated& g, hipStream_t s) { return by_type<true, false, E_KEEP>(p, g, s); }
hipError_t launch_gated_backward(const Grouped& p, const Gated& g, hipStream_t s) {
    return by_type<false, true, E_GRAD>(p, g, s);
}

// Up to half a tile of 64 x 128 a compute unit: as many parts as give each one, of
// eight k tiles at least (48 rows of 4096 x 14336: 114 us on 32 tiles).
int grouped_splits(const Grouped& p) {
    const int64_t tiles = tiles_of<false, 64>(p), kts = (int64_t)p.nseg * ((p.kpad + 63) / 64);
    if (tiles * 2 > device_cus()) return 1;
    const int64_t want = device_cus() / tiles, most = kts / 8;
    return (int)(want < most ? want : most > 1 ? most : 1);
}

int64_t grouped_outputs(const Grouped& p) {
    const int ranks = p.o_rank ? p.nout / (p.bps * p.S) : 1;
    return (int64_t)p.R * p.ldo * ranks;
}

hipError_t launch_grouped_split(const Grouped& call, int splits, float* ws, hipStream_t s) {
    Grouped p = call;
    p.out = ws;
    p.out_dtype = SG_F32;
    Gated g{};
    g.splits = splits;
    g.slab = grouped_outputs(p);
    hipError_t e;
    if (p.mode == G_F16) e = p.transposed ? split_mode<G_F16, true>(p, g, s) : split_mode<G_F16, false>(p, g, s);
    else e = p.transposed ? split_mode<G_BF16, true>(p, g, s) : split_mode<G_BF16, false>(p, g, s);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((g.slab / p.ldo * ((p.ldo + 7) / 8) + 255) / 256));
    if (call.out_dtype == SG_F32)
        launch(split_sum_kernel<SG_F32>, grid, dim3(256), 0, s, ws, splits, g.slab, p.ldo, p.offsets, p.E, p.R, call.out);
    else if (call.out_dtype == SG_BF16)
        launch(split_sum_kernel<SG_BF16>, grid, dim3(256), 0, s, ws, splits, g.slab, p.ldo, p.offsets, p.E, p.R, call.out);
    else
        launch(split_sum_kernel<SG_F16>, grid, dim3(256), 0, s, ws, splits, g.slab, p.ldo, p.offsets, p.E, p.R, call.out);
    return hipGetLastError();
}

}  // namespace sg
