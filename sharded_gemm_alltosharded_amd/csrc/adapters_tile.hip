// The shared projection's product with the adapters' part in its epilogue
// (grouped_tile.h, adapt_blocks).
#include "grouped_tile.h"

namespace sg {
namespace {

template <int MODE, bool AL>
hipError_t by_mode(const Grouped& p, const Adapted& d, hipStream_t s) {
    if (p.transposed) return tile_mode<MODE, false, true, AL, E_ADAPT>(p, s, d);
    return p.swiglu ? tile_mode<MODE, true, false, AL, E_ADAPT>(p, s, d) : tile_mode<MODE, false, false, AL, E_ADAPT>(p, s, d);
}

}  // namespace

hipError_t launch_adapted(const Grouped& p, const Adapted& d, hipStream_t s) {
    const bool al = (uintptr_t)p.A % 16 == 0 && p.lda % 8 == 0 && p.a_rank % 8 == 0 && p.kl % 8 == 0;  // as in launch_grouped
    if (p.mode == G_F16) return al ? by_mode<G_F16, true>(p, d, s) : by_mode<G_F16, false>(p, d, s);
    return al ? by_mode<G_BF16, true>(p, d, s) : by_mode<G_BF16, false>(p, d, s);
}

// From nine rows on (up to eight stream the weights faster), where tiles of 64 x 128
// give half of the compute units one.  Fewer are split over their inputs, in the plain
// grouped product (adapters_api.hip, split_product) or, of a sharded-to-all layer on
// several ranks, in the layer's own call.
bool adapted_fills(const Grouped& p) {
    return p.R > 8 && (p.swiglu ? tiles_of<true, 64>(p) : tiles_of<false, 64>(p)) * 2 > device_cus();
}

}  // namespace sg
