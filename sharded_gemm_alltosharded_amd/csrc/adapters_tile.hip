// The shared projection's product with the adapters' part in its epilogue
// (grouped_tile.h, adapt_blocks).
#include "grouped_tile.h"

namespace sg {
namespace {

template <int MODE>
hipError_t by_mode(const Grouped& p, const Adapted& d, hipStream_t s) {
    if (p.transposed) return tile_mode<MODE, false, true, true, E_ADAPT>(p, s, d);
    return p.swiglu ? tile_mode<MODE, true, false, true, E_ADAPT>(p, s, d) : tile_mode<MODE, false, false, true, E_ADAPT>(p, s, d);
}

}  // namespace

hipError_t launch_adapted(const Grouped& p, const Adapted& d, hipStream_t s) {
    return p.mode == G_F16 ? by_mode<G_F16>(p, d, s) : by_mode<G_BF16>(p, d, s);
}

// From nine rows on (up to eight stream the weights faster), where tiles of 64 x 128
// give half of the compute units one: fewer are split over their inputs by the layer's
// own call.
bool adapted_fills(const Grouped& p) {
    return p.R > 8 && (p.swiglu ? tiles_of<true, 64>(p) : tiles_of<false, 64>(p)) * 2 > device_cus();
}

}  // namespace sg
