// The tiled projection kernels on 8-bit integers with row scales.
#include "linear_tile.hpp"

namespace skg_host {

int tile_kernels_int8(bool gated, TileKernel *out) { return tile_pick<skg::kInt8Row>(gated, false, out); }

}  // namespace skg_host
