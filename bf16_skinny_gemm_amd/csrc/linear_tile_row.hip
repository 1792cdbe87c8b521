// The tiled projection kernels on e4m3 with row scales.
#include "linear_tile.hpp"

namespace skg_host {

int tile_kernels_row(bool gated, bool exact, TileKernel *out) { return tile_pick<1>(gated, exact, out); }

}  // namespace skg_host
