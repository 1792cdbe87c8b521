// The tiled projection kernels on e4m3 with block scales.
#include "linear_tile.hpp"

namespace skg_host {

int tile_kernels_block(bool gated, bool exact, TileKernel *out) { return tile_pick<2>(gated, exact, out); }

}  // namespace skg_host
