// The tiled projection kernels on bfloat16.
#include "linear_tile.hpp"

namespace skg_host {

int tile_kernels_bf16(bool gated, bool exact, TileKernel *out) { return tile_pick<0>(gated, exact, out); }

}  // namespace skg_host
