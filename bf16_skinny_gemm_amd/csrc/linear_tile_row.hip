// The many-row projection kernels of one element type and scale mode.
#include "linear_tile.hpp"

namespace skg_host {

TileKernel tile_kernel_row(bool gated, bool exact, int size)
{
    return tile_pick<1>(gated, exact, size);
}

}  // namespace skg_host
