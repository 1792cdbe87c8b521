// The few-row projection kernels of one element type and scale mode.
#include "linear_small.hpp"

namespace skg_host {

SmallKernel small_kernel_bf16(int M, bool gated, int nr, bool exact)
{
    return small_pick<0>(M, gated, nr, exact);
}

}  // namespace skg_host
