// The streaming projection kernels on e4m3 with row scales.
#include "linear_stream.hpp"

namespace skg_host {

int stream_kernels_row(int M, bool gated, bool exact, StreamKernel *out)
{
    return stream_pick<1>(M, gated, exact, out);
}

}  // namespace skg_host
