// The streaming projection kernels on bfloat16.
#include "linear_stream.hpp"

namespace skg_host {

int stream_kernels_bf16(int M, bool gated, bool exact, StreamKernel *out)
{
    return stream_pick<0>(M, gated, exact, out);
}

}  // namespace skg_host
