// The streaming projection kernels on 8-bit integers with row scales.
#include "linear_stream.hpp"

namespace skg_host {

int stream_kernels_int8(int M, bool gated, StreamKernel *out) { return stream_pick<skg::kInt8Row>(M, gated, false, out); }

}  // namespace skg_host
