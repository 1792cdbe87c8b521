// What the launchers of include/skinny_ops.h share: the device check and the launch.
#pragma once

#include <hip/hip_runtime.h>

#include "skinny_ops.h"

namespace skg_host {

// SKINNY_OK where the current device is a gfx950; *cus: its compute units.
int ops_device(int *cus);

// Launch, and on failure clear the runtime's last error so that a refusal is reported
// once, here, and not again by the caller's next HIP call.
inline int ops_launch(const void *fn, dim3 grid, int block, void **args, hipStream_t s)
{
    if (hipLaunchKernel(fn, grid, dim3((unsigned)block), args, 0, s) == hipSuccess)
        return SKINNY_OK;
    (void)hipGetLastError();
    return SKINNY_ERR_LAUNCH;
}

}  // namespace skg_host
