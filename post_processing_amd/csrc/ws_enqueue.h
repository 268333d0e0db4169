// ws_enqueue.h -- how the operators' entry points enqueue their kernels.
// Internal to the library.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ws.h"

namespace ws {

// The device the caller names must exist and be its thread's current one.
inline int device_ready(int32_t device) {
    int ndev = 0;
    if (hipGetDeviceCount(&ndev) != hipSuccess || device >= ndev) return WS_E_NO_DEVICE;
    int cur = -1;
    if (hipGetDevice(&cur) != hipSuccess) return WS_E_HIP;
    return cur == device ? WS_OK : WS_E_INVALID_ARG;
}

// Enqueues one kernel; its parameters are one struct, copied by the call.
template <typename P>
int launch_grid(void (*kernel)(P), dim3 groups, int threads, const P& params, hipStream_t s,
                size_t lds = 0) {
    P copy = params;
    void* args[] = {&copy};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), groups,
                                         dim3((uint32_t)threads), args, lds, s);
    return e == hipSuccess ? WS_OK : WS_E_HIP;
}

template <typename P>
int launch(void (*kernel)(P), int64_t groups, int threads, const P& params, hipStream_t s,
           size_t lds = 0) {
    return launch_grid(kernel, dim3((uint32_t)groups), threads, params, s, lds);
}

}  // namespace ws
