// kd_host.h -- host-side helpers shared by the C entry points (library internal).
#pragma once
#include <cuda_runtime.h>

#include "kd.h"

namespace kd {

// Set the calling thread's last-error message (printf form) and return st.
kd_status failf(kd_status st, const char* fmt, ...);

cudaError_t beam_init_attributes();

}  // namespace kd

// Return KD_ERR_CUDA (KD_ERR_OOM for a failed allocation) with the call's text if a CUDA call fails.
#define KD_TRY(call)                                                                                       \
    do {                                                                                                   \
        const cudaError_t e_ = (call);                                                                     \
        if (e_ != cudaSuccess)                                                                             \
            return kd::failf(e_ == cudaErrorMemoryAllocation ? KD_ERR_OOM : KD_ERR_CUDA, "%s: %s (%s:%d)", \
                             #call, cudaGetErrorString(e_), __FILE__, __LINE__);                           \
    } while (0)
