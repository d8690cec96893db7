// kd_host.h -- host-side helpers shared by the C entry points (library internal).
#pragma once
#include <cuda_runtime.h>

#include <mutex>

#include "kd.h"

namespace kd {

// Set the calling thread's last-error message (printf form) and return st.
kd_status failf(kd_status st, const char* fmt, ...);

// Set-up made once per device, by the first call there that needs it; its result stands.
class OncePerDevice {
public:
    static constexpr int DEVICES = 64;

private:
    std::once_flag once_[DEVICES];
    cudaError_t err_[DEVICES] = {};

public:
    template <typename F>
    cudaError_t operator()(int dev, F f) {
        if (dev < 0 || dev >= DEVICES) return cudaErrorInvalidDevice;
        std::call_once(once_[dev], [&] { err_[dev] = f(); });
        return err_[dev];
    }
};

// The current device's number of SMs, asked for once per device.
inline cudaError_t current_sms(int* n) {
    static OncePerDevice once;
    static int counts[OncePerDevice::DEVICES];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = once(dev, [dev] { return cudaDeviceGetAttribute(&counts[dev], cudaDevAttrMultiProcessorCount, dev); });
    if (e == cudaSuccess) *n = counts[dev];
    return e;
}

}  // namespace kd

// Return KD_ERR_CUDA (KD_ERR_OOM for a failed allocation) with the call's text if a CUDA call fails.
#define KD_TRY(call)                                                                                       \
    do {                                                                                                   \
        const cudaError_t e_ = (call);                                                                     \
        if (e_ != cudaSuccess)                                                                             \
            return kd::failf(e_ == cudaErrorMemoryAllocation ? KD_ERR_OOM : KD_ERR_CUDA, "%s: %s (%s:%d)", \
                             #call, cudaGetErrorString(e_), __FILE__, __LINE__);                           \
    } while (0)
