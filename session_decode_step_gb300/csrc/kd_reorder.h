// kd_reorder.h -- launch interface of the cache reorder (library internal).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "kd.h"

namespace kd {

// One plane of a cache: [layers][slots][heads][cap] rows of row_bytes bytes.
struct ReorderPlane {
    void* base;
    int row_bytes;
};
struct ReorderPlan {
    ReorderPlane plane[4];
    int n_planes, layers, slots, heads, cap;
    int window, sinks;  // window 0: every row moves
};

// Slot dst[i] (i < n <= KD_REORDER_MAX, distinct) becomes what slot src[i] held
// before the call in its first len[i] rows (with a window: the rows t of them
// with t < sinks or t > len[i] - window).  All arguments valid.
cudaError_t launch_kv_reorder(const ReorderPlan& p, const int32_t* dst, const int32_t* src, const int32_t* len, int n,
                              cudaStream_t s);

}  // namespace kd
