// kd_attn_common.cuh -- pieces shared by the split-K attention kernels over
// fp16 KV (kd_attn.cu) and over Q8_0 KV (kd_attn_q8.cu): the work-item table,
// ldmatrix wrappers, the fp16 hi/lo split, bounded polls.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "kd_device.cuh"
#include "kd_kernels.h"
#include "kd_window.h"

namespace kd {

constexpr int AT_C = ATT_CHUNK;  // keys per work item (split)
constexpr int AT_WARPS = 8;      // consumer warps per CTA (two per SM sub-partition)
constexpr int AT_KT = AT_C / 16;  // 16-key tiles (and 16-key steps) of a work item
static_assert(AT_C % 16 == 0 && AT_C <= 64, "a work item is whole 16-key tiles, at most 4");

// Work items are ordered session-major, then split, then KV head.
struct AttnItem {
    int b, s, kvh, n, ns, slot;  // session, split, KV head, keys in this split, splits of the session, its slot
    int start, h0, h1;           // windowed rows: the split's first key, and its hidden keys [h0, h1)
};
// The first key of an item.
template <bool WIN>
__device__ __forceinline__ int item_start(const AttnItem& it) {
    return WIN ? it.start : it.s * AT_C;
}

// The session table of a launch, held one session per lane (B <= 32): the
// session's slot, position, split count and first item.  Built once per warp
// from the step's descriptor; an item's session is then found by a ballot over
// the lanes' first items, with no memory access.
struct AttnTable {
    int slot, pos, ns, base, n_items;
    __device__ __forceinline__ void build(const AttnArgs& a, int lane) {
        slot = lane < a.B ? a.slot[lane] : 0;
        pos = lane < a.B ? a.pos[lane] : 0;
        ns = lane < a.B ? (pos + ATT_CHUNK) / ATT_CHUNK : 0;  // ceil((pos+1)/C)
        int incl = ns * a.nkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL_MASK, incl, o);
            if (lane >= o) incl += v;
        }
        base = incl - ns * a.nkv;
        n_items = __shfl_sync(FULL_MASK, incl, 31);
    }
    // Warp-uniform item index (< n_items); every lane gets the same answer.
    __device__ __forceinline__ AttnItem item(const AttnArgs& a, int lane, int x) const {
        const unsigned m = __ballot_sync(FULL_MASK, lane < a.B && base <= x);
        const int b = 31 - __clz(m);
        AttnItem it;
        it.b = b;
        const int r = x - __shfl_sync(FULL_MASK, base, b);
        it.s = r / a.nkv;
        it.kvh = r - it.s * a.nkv;
        it.n = min(ATT_CHUNK, __shfl_sync(FULL_MASK, pos, b) + 1 - it.s * ATT_CHUNK);
        it.ns = __shfl_sync(FULL_MASK, ns, b);
        it.slot = __shfl_sync(FULL_MASK, slot, b);
        return it;
    }
};

// The same for windowed rows (win_plan): a session's items cover its leading keys,
// then its window.
struct AttnWinTable {
    int slot, pos, base, n_items;
    __device__ __forceinline__ void build(const AttnWinArgs& a, int lane) {
        slot = 0;
        pos = 0;
        if (!a.slot) {  // the rows came with the launch
            base = a.vitems;
            if (lane < a.B) {
                slot = a.vslot[lane];
                pos = a.vpos[lane];
                base = a.vbase[lane];
            }
            n_items = a.vitems;
            return;
        }
        if (lane < a.B) {
            slot = a.slot[lane];
            pos = a.pos[lane];
        }
        const int n = lane < a.B ? win_plan(pos, a.window, a.sinks).ns * a.nkv : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL_MASK, incl, o);
            if (lane >= o) incl += v;
        }
        base = incl - n;
        n_items = __shfl_sync(FULL_MASK, incl, 31);
    }
    __device__ __forceinline__ AttnItem item(const AttnWinArgs& a, int lane, int x) const {
        const unsigned m = __ballot_sync(FULL_MASK, lane < a.B && base <= x);
        const int b = 31 - __clz(m);
        AttnItem it;
        it.b = b;
        const int r = x - __shfl_sync(FULL_MASK, base, b);
        it.s = a.nkv_inv ? (int)__umulhi((unsigned)r, a.nkv_inv) : r;
        it.kvh = r - it.s * a.nkv;
        it.slot = __shfl_sync(FULL_MASK, slot, b);
        const int p = __shfl_sync(FULL_MASK, pos, b);
        const WinPlan w = win_plan(p, a.window, a.sinks);
        it.ns = w.ns;
        if (it.s < w.nsA) {
            it.start = it.s * ATT_CHUNK;
            it.n = min(ATT_CHUNK, a.sinks - it.start);
            it.h0 = it.h1 = 0;
        } else {
            it.start = w.startB + (it.s - w.nsA) * ATT_CHUNK;
            it.n = min(ATT_CHUNK, p + 1 - it.start);
            it.h0 = max(0, a.sinks - it.start);
            it.h1 = min(it.n, w.lo - it.start);
        }
        return it;
    }
};
template <bool WIN>
using AttnTableOf = typename std::conditional<WIN, AttnWinTable, AttnTable>::type;
template <bool WIN>
using AttnArgsOf = typename std::conditional<WIN, AttnWinArgs, AttnArgs>::type;

// A bounded wait ran out: reported at once where the fault word lives across calls;
// a call's own word is set by the merge, from the CTA's marked records.
template <bool WIN>
__device__ __forceinline__ void report_wait(const AttnArgsOf<WIN>& a) {
    if constexpr (WIN) {
        if (a.clear_err) return;
    }
    atomicOr(a.err, ERR_WAIT_TIMEOUT);
}
// Mark the records of all of a CTA's items: their contents are not to be trusted.
__device__ __forceinline__ void mark_records(const AttnWinArgs& a, const AttnWinTable& tab, int lane, int warp, int warps,
                                             int nk, int gq, int hd) {
    for (int k = warp; k < nk; k += warps) {
        const AttnItem it = tab.item(a, lane, (int)blockIdx.x + k * (int)gridDim.x);
        if (lane < gq) {
            float* dst = a.part + (((size_t)it.b * a.nh + (size_t)it.kvh * gq + lane) * a.max_splits + it.s) * ATT_REC(hd);
            *reinterpret_cast<float4*>(dst + hd) = make_float4(0.0f, 1.0f, __int_as_float(REC_FAULT), 0.0f);
        }
    }
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                              uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

// fp32 pair -> fp16 pair (low half = first element), and the fp16 pair of what
// that rounding left over: hi + lo carries about 22 significant bits.
__device__ __forceinline__ uint32_t f2_hi(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t f2_lo(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(__fsub_rn(x, f.x), __fsub_rn(y, f.y));
    return *reinterpret_cast<const uint32_t*>(&l);
}

// Bounded poll of a shared-memory word until it holds v (false: gave up).
__device__ __forceinline__ bool wait_value(const volatile int* p, int v) {
    if (*p == v) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 0; i < WAIT_MAX_POLLS; ++i) {
        if (*p == v) return true;
        if ((i & 255u) == 255u && global_timer_ns() - t0 > WAIT_MAX_NS) break;
    }
    return false;
}

}  // namespace kd
