// kd_window.h -- windowed attention (library internal): a row at position p sees
// the keys t <= p with t < sinks (the first tokens, which stay visible) or
// t > p - window.  The work-item plan, shared by the host and the kernels, and
// the launch interface.
#pragma once
#include <cuda_fp16.h>

#include "kd_kernels.h"

namespace kd {

// The work items of a windowed row at position pos.  Its visible keys are the
// leading [0, min(sinks, lo)) and the window [lo, pos], lo = max(0, pos + 1 -
// window).  Items are ATT_CHUNK keys each: nsA over the leading keys, then the
// window's from startB = lo rounded down to 8 keys (the tails' 8-row boxes and
// the Q8_0 scales' 16-byte copies stay aligned; at most 7 hidden keys are read).
// Where that would be more items than the whole row has (or the leading keys
// reach the window) the items cover [0, pos] and hidden keys are masked: fewer
// than ATT_CHUNK, so no item is hidden as a whole.  A row never has more items
// than without a window, and they depend on its own position only.
struct WinPlan {
    int lo, nsA, startB, ns;
};
__host__ __device__ inline WinPlan win_plan(int pos, int window, int sinks) {
    WinPlan w;
    w.lo = pos + 1 > window ? pos + 1 - window : 0;
    const int lo8 = w.lo & ~7, all = pos / ATT_CHUNK + 1;
    w.nsA = 0;
    w.startB = 0;
    w.ns = all;
    if (lo8 > sinks) {
        const int a = (sinks + ATT_CHUNK - 1) / ATT_CHUNK, b = (pos + 1 - lo8 + ATT_CHUNK - 1) / ATT_CHUNK;
        if (a + b <= all) {
            w.nsA = a;
            w.startB = lo8;
            w.ns = a + b;
        }
    }
    return w;
}
// The most items a row of a slot of cap positions can have.
__host__ __device__ inline int win_max_items(int cap, int window, int sinks) {
    const int a = sinks < cap ? sinks : cap, b = window < cap ? window : cap;
    const int all = (cap + ATT_CHUNK - 1) / ATT_CHUNK;
    const int part = (a + ATT_CHUNK - 1) / ATT_CHUNK + (b + 7 + ATT_CHUNK - 1) / ATT_CHUNK;
    return part < all ? part : all;
}

// slot == nullptr: the rows' slots and positions are in vslot and vpos, passed
// with the launch (nothing has to be staged in device memory first).
constexpr int WIN_MAX_KV_HEADS = 1024;  // a row's items, at most 1024 per head, stay within nkv_inv's range
struct AttnWinArgs : AttnArgs {
    int window, sinks;  // window >= 1, sinks >= 0
    int vslot[16], vpos[16];
    int vbase[16], vitems;  // the rows' first items and the number of items, with vslot
    unsigned nkv_inv;       // ceil(2^32 / nkv): x / nkv = mulhi(x, nkv_inv) for x < 2^32 / nkv
    // Op-level calls: the kernel appends the new rows itself.  The warp whose
    // item ends in row b's new position converts the row (fp32 [B][nkv][hd]),
    // writes it to the cache (fp16 rows, or Q8_0 quants and scales) and into its
    // tile, whose copy may have read the old row.  nullptr: already appended.
    const float *k_new, *v_new;
    void *k_dst, *v_dst;
    __half *ks_dst, *vs_dst;
    // The call's fault word is its own: the first kernel clears it, the Q8_0 split marks the
    // records of a CTA that gave up a wait, and the merge reports them (a word
    // cleared and set by CTAs of one launch would depend on their order).
    int clear_err;
};
// A record's third padding word marks it (0: valid).
constexpr int REC_VALID = 0, REC_FAULT = 1;
// Set what the kernels take from the shape (nkv_inv) and, for op-level calls, the
// items of the B rows at vpos.
inline void win_fill(AttnWinArgs& a, bool rows) {
    a.nkv_inv = (unsigned)((0x100000000ull + (unsigned)a.nkv - 1) / (unsigned)a.nkv);
    if (a.nkv == 1) a.nkv_inv = 0;  // 2^32 does not fit: x itself
    a.vitems = 0;
    for (int b = 0; rows && b < a.B; ++b) {
        a.vbase[b] = a.vitems;
        a.vitems += win_plan(a.vpos[b], a.window, a.sinks).ns * a.nkv;
    }
}
// Set up the windowed Q8_0 kernels on device dev, the current one, before their first launch there.
cudaError_t attn_q8_win_prepare(int dev);
cudaError_t attn_q8_win_split_attributes();  // its parts
cudaError_t attn_win_combine_attributes();
cudaError_t launch_attn_split_q8(const AttnWinArgs& a, const AttnMaps& maps, int grid, bool pdl, cudaStream_t s);
cudaError_t launch_attn_combine(const AttnWinArgs& a, bool pdl, cudaStream_t s);
// fp16 rows, in one launch (kd_attn_chain.cu).  From WIN_CHAIN_ITEMS items of a row's
// capacity on, the keys are shared out wider.
constexpr int WIN_CHAIN_ITEMS = 32;
// Set up the kernels of a shape on device dev, the current one (a launch does so for its own).
cudaError_t attn_chain_prepare(int hd, int group, int max_splits, int dev);
// max_keys: no row sees more.  dev: the current device, num_sms its SMs.
cudaError_t launch_attn_chain(const AttnWinArgs& a, int max_keys, int dev, int num_sms, bool pdl, cudaStream_t s);
}  // namespace kd
