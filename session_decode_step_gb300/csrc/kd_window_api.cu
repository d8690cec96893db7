// kd_window_api.cu -- the windowed attention's op-level entry points: KV append and
// attention over the leading and the last keys (kd_window.h) in one launch, after
// which a Q8_0 cache needs a merge.
// Slots and positions travel with the launches, so a call copies nothing to the
// device and can be captured into a graph (they are then part of it).
#include <cmath>

#include "kd_host.h"
#include "kd_window.h"

namespace kd {

cudaError_t attn_q8_win_prepare(int dev) {
    static OncePerDevice once;
    return once(dev, [] {
        const cudaError_t e = attn_q8_win_split_attributes();
        return e == cudaSuccess ? attn_win_combine_attributes() : e;
    });
}

static kd_status window_call(const char* fn, bool q8, const float* q, const float* k_new, const float* v_new, void* kc,
                             void* vc, uint16_t* ks, uint16_t* vs, const int32_t* slots, const int32_t* positions,
                             int32_t B, int32_t nh, int32_t nkv, int32_t hd, int32_t n_slots, int32_t cap,
                             int32_t window, int32_t sinks, uint16_t* out, void* ws, size_t ws_bytes, kd_stream stream) {
    if (!q || !k_new || !v_new || !kc || !vc || (q8 && (!ks || !vs)) || !slots || !positions || !out || !ws)
        return failf(KD_ERR_INVALID_ARG, "%s: null argument", fn);
    if (B < 1 || B > KD_MAX_BATCH) return failf(KD_ERR_BATCH, "%s: B=%d outside [1, %d]", fn, B, KD_MAX_BATCH);
    if (nkv < 1 || nh < 1 || nh % nkv || !(q8 ? attn_q8_supported(hd, nh / nkv) : attn_supported(hd, nh / nkv)))
        return failf(KD_ERR_UNSUPPORTED, "%s: head_dim %d, %d query heads, %d KV heads", fn, hd, nh, nkv);
    if (nkv > WIN_MAX_KV_HEADS)
        return failf(KD_ERR_UNSUPPORTED, "%s: %d KV heads (at most %d)", fn, nkv, WIN_MAX_KV_HEADS);
    if (n_slots < 1 || cap < 1 || (q8 && cap % 2)) return failf(KD_ERR_INVALID_ARG, "%s: n_slots %d, cap %d", fn, n_slots, cap);
    if (window < 1 || sinks < 0) return failf(KD_ERR_INVALID_ARG, "%s: window %d, sinks %d", fn, window, sinks);
    if (cap > ATT_MAX_SPLITS * ATT_CHUNK)
        return failf(KD_ERR_UNSUPPORTED, "%s: cap %d exceeds %d", fn, cap, ATT_MAX_SPLITS * ATT_CHUNK);
    if ((int64_t)n_slots * nkv > 0x7fffffff / cap)
        return failf(KD_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 cache rows", fn);
    if (ws_bytes < kd_attn_window_workspace_bytes(B, nh, hd, cap, window, sinks))
        return failf(KD_ERR_INVALID_ARG, "%s: workspace too small", fn);
    const uintptr_t u16 = (uintptr_t)ws | (uintptr_t)kc | (uintptr_t)vc | (uintptr_t)ks | (uintptr_t)vs | (q8 ? (uintptr_t)q : 0);
    if ((u16 & 15) || ((uintptr_t)q & 7))
        return failf(KD_ERR_INVALID_ARG, "%s: caches and workspace must be 16-byte aligned, q %d-byte", fn, q8 ? 16 : 8);
    if ((((uintptr_t)k_new | (uintptr_t)v_new) & 3) || ((uintptr_t)out & 1))
        return failf(KD_ERR_INVALID_ARG, "%s: k_new and v_new must be 4-byte aligned, out 2-byte", fn);
    AttnWinArgs t{};
    int max_keys = 0;
    for (int b = 0; b < B; ++b) {
        if (slots[b] < 0 || slots[b] >= n_slots) return failf(KD_ERR_BAD_SESSION, "%s: slot %d", fn, slots[b]);
        for (int j = 0; j < b; ++j)
            if (slots[j] == slots[b]) return failf(KD_ERR_BAD_SESSION, "%s: slot %d repeated", fn, slots[b]);
        if (positions[b] < 0 || positions[b] >= cap)
            return failf(KD_ERR_POSITION, "%s: position %d outside [0, %d)", fn, positions[b], cap);
        t.vslot[b] = slots[b];
        t.vpos[b] = positions[b];
        const int64_t seen = (int64_t)window + sinks < positions[b] + 1 ? window + sinks : positions[b] + 1;
        if (seen > max_keys) max_keys = (int)seen;
    }
    int dev = 0, sms = 0;
    KD_TRY(cudaGetDevice(&dev));
    KD_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    cudaStream_t s = (cudaStream_t)stream;
    t.q = q;
    t.B = B;
    t.nh = nh;
    t.nkv = nkv;
    t.hd = hd;
    t.cap = cap;
    t.scale = 1.0f / std::sqrt((float)hd);
    t.part = (float*)((char*)ws + 256);
    t.max_splits = win_max_items(cap, window, sinks);
    t.out = (__half*)out;
    t.err = (int*)ws + 2 * KD_MAX_BATCH;  // where kd_attn_device_status looks
    t.ks = (const __half*)ks;
    t.vs = (const __half*)vs;
    t.window = window;
    t.sinks = sinks;
    t.k_new = k_new;
    t.v_new = v_new;
    t.k_dst = kc;
    t.v_dst = vc;
    t.ks_dst = (__half*)ks;
    t.vs_dst = (__half*)vs;
    t.clear_err = 1;
    win_fill(t, true);
    t.kc = (const __half*)kc;
    t.vc = (const __half*)vc;
    if (!q8) {
        KD_TRY(launch_attn_chain(t, max_keys, dev, sms, true, s));
        return KD_OK;
    }
    KD_TRY(attn_q8_win_prepare(dev));
    AttnMaps maps;
    KD_TRY(make_attn_q8_maps((const uint8_t*)kc, (const uint8_t*)vc, (long)n_slots * nkv * cap, &maps));
    // persistent CTAs, no more than there are items
    KD_TRY(launch_attn_split_q8(t, maps, t.vitems < sms ? t.vitems : sms, true, s));
    KD_TRY(launch_attn_combine(t, true, s));
    return KD_OK;
}

}  // namespace kd

extern "C" {

size_t kd_attn_window_workspace_bytes(int32_t B, int32_t n_heads, int32_t head_dim, int32_t cap, int32_t window,
                                      int32_t sinks) {
    if (B < 1 || n_heads < 1 || head_dim < 1 || cap < 1 || window < 1 || sinks < 0) return 0;
    return 256 + (size_t)B * n_heads * kd::win_max_items(cap, window, sinks) * kd::ATT_REC(head_dim) * sizeof(float);
}

kd_status kd_attn_window_append_decode(const float* q, const float* k_new, const float* v_new, uint16_t* k_cache,
                                       uint16_t* v_cache, const int32_t* slots, const int32_t* positions, int32_t B,
                                       int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t n_slots,
                                       int32_t cap, int32_t window, int32_t sinks, uint16_t* out, void* workspace,
                                       size_t workspace_bytes, kd_stream stream) {
    return kd::window_call("kd_attn_window_append_decode", false, q, k_new, v_new, k_cache, v_cache, nullptr, nullptr,
                           slots, positions, B, n_heads, n_kv_heads, head_dim, n_slots, cap, window, sinks, out,
                           workspace, workspace_bytes, stream);
}

kd_status kd_attn_window_append_decode_q8(const float* q, const float* k_new, const float* v_new, uint8_t* k_quants,
                                          uint16_t* k_scales, uint8_t* v_quants, uint16_t* v_scales,
                                          const int32_t* slots, const int32_t* positions, int32_t B, int32_t n_heads,
                                          int32_t n_kv_heads, int32_t n_slots, int32_t cap, int32_t window,
                                          int32_t sinks, uint16_t* out, void* workspace, size_t workspace_bytes,
                                          kd_stream stream) {
    return kd::window_call("kd_attn_window_append_decode_q8", true, q, k_new, v_new, k_quants, v_quants, k_scales,
                           v_scales, slots, positions, B, n_heads, n_kv_heads, 128, n_slots, cap, window, sinks, out,
                           workspace, workspace_bytes, stream);
}

}  // extern "C"
