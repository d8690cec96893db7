// kd_paged_append.cu -- new keys (rotated on the way) and values into the pages of fp16 or
// Q8_0 caches, and the queries rotated alongside, in one launch.
//
// A lane owns 4 dims of a head, so a warp takes a head of 128 (two of 64) of one token:
// K heads, V heads, then query heads, four of them in flight.  The lane's angles are
// formed once per warp; the other half of a pair is a neighbour's register (a shuffle), or
// for rotated parts that do not split into lanes an element of the input again.  A row's
// place comes from the page table by one look-up per warp.
// Q8_0 rows: the 8 lanes of a 32-value block find its maximum by shuffles and store 4 codes
// each.  There k is rounded to fp32 exactly once (kd_rope.cuh) before the division, so that
// a code never depends on how the rotation was summed.
//
// Few tokens are bound by a launch and two dependent loads (a position's page, then the
// row); many by memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kd_host.h"
#include "kd_rope.cuh"
#include "kd_rope.h"

namespace kd {

struct AppendArgs {
    const void *k, *v, *q;
    int64_t k_ld, v_ld, q_ld;
    void *kp, *vp;      // pages: fp16 rows, or quants
    __half *ks, *vs;    // scales (Q8_0)
    float* q_out;
    const int* table;
    int* fault;
    int table_ld, n_seqs, tokens, nh, nkv, n_pages, ps;
    int per, groups;    // heads of one warp, warps of a token
    int vec;            // every input head starts on a multiple of 4 elements
    int rotate;
    RopeAngles<64> r;
    int start[KD_PAGED_MAX_SEQS], first[KD_PAGED_MAX_SEQS + 1];  // a session's first new position; its first new row
};

template <typename T>
struct alignas(sizeof(T) * 4) Four {
    T v[4];
};
__device__ __forceinline__ float in_f(float x) { return x; }
__device__ __forceinline__ float in_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float in_f(__nv_bfloat16 x) { return __bfloat162float(x); }

constexpr int APPEND_WARPS = 8;

template <typename T, bool Q8, int HD>
__global__ void __launch_bounds__(APPEND_WARPS * 32) paged_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int LANES = HD / 4, ROWS = 32 / LANES;  // lanes of a head, heads at a time
    constexpr int U = 4;                              // of them in flight
    __shared__ float2 tab[ROPE_TAB];
    __shared__ unsigned long long turns[64];
    if (threadIdx.x < ROPE_TAB) tab[threadIdx.x] = ROPE_COS[threadIdx.x];
    if (threadIdx.x >= 128 && threadIdx.x < 192) turns[threadIdx.x - 128] = a.r.turns[threadIdx.x - 128];
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = (int64_t)blockIdx.x * APPEND_WARPS + warp;
    const int token = (int)(unit / a.groups);
    if (token >= a.tokens) return;
    const int heads = 2 * a.nkv + a.nh;
    const int h0 = (int)(unit - (int64_t)token * a.groups) * a.per, h1 = min(heads, h0 + a.per);
    // the token's session, its position and the row that it goes to
    int lo = 0, hi = a.n_seqs;  // first[lo] <= token < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.first[mid] <= token) lo = mid;
        else hi = mid;
    }
    const int pos = a.start[lo] + (token - a.first[lo]);
    const int in_table = pos / a.ps, in_page = pos - in_table * a.ps;
    int page = -1;
    if (h0 < 2 * a.nkv) {
        page = a.table[(int64_t)lo * a.table_ld + in_table];
        if ((unsigned)page >= (unsigned)a.n_pages) {
            if (a.fault && lane == 0) *a.fault = 1;
            page = -1;
        }
    }
    const int sub = lane / LANES, d = lane % LANES * 4;  // the head of the warp's, and the lane's dims d .. d + 3

    float4 x[U], y[U];  // the lane's values, and their partners where no lane has them
    const int half = a.r.rot / 2;
    const bool turned = a.rotate && d < a.r.rot;
    const bool shuffles = half % 4 == 0;
    const int partner = lane + (a.r.pairs ? 0 : d < half ? half / 4 : -(half / 4));
    auto source = [&](int h) -> const T* {
        if (h < a.nkv) return (const T*)a.k + token * a.k_ld + (int64_t)h * HD;
        if (h < 2 * a.nkv) return (const T*)a.v + token * a.v_ld + (int64_t)(h - a.nkv) * HD;
        return (const T*)a.q + token * a.q_ld + (int64_t)(h - 2 * a.nkv) * HD;
    };
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int hh = h + i * ROWS + sub;
            if (hh >= h1) continue;
            const T* p = source(hh);
            if (a.vec) {
                const Four<T> f = *reinterpret_cast<const Four<T>*>(p + d);
                x[i] = make_float4(in_f(f.v[0]), in_f(f.v[1]), in_f(f.v[2]), in_f(f.v[3]));
            } else {
                x[i] = make_float4(in_f(p[d]), in_f(p[d + 1]), in_f(p[d + 2]), in_f(p[d + 3]));
            }
            if (turned && !a.r.pairs && !shuffles) {
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = d + e < a.r.rot ? in_f(p[d + e < half ? d + e + half : d + e - half]) : 0.0f;
                y[i] = make_float4(o[0], o[1], o[2], o[3]);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < U; ++i) x[i] = y[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    load(h0);
    float2 c[4], s[4];
    if (turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int pair = a.r.pairs ? (d + e) >> 1 : d + e < half ? d + e : d + e - half;
            if (a.r.pairs && (e & 1)) {
                c[e] = c[e - 1];
                s[e] = s[e - 1];
            } else {
                rope_angle<true>(turns[min(pair, 63)], pos, a.r.mh, a.r.ml, tab, c[e], s[e]);
            }
        }
    }
    for (int h = h0; h < h1; h += U * ROWS) {
        float4 out[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float4 o = y[i];
            if (!a.r.pairs && shuffles) {
                o.x = __shfl_sync(FULL_MASK, x[i].x, partner);
                o.y = __shfl_sync(FULL_MASK, x[i].y, partner);
                o.z = __shfl_sync(FULL_MASK, x[i].z, partner);
                o.w = __shfl_sync(FULL_MASK, x[i].w, partner);
            } else if (a.r.pairs) {
                o = make_float4(x[i].y, x[i].x, x[i].w, x[i].z);
            }
            const int hh = h + i * ROWS + sub;
            const bool value = hh >= a.nkv && hh < 2 * a.nkv;
            out[i] = x[i];
            if (turned && !value) {
                const float in[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, other[4] = {o.x, o.y, o.z, o.w};
                float r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float sign = (a.r.pairs ? (e & 1) != 0 : d + e >= half) ? 1.0f : -1.0f;
                    r[e] = d + e < a.r.rot ? rope_turn<true>(in[e], other[e], c[e], s[e], sign) : in[e];
                }
                out[i] = make_float4(r[0], r[1], r[2], r[3]);
            }
        }
        const int now = h;
        if (h + U * ROWS < h1) load(h + U * ROWS);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int hh = now + i * ROWS + sub;
            const float4 o = out[i];
            uint32_t code = 0;
            __half scale{};
            if constexpr (Q8) {  // as q8_quant: 8 lanes hold a block
                float m = fmaxf(fmaxf(fabsf(o.x), fabsf(o.y)), fmaxf(fabsf(o.z), fabsf(o.w)));
#pragma unroll
                for (int b = 1; b < 8; b <<= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, b));
                const float dd = __fdiv_rn(m, 127.0f);
                scale = __float2half_rn(dd);
                auto quant = [&](float v) -> uint32_t {
                    return (uint32_t)((dd > 0.0f ? max(-127, min(127, (int)roundf(__fdiv_rn(v, dd)))) : 0) + 128);
                };
                code = quant(o.x) | quant(o.y) << 8 | quant(o.z) << 16 | quant(o.w) << 24;
            }
            if (hh >= h1) continue;
            if (hh >= 2 * a.nkv) {
                *reinterpret_cast<float4*>(a.q_out + ((int64_t)token * a.nh + hh - 2 * a.nkv) * HD + d) = o;
            } else if (page >= 0) {
                const bool value = hh >= a.nkv;
                const int64_t row = ((int64_t)page * a.nkv + (value ? hh - a.nkv : hh)) * a.ps + in_page;
                if constexpr (Q8) {
                    reinterpret_cast<uint32_t*>(value ? a.vp : a.kp)[row * (HD / 4) + lane] = code;
                    if ((lane & 7) == 0) (value ? a.vs : a.ks)[row * (HD / 32) + (lane >> 3)] = scale;
                } else {
                    const __half2 w0 = __floats2half2_rn(o.x, o.y), w1 = __floats2half2_rn(o.z, o.w);
                    *reinterpret_cast<uint2*>((__half*)(value ? a.vp : a.kp) + row * HD + d) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&w0), *reinterpret_cast<const uint32_t*>(&w1));
                }
            }
        }
    }
}

template <typename T>
static cudaError_t launch_append(AppendArgs& a, bool q8, int hd, cudaStream_t s) {
    auto fours = [&](const void* p, int64_t ld) { return ((uintptr_t)p & (4 * sizeof(T) - 1)) == 0 && ld % 4 == 0; };
    a.vec = fours(a.k, a.k_ld) && fours(a.v, a.v_ld) && (!a.nh || fours(a.q, a.q_ld));
    // Heads of a warp: as many as leave every SM some forty warps (the angles are formed once for them).
    const int heads = 2 * a.nkv + a.nh;
    int64_t per = (int64_t)a.tokens * heads / (152 * 48);
    per = per < 4 ? 4 : per > heads ? heads : (per + 3) / 4 * 4;
    a.per = (int)per;
    a.groups = (heads + a.per - 1) / a.per;
    const int64_t units = (int64_t)a.tokens * a.groups;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)((units + APPEND_WARPS - 1) / APPEND_WARPS));
    cfg.blockDim = dim3(APPEND_WARPS * 32);
    cfg.stream = s;
    if (q8) return cudaLaunchKernelEx(&cfg, paged_append_kernel<T, true, 128>, a);
    return hd == 64 ? cudaLaunchKernelEx(&cfg, paged_append_kernel<T, false, 64>, a)
                    : cudaLaunchKernelEx(&cfg, paged_append_kernel<T, false, 128>, a);
}

static kd_status append_call(const char* fn, bool q8, const kd_rope_table* rope, const void* k, int64_t k_ld, const void* v,
                             int64_t v_ld, const void* q, int64_t q_ld, int32_t dtype, void* kp, uint16_t* ks, void* vp,
                             uint16_t* vs, const int32_t* table, int32_t table_ld, const int32_t* starts,
                             const int32_t* counts, int32_t n_seqs, int32_t nh, int32_t nkv, int32_t hd, int32_t n_pages,
                             int32_t ps, float* q_out, int32_t* fault, kd_stream stream) {
    if (!k || !v || !kp || !vp || (q8 && (!ks || !vs)) || !table || !starts || !counts || (nh > 0 && (!q || !q_out)))
        return failf(KD_ERR_INVALID_ARG, "%s: null argument", fn);
    if (n_seqs < 1 || n_seqs > KD_PAGED_MAX_SEQS)
        return failf(KD_ERR_BATCH, "%s: n_seqs=%d outside [1, %d]", fn, n_seqs, KD_PAGED_MAX_SEQS);
    if (hd != 128 && (q8 || hd != 64)) return failf(KD_ERR_UNSUPPORTED, "%s: head_dim %d", fn, hd);
    if (ps < 16 || ps % 16 || ps > 65536) return failf(KD_ERR_UNSUPPORTED, "%s: page_size %d", fn, ps);
    if (dtype < KD_F32 || dtype > KD_BF16) return failf(KD_ERR_INVALID_ARG, "%s: dtype %d", fn, dtype);
    if (nkv < 1 || nh < 0 || n_pages < 1 || table_ld < 1)
        return failf(KD_ERR_INVALID_ARG, "%s: %d KV heads, %d query heads, n_pages %d, table_ld %d", fn, nkv, nh, n_pages, table_ld);
    if ((int64_t)nkv * 2 + nh > 0xffffff) return failf(KD_ERR_UNSUPPORTED, "%s: %d KV heads, %d query heads", fn, nkv, nh);
    if ((!nh && (q || q_out))) return failf(KD_ERR_INVALID_ARG, "%s: queries without n_heads", fn);
    if (rope) {
        const kd_status st = rope_table_check(fn, rope);
        if (st != KD_OK) return st;
        if (rope->head_dim != hd)
            return failf(KD_ERR_INVALID_ARG, "%s: a rotation of heads of %d for head_dim %d", fn, rope->head_dim, hd);
    }
    const uintptr_t mask = dtype == KD_F32 ? 3 : 1;
    if ((((uintptr_t)kp | (uintptr_t)vp | (uintptr_t)ks | (uintptr_t)vs | (uintptr_t)q_out) & 15) ||
        (((uintptr_t)k | (uintptr_t)v | (uintptr_t)q) & mask) || (((uintptr_t)table | (uintptr_t)fault) & 3))
        return failf(KD_ERR_INVALID_ARG, "%s: misaligned pointer (pages and q_out 16-byte)", fn);
    AppendArgs a = {};
    int64_t total = 0;
    for (int b = 0; b < n_seqs; ++b) {
        if (starts[b] < 0 || counts[b] < 0 || (int64_t)starts[b] + counts[b] > (int64_t)table_ld * ps)
            return failf(KD_ERR_POSITION, "%s: %d rows from position %d on in tables of %d pages of %d", fn, counts[b],
                         starts[b], table_ld, ps);
        a.start[b] = starts[b];
        a.first[b] = (int)total;
        total += counts[b];
        if (total * (2 * (int64_t)nkv + nh) > 0x7fffffff)
            return failf(KD_ERR_UNSUPPORTED, "%s: 2^31 or more new heads", fn);
    }
    a.first[n_seqs] = (int)total;
    if (k_ld < (int64_t)nkv * hd || v_ld < (int64_t)nkv * hd || (nh && q_ld < (int64_t)nh * hd) ||
        k_ld > INT64_MAX / 4 / (total + 1) || v_ld > INT64_MAX / 4 / (total + 1) || (nh && q_ld > INT64_MAX / 4 / (total + 1)))
        return failf(KD_ERR_INVALID_ARG, "%s: k_ld %lld, v_ld %lld, q_ld %lld", fn, (long long)k_ld, (long long)v_ld, (long long)q_ld);
    if (!total) return KD_OK;
    a.k = k;
    a.v = v;
    a.q = q;
    a.k_ld = k_ld;
    a.v_ld = v_ld;
    a.q_ld = q_ld;
    a.kp = kp;
    a.vp = vp;
    a.ks = (__half*)ks;
    a.vs = (__half*)vs;
    a.q_out = q_out;
    a.table = table;
    a.fault = fault;
    a.table_ld = table_ld;
    a.n_seqs = n_seqs;
    a.tokens = (int)total;
    a.nh = nh;
    a.nkv = nkv;
    a.n_pages = n_pages;
    a.ps = ps;
    a.rotate = rope != nullptr;
    if (rope) rope_fill(a.r, *rope);
    cudaStream_t s = (cudaStream_t)stream;
    switch (dtype) {
        case KD_F32: KD_TRY(launch_append<float>(a, q8, hd, s)); break;
        case KD_F16: KD_TRY(launch_append<__half>(a, q8, hd, s)); break;
        default: KD_TRY(launch_append<__nv_bfloat16>(a, q8, hd, s));
    }
    return KD_OK;
}

}  // namespace kd

extern "C" {

kd_status kd_paged_append(const kd_rope_table* rope, const void* k_new, int64_t k_ld, const void* v_new, int64_t v_ld,
                          const void* q, int64_t q_ld, int32_t dtype, uint16_t* k_pages, uint16_t* v_pages,
                          const int32_t* table, int32_t table_ld, const int32_t* starts, const int32_t* counts,
                          int32_t n_seqs, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t n_pages,
                          int32_t page_size, float* q_out, int32_t* fault, kd_stream stream) {
    return kd::append_call("kd_paged_append", false, rope, k_new, k_ld, v_new, v_ld, q, q_ld, dtype, k_pages, nullptr, v_pages,
                           nullptr, table, table_ld, starts, counts, n_seqs, n_heads, n_kv_heads, head_dim, n_pages,
                           page_size, q_out, fault, stream);
}

kd_status kd_paged_append_q8(const kd_rope_table* rope, const void* k_new, int64_t k_ld, const void* v_new, int64_t v_ld,
                             const void* q, int64_t q_ld, int32_t dtype, uint8_t* k_quants, uint16_t* k_scales,
                             uint8_t* v_quants, uint16_t* v_scales, const int32_t* table, int32_t table_ld,
                             const int32_t* starts, const int32_t* counts, int32_t n_seqs, int32_t n_heads,
                             int32_t n_kv_heads, int32_t n_pages, int32_t page_size, float* q_out, int32_t* fault,
                             kd_stream stream) {
    return kd::append_call("kd_paged_append_q8", true, rope, k_new, k_ld, v_new, v_ld, q, q_ld, dtype, k_quants, k_scales,
                           v_quants, v_scales, table, table_ld, starts, counts, n_seqs, n_heads, n_kv_heads, 128, n_pages,
                           page_size, q_out, fault, stream);
}

}  // extern "C"
