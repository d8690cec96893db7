// kd_paged_append.cu -- new keys (rotated on the way) and values into the pages of fp16 or
// Q8_0 caches, and the queries rotated alongside, in one launch.
//
// A lane owns 4 dims of a head, so a warp takes a head of 128 (two of 64) of one token:
// K heads, V heads, then query heads, four of them in flight.  The token's angles are
// formed once per warp, one or two by a lane; the other half of a pair is a neighbour's register (a shuffle), or
// for rotated parts that do not split into lanes an element of the input again.  A row's
// place comes from the page table by one look-up per warp.
// Q8_0 rows: the 8 lanes of a 32-value block find its maximum by shuffles and store 4 codes
// each.  There k is rounded to fp32 exactly once (kd_rope.cuh) before the division, so that
// a code never depends on how the rotation was summed.  (Keys below 2^-120 aside: what their products' roundings leave out is
// less than fp32 holds.  Their scales are 0.)
//
// Few tokens are bound by a launch and two dependent loads (a position's page, then the
// row): 8 tokens of 32 + 8 heads take 2.3 us, an empty launch 2.1.  Many are bound by issue, near
// memory's rate: 8.8 k bf16 tokens of 32 + 8 heads of 128 (277 MB) 49 us, 5.6 TB/s; with K, V and queries
// in one loop, a head's kind asked for each time, 64; with blocks that stay and take the next token, 62 (the last ones are
// waited for).  6.3 k tokens of 8 heads into Q8_0 21.4 us, 23 with inputs that are not in L2 (floor 5.9): the exact rotation, three shuffles a maximum and the codes;
// with each lane forming its own four angles, twice each in a warp, 24.7 and 2.7 for the 8 tokens.
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
    int rotate;
    RopeAngles<64> r;
    int start[KD_PAGED_MAX_SEQS], first[KD_PAGED_MAX_SEQS + 1];  // a session's first new position; its first new row
};

template <typename T>
struct alignas(sizeof(T) * 4) Four {
    T v[4];
};
// Four codes q + 128, q = x / d in fp32 rounded half away from zero, within [-127, 127]; 0 for d = 0.
// |x| <= 127 d but for a rounding.  x times the reciprocal of d is within 127 2^-22 = 3e-5 of the
// rounded quotient, so where it lies farther than 6e-5 from the middle between two whole numbers
// the nearest one is the quotient's, too; there, or for a d without a finite reciprocal, the
// division decides (a thousandth of the warps; 6340 rows of 16 heads take 32.5 us, 37.1 with a division each).
__device__ __forceinline__ uint32_t q8_codes(const float (&x)[4], float d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    const float2 rr = make_float2(r, r), big = make_float2(12582912.0f, 12582912.0f), back = make_float2(-12582912.0f, -12582912.0f);
    const float2 y0 = f2_mul(make_float2(x[0], x[1]), rr), y1 = f2_mul(make_float2(x[2], x[3]), rr);
    const float2 z0 = f2_add(y0, big), z1 = f2_add(y1, big);  // 1.5 2^23 + the nearest whole number: its low byte is there
    const float2 minus = make_float2(-1.0f, -1.0f);
    const float2 o0 = f2_fma(f2_add(z0, back), minus, y0), o1 = f2_fma(f2_add(z1, back), minus, y1);
    const float off = fmaxf(fmaxf(fabsf(o0.x), fabsf(o0.y)), fmaxf(fabsf(o1.x), fabsf(o1.y)));
    const float sum = __fadd_rn(__fadd_rn(o0.x, o0.y), __fadd_rn(o1.x, o1.y));  // NaN where one is
    if (off < 0.49994f && sum == sum)
        return __byte_perm(__byte_perm(__float_as_uint(z0.x), __float_as_uint(z0.y), 0x0040),
                           __byte_perm(__float_as_uint(z1.x), __float_as_uint(z1.y), 0x0040), 0x5410) ^ 0x80808080u;
    uint32_t code = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int q = d > 0.0f ? max(-127, min(127, (int)roundf(__fdiv_rn(x[e], d)))) : 0;
        code |= (uint32_t)(q + 128) << (8 * e);
    }
    return code;
}

// Small blocks: a new one takes a finished one's place sooner (8 tokens 2.3 us, 2.5 with 8 warps; Q8_0 rows 21.7, 23.2).
constexpr int APPEND_WARPS = 4;
constexpr int APPEND_PER_SM = 7;  // 72 registers a thread: long prompts 48.4 us, 51.1 with 6 blocks, 51.5 with 8
// Heads in flight per lane group: 16 registers of them (long prompts 48.4 us, 50.2 with 8); Q8_0, which needs more for its codes, 8
// (21.4 us, 22.5 with 16).
template <typename T, bool Q8>
__host__ __device__ constexpr int append_flight() {
    return (Q8 ? 8 : 16) / (int)sizeof(T);
}

// VEC: every input head starts on a multiple of 4 elements.
template <typename T, bool Q8, int HD, bool VEC>
__global__ void __launch_bounds__(APPEND_WARPS * 32, APPEND_PER_SM) paged_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int LANES = HD / 4, ROWS = 32 / LANES;  // lanes of a head, heads at a time
    constexpr int U = append_flight<T, Q8>();         // of them in flight
    __shared__ float2 tab[ROPE_TAB];
    __shared__ unsigned long long turns[64];
    __shared__ float4 angles[APPEND_WARPS][4 * 18];  // of the warp's token: pair p at [p % 4][p / 4], 18 apart, so in different banks
    static_assert(APPEND_WARPS * 32 >= ROPE_TAB && APPEND_WARPS * 32 >= 64, "a thread an entry");
    if (threadIdx.x < ROPE_TAB) tab[threadIdx.x] = ROPE_COS[threadIdx.x];
    if (threadIdx.x < 64) turns[threadIdx.x] = a.r.turns[threadIdx.x];
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = 2 * a.nkv + a.nh;
    const int sub = lane / LANES, d = lane % LANES * 4;  // the head of the warp's, and the lane's dims d .. d + 3
    const int half = a.r.rot / 2;
    const bool turned = a.rotate && d < a.r.rot;
    const bool shuffles = half % 4 == 0;
    const int partner = lane + (a.r.pairs ? 0 : d < half ? half / 4 : -(half / 4));
    const int unit = blockIdx.x * APPEND_WARPS + warp;
    const int token = unit / a.groups;
    if (token >= a.tokens) return;
    const int h0 = (unit - token * a.groups) * a.per, h1 = min(heads, h0 + a.per);
    // The warp's heads: [k0, k1) of K, [v0, v1) of V, [q0, q1) of the queries.
    const int k0 = min(h0, a.nkv), k1 = min(h1, a.nkv);
    const int v0 = min(max(h0 - a.nkv, 0), a.nkv), v1 = min(max(h1 - a.nkv, 0), a.nkv);
    const int q0 = max(h0 - 2 * a.nkv, 0), q1 = max(h1 - 2 * a.nkv, 0);
    const T* ksrc = (const T*)a.k + token * a.k_ld + (k0 + sub) * HD;
    const T* vsrc = (const T*)a.v + token * a.v_ld + (v0 + sub) * HD;
    const T* qsrc = (const T*)a.q + token * a.q_ld + (int64_t)(q0 + sub) * HD;
    Four<T> raw[U];
    // U flights of heads, `left` of them there
    auto load = [&](const T* src, int left) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i * ROWS + sub < left) {
                const T* p = src + i * ROWS * HD + d;
                if constexpr (VEC) {
                    raw[i] = *reinterpret_cast<const Four<T>*>(p);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) raw[i].v[e] = p[e];
                }
            }
    };
    // the first flight before the angles
    if (k0 < k1) load(ksrc, k1 - k0);
    else if (v0 < v1) load(vsrc, v1 - v0);
    else load(qsrc, q1 - q0);
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
    if (h0 < 2 * a.nkv) page = a.table[(int64_t)lo * a.table_ld + in_table];

    float ch[4], cl[4], sh[4], sl[4];  // the sines with the sign that they are added with
    if (a.rotate && (k0 < k1 || q0 < q1)) {
        // each pair's angle by one lane, then to those that hold its dims
        for (int p = lane; p < half; p += 32) {
            float2 c, s;
            rope_angle<true>(turns[p], pos, a.r.mh, a.r.ml, tab, c, s);
            angles[warp][(p & 3) * 18 + (p >> 2)] = make_float4(c.x, c.y, s.x, s.y);
        }
        __syncwarp();
        if (turned) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int pair = min(a.r.pairs ? (d + e) >> 1 : d + e < half ? d + e : d + e - half, half - 1);
                const float4 v = angles[warp][(pair & 3) * 18 + (pair >> 2)];
                const bool plus = a.r.pairs ? (e & 1) != 0 : d + e >= half;
                ch[e] = v.x, cl[e] = v.y, sh[e] = plus ? v.z : -v.z, sl[e] = plus ? v.w : -v.w;
            }
        }
    }
    if ((unsigned)page >= (unsigned)a.n_pages) {
        if (a.fault && h0 < 2 * a.nkv && lane == 0) *a.fault = 1;
        page = -1;
    }
    // The lane's values of flight i in fp32, rotated.
    auto values = [&](int i, const T* src, bool have, bool rotates, float (&x)[4]) {
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = to_f(raw[i].v[e]);
        if (!rotates || !a.rotate) return;
        if (a.r.pairs) {
            o[0] = x[1], o[1] = x[0], o[2] = x[3], o[3] = x[2];
        } else if (shuffles) {
            if constexpr (sizeof(T) == 2) {
                const uint2 w = *reinterpret_cast<const uint2*>(&raw[i]);
                uint2 r;
                r.x = __shfl_sync(FULL_MASK, w.x, partner);
                r.y = __shfl_sync(FULL_MASK, w.y, partner);
                const Four<T> f = *reinterpret_cast<const Four<T>*>(&r);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = to_f(f.v[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = __shfl_sync(FULL_MASK, x[e], partner);
            }
        } else {
            const T* p = src + i * ROWS * HD;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = have && d + e < a.r.rot ? to_f(p[d + e < half ? d + e + half : d + e - half]) : 0.0f;
        }
        if (turned) {
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float2 r = rope_turn2<true>(make_float2(x[e], x[e + 1]), make_float2(o[e], o[e + 1]),
                                                  make_float2(ch[e], ch[e + 1]), make_float2(cl[e], cl[e + 1]),
                                                  make_float2(sh[e], sh[e + 1]), make_float2(sl[e], sl[e + 1]),
                                                  make_float2(-ch[e], -ch[e + 1]), make_float2(-sh[e], -sh[e + 1]));
                x[e] = r.x;  // rot is even, but the last lane may have two dims of it only
                x[e + 1] = r.y;
                if (d + e + 2 >= a.r.rot) break;
            }
        }
    };
    // Rows of K or V from head `first` on, `left` of them.
    auto rows = [&](const T* src, bool loaded, bool rotates, int first, int left, void* dst, __half* scales) {
        int64_t row = ((int64_t)page * a.nkv + first + sub) * a.ps + in_page;
        for (; left > 0; left -= U * ROWS, src += U * ROWS * HD, row += (int64_t)U * ROWS * a.ps) {
            if (!loaded) load(src, left);
            loaded = false;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (i * ROWS >= left) break;
                const bool have = i * ROWS + sub < left;
                const int64_t at = row + (int64_t)i * ROWS * a.ps;
                float x[4];
                values(i, src, have, rotates, x);
                if constexpr (Q8) {  // as q8_quant: 8 lanes hold a block
                    float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
                    for (int b = 1; b < 8; b <<= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, b));
                    const float dd = __fdiv_rn(m, 127.0f);
                    const uint32_t code = q8_codes(x, dd);
                    if (page >= 0) {
                        reinterpret_cast<uint32_t*>(dst)[at * (HD / 4) + lane] = code;
                        if ((lane & 7) == 0) scales[at * (HD / 32) + (lane >> 3)] = __float2half_rn(dd);
                    }
                } else if (have && page >= 0) {
                    const __half2 w0 = __floats2half2_rn(x[0], x[1]), w1 = __floats2half2_rn(x[2], x[3]);
                    *reinterpret_cast<uint2*>((__half*)dst + at * HD + d) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&w0), *reinterpret_cast<const uint32_t*>(&w1));
                }
            }
        }
    };
    rows(ksrc, true, true, k0, k1 - k0, a.kp, a.ks);
    rows(vsrc, k0 >= k1, false, v0, v1 - v0, a.vp, a.vs);
    bool loaded = k0 >= k1 && v0 >= v1;
    float* out = a.q_out + ((int64_t)token * a.nh + q0 + sub) * HD + d;
    for (int left = q1 - q0; left > 0; left -= U * ROWS, qsrc += U * ROWS * HD, out += U * ROWS * HD) {
        if (!loaded) load(qsrc, left);
        loaded = false;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i * ROWS >= left) break;
            const bool have = i * ROWS + sub < left;
            float x[4];
            values(i, qsrc, have, true, x);
            if (have) *reinterpret_cast<float4*>(out + i * ROWS * HD) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
}

template <typename T>
static cudaError_t launch_append(AppendArgs& a, bool q8, int hd, cudaStream_t s) {
    auto fours = [&](const void* p, int64_t ld) { return ((uintptr_t)p & (4 * sizeof(T) - 1)) == 0 && ld % 4 == 0; };
    const bool vec = fours(a.k, a.k_ld) && fours(a.v, a.v_ld) && (!a.nh || fours(a.q, a.q_ld));
    // Heads of a warp: as many as leave every SM some forty warps (the angles are formed once for
    // them), whole flights where it has several.
    const int U = q8 ? append_flight<T, true>() : append_flight<T, false>();
    const int heads = 2 * a.nkv + a.nh, rows = hd == 64 ? 2 : 1;
    int sms = 0;
    const cudaError_t e = current_sms(&sms);
    if (e != cudaSuccess) return e;
    int64_t per = (int64_t)a.tokens * heads / (sms * 40);
    per = per < rows ? rows : per < U * rows ? per / rows * rows : per / (U * rows) * (U * rows);
    a.per = (int)(per < heads ? per : heads);
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
#define KD_APPEND(VEC_)                                                                                                       \
    return q8 ? cudaLaunchKernelEx(&cfg, paged_append_kernel<T, true, 128, VEC_>, a)                                          \
              : hd == 64 ? cudaLaunchKernelEx(&cfg, paged_append_kernel<T, false, 64, VEC_>, a)                               \
                         : cudaLaunchKernelEx(&cfg, paged_append_kernel<T, false, 128, VEC_>, a)
    if (vec) KD_APPEND(true);
    KD_APPEND(false);
#undef KD_APPEND
}

static kd_status append_call(const char* fn, bool q8, const kd_rope_table* rope, const void* k, int64_t k_ld, const void* v,
                             int64_t v_ld, const void* q, int64_t q_ld, int32_t dtype, void* kp, uint16_t* ks, void* vp,
                             uint16_t* vs, const int32_t* table, int32_t table_ld, const int32_t* starts,
                             const int32_t* counts, int32_t n_seqs, int32_t nh, int32_t nkv, int32_t hd, int32_t n_pages,
                             int32_t ps, float* q_out, int32_t* fault, kd_stream stream) {
    if (!kp || !vp || (q8 && (!ks || !vs)) || !table || !starts || !counts)
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
        if (starts[b] < 0 || counts[b] < 0 || (int64_t)starts[b] + counts[b] > (int64_t)table_ld * ps ||
            (int64_t)starts[b] + counts[b] > 0x7fffffff)
            return failf(KD_ERR_POSITION, "%s: %d rows from position %d on in tables of %d pages of %d", fn, counts[b],
                         starts[b], table_ld, ps);
        a.start[b] = starts[b];
        a.first[b] = (int)total;
        total += counts[b];
        if (total * (2 * (int64_t)nkv + nh) > 0x7fffffff - APPEND_WARPS)
            return failf(KD_ERR_UNSUPPORTED, "%s: 2^31 or more new heads", fn);
    }
    a.first[n_seqs] = (int)total;
    if (k_ld < (int64_t)nkv * hd || v_ld < (int64_t)nkv * hd || (nh && q_ld < (int64_t)nh * hd) ||
        k_ld > INT64_MAX / 4 / (total + 1) || v_ld > INT64_MAX / 4 / (total + 1) || (nh && q_ld > INT64_MAX / 4 / (total + 1)))
        return failf(KD_ERR_INVALID_ARG, "%s: k_ld %lld, v_ld %lld, q_ld %lld", fn, (long long)k_ld, (long long)v_ld, (long long)q_ld);
    if (!total) return KD_OK;
    if (!k || !v || (nh > 0 && (!q || !q_out))) return failf(KD_ERR_INVALID_ARG, "%s: null argument", fn);
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
