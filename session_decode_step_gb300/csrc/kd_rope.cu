// kd_rope.cu -- rotary positions: the plan on the host, and rows of heads rotated
// in place or to another place.
//
// A thread holds both halves of four pairs (of two or one where sizes or alignment do not allow that), forms
// their angles once and takes them through its share of the token's heads, four heads' loads in flight;
// dims that pass move in the same chunks.  As a pair never leaves the thread, x may be written in place.  fp32
// results are rounded once (the angle and the products are carried as pairs of fp32); fp16
// and bf16 ones are formed in fp32, whose error is 2^-13 and 2^-16 of theirs.
//
// Bound by memory for many tokens: 8191 tokens of 40 fp16 heads of 128 (168 MB) 27.4 us, 6.1 TB/s, 0.90 of the measured
// copy; with eight pairs a thread 30.4 us (half the threads fit), interleaved pairs of 8192 x 32 heads 25.5 against 26.7 us.
// Eight tokens of 32 fp32 heads take 2.3 us, an empty launch 2.1.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "kd_host.h"
#include "kd_rope.cuh"
#include "kd_rope.h"

namespace kd {

struct RopeArgs {
    const void* x;
    void* out;
    const int* pos;
    int64_t ld, ld_out;
    int tokens, heads, hd;
    int per, groups;  // heads per thread, threads per token and chunk
    int nr, nc;       // chunks of P pairs, and with the unrotated dims' chunks of P
    RopeAngles<KD_ROPE_MAX_DIM / 2> r;
};

template <typename T, int P>
struct alignas(sizeof(T) * P) RopeVec {
    T v[P];
};
__device__ __forceinline__ void from_f(float x, float& o) { o = x; }
__device__ __forceinline__ void from_f(float x, __half& o) { o = __float2half_rn(x); }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16& o) { o = __float2bfloat16_rn(x); }

constexpr int ROPE_THREADS = 256;

template <typename T, bool PAIRS, int P>
__global__ void __launch_bounds__(ROPE_THREADS, 3) rope_kernel(const __grid_constant__ RopeArgs a) {
    using V = RopeVec<T, P>;
    constexpr bool EXACT = std::is_same<T, float>::value;
    constexpr int U = 4;  // heads in flight
    __shared__ float2 tab[ROPE_TAB];
    __shared__ unsigned long long turns[KD_ROPE_MAX_DIM / 2];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, n = blockDim.x * blockDim.y;
    for (int i = tid; i < ROPE_TAB; i += n) tab[i] = ROPE_COS[i];
    for (int i = tid; i < a.r.rot / 2; i += n) turns[i] = a.r.turns[i];
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int64_t unit = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int token = (int)(unit / a.groups), chunk = threadIdx.x;
    if (token >= a.tokens) return;
    const int h0 = (int)(unit - (int64_t)token * a.groups) * a.per, h1 = min(a.heads, h0 + a.per);
    // The chunk's two vectors: of P pairs, or behind them of dims that pass unchanged.
    const bool turned = chunk < a.nr;
    if (!turned && a.x == a.out) return;
    const int d0 = PAIRS ? 2 * P * chunk : turned ? P * chunk : a.r.rot + 2 * P * (chunk - a.nr);
    const int d1 = PAIRS || !turned ? d0 + P : d0 + a.r.rot / 2;
    const T* x = (const T*)a.x + token * a.ld;
    T* out = (T*)a.out + token * a.ld_out;
    V u[U], w[U];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (h + i < h1) {
                u[i] = *reinterpret_cast<const V*>(x + (int64_t)(h + i) * a.hd + d0);
                w[i] = *reinterpret_cast<const V*>(x + (int64_t)(h + i) * a.hd + d1);
            }
    };
    load(h0);
    float ch[P], cl[P], sh[P], sl[P];
    if (turned) {
        const int pos = a.pos[token];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 c, s;
            rope_angle<EXACT>(turns[min(P * chunk + i, KD_ROPE_MAX_DIM / 2 - 1)], pos, a.r.mh, a.r.ml, tab, c, s);
            ch[i] = c.x, cl[i] = c.y, sh[i] = s.x, sl[i] = s.y;
        }
    }
    // Pair i of the chunk, interleaved: p and q.  (The last chunk may hold dims that pass.)
    auto turn_pair = [&](T& p, T& q, int i) {
        const float pf = to_f(p), qf = to_f(q);
        const float2 r = rope_turn2<EXACT>(make_float2(pf, qf), make_float2(qf, pf), make_float2(ch[i], ch[i]), make_float2(cl[i], cl[i]),
                                           make_float2(-sh[i], sh[i]), make_float2(-sl[i], sl[i]), make_float2(-ch[i], -ch[i]),
                                           make_float2(sh[i], -sh[i]));
        if (P * chunk + i < a.r.rot / 2) {
            from_f(r.x, p);
            from_f(r.y, q);
        }
    };
    auto turn = [&](V& a0, V& a1) {
        if constexpr (PAIRS && P == 1) {
            turn_pair(a0.v[0], a1.v[0], 0);
        } else if constexpr (PAIRS) {
#pragma unroll
            for (int i = 0; i < P / 2; ++i) {
                turn_pair(a0.v[2 * i], a0.v[2 * i + 1], i);
                turn_pair(a1.v[2 * i], a1.v[2 * i + 1], P / 2 + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                constexpr int last = P - 1;
                const int k = i + 1 < P ? i + 1 : last;  // P = 1: the same again
                const float2 p = make_float2(to_f(a0.v[i]), to_f(a0.v[k])), q = make_float2(to_f(a1.v[i]), to_f(a1.v[k]));
                const float2 c = make_float2(ch[i], ch[k]), s = make_float2(sh[i], sh[k]);
                const float2 c2 = make_float2(cl[i], cl[k]), s2 = make_float2(sl[i], sl[k]);
                const float2 nc = f2_neg(c), ns = f2_neg(s);
                const float2 rp = rope_turn2<EXACT>(p, q, c, c2, ns, f2_neg(s2), nc, s), rq = rope_turn2<EXACT>(q, p, c, c2, s, s2, nc, ns);
                from_f(rp.x, a0.v[i]);
                from_f(rp.y, a0.v[k]);
                from_f(rq.x, a1.v[i]);
                from_f(rq.y, a1.v[k]);
            }
        }
    };
    for (int h = h0; h < h1; h += U) {
        if (h > h0) load(h);
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (h + k < h1) {
                if (turned) turn(u[k], w[k]);
                *reinterpret_cast<V*>(out + (int64_t)(h + k) * a.hd + d0) = u[k];
                *reinterpret_cast<V*>(out + (int64_t)(h + k) * a.hd + d1) = w[k];
            }
    }
}

template <typename T, int P>
static cudaError_t launch_rope_p(RopeArgs& a, int sms, cudaStream_t s) {
    a.nr = a.r.pairs ? (a.r.rot + 2 * P - 1) / (2 * P) : a.r.rot / 2 / P;
    a.nc = a.hd / (2 * P);
    const int by = ROPE_THREADS / a.nc;
    // Heads per thread: the angles are formed once for them, and a thread that loops keeps
    // loads in flight; but every SM should have a thousand threads' worth of work first.
    const int64_t threads = (int64_t)a.tokens * a.heads * a.nc;
    int64_t per = threads / ((int64_t)sms * 512);
    per = per < 1 ? 1 : per > 8 ? 8 : per;
    a.per = (int)per;
    a.groups = (a.heads + a.per - 1) / a.per;
    const int64_t units = (int64_t)a.tokens * a.groups;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)((units + by - 1) / by));
    cfg.blockDim = dim3(a.nc, by);
    cfg.stream = s;
    return a.r.pairs ? cudaLaunchKernelEx(&cfg, rope_kernel<T, true, P>, a) : cudaLaunchKernelEx(&cfg, rope_kernel<T, false, P>, a);
}

// Heads of an odd number of dims: a thread a dim.  Such heads rotate an even number of them.
template <typename T>
__global__ void __launch_bounds__(ROPE_THREADS) rope_odd_kernel(const __grid_constant__ RopeArgs a) {
    constexpr bool EXACT = std::is_same<T, float>::value;
    __shared__ float2 tab[ROPE_TAB];
    for (int i = threadIdx.x; i < ROPE_TAB; i += ROPE_THREADS) tab[i] = ROPE_COS[i];
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    // a pair, or one of the dims behind them
    const int half = a.r.rot / 2, units = a.hd - half;
    const int64_t i = (int64_t)blockIdx.x * ROPE_THREADS + threadIdx.x, head = i / units;
    const int token = (int)(head / a.heads), e = (int)(i - head * units);
    if (token >= a.tokens) return;
    const int h = (int)(head - (int64_t)token * a.heads);
    const T* x = (const T*)a.x + token * a.ld + (int64_t)h * a.hd;
    T* out = (T*)a.out + token * a.ld_out + (int64_t)h * a.hd;
    if (e >= half) {
        out[e + half] = x[e + half];
        return;
    }
    const int d0 = a.r.pairs ? 2 * e : e, d1 = a.r.pairs ? d0 + 1 : e + half;
    const float p = to_f(x[d0]), q = to_f(x[d1]);
    float2 c, s;
    rope_angle<EXACT>(a.r.turns[e], a.pos[token], a.r.mh, a.r.ml, tab, c, s);
    const float2 r = rope_turn2<EXACT>(make_float2(p, q), make_float2(q, p), make_float2(c.x, c.x), make_float2(c.y, c.y),
                                       make_float2(-s.x, s.x), make_float2(-s.y, s.y), make_float2(-c.x, -c.x), make_float2(s.x, -s.x));
    from_f(r.x, out[d0]);
    from_f(r.y, out[d1]);
}

template <typename T>
static cudaError_t launch_rope(RopeArgs& a, cudaStream_t s) {
    constexpr int W = 4;
    // vectors of p: addresses and strides lie on multiples of p, heads are whole pairs of vectors, and so are the
    // two halves of what is rotated
    auto fits = [&](int p) {
        return a.hd % (2 * p) == 0 && a.ld % p == 0 && a.ld_out % p == 0 && (a.r.pairs || a.r.rot % (2 * p) == 0) &&
               (((uintptr_t)a.x | (uintptr_t)a.out) & (p * sizeof(T) - 1)) == 0;
    };
    int sms = 0;
    const cudaError_t e = current_sms(&sms);
    if (e != cudaSuccess) return e;
    if (fits(W)) return launch_rope_p<T, W>(a, sms, s);
    if (fits(2)) return launch_rope_p<T, 2>(a, sms, s);
    if (a.hd % 2 == 0) return launch_rope_p<T, 1>(a, sms, s);
    const int64_t threads = (int64_t)a.tokens * a.heads * (a.hd - a.r.rot / 2);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)((threads + ROPE_THREADS - 1) / ROPE_THREADS));
    cfg.blockDim = dim3(ROPE_THREADS);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, rope_odd_kernel<T>, a);
}

kd_status rope_table_check(const char* fn, const kd_rope_table* t) {
    if (t->head_dim < 2 || t->head_dim > KD_ROPE_MAX_DIM || t->rot_dim < 2 || t->rot_dim % 2 || t->rot_dim > t->head_dim ||
        (t->layout != KD_ROPE_HALF && t->layout != KD_ROPE_PAIRS) || t->reserved || !std::isfinite((float)t->magnitude))
        return failf(KD_ERR_INVALID_ARG, "%s: not a table that kd_rope_plan made (head_dim %d, rot_dim %d, layout %d)", fn,
                     t->head_dim, t->rot_dim, t->layout);
    return KD_OK;
}

// Numbers of twice a double's length, as a sum hi + lo of two (|lo| at most half of hi's last bit), good to some 2^-100: a
// frequency rounded to a double turns by 2^-55 of a turn too much a position, 2^-36 rad at 131072.
struct Two {
    double hi, lo;
};
static Two sum_of(double x, double y) {
    const double s = x + y, b = s - x;
    return {s, (x - (s - b)) + (y - b)};
}
static Two negative(Two x) { return {-x.hi, -x.lo}; }
static Two plus(Two x, Two y) {
    const Two s = sum_of(x.hi, y.hi), t = sum_of(x.lo, y.lo), u = sum_of(s.hi, s.lo + t.hi);
    return sum_of(u.hi, u.lo + t.lo);
}
static Two times(Two x, Two y) {
    const double p = x.hi * y.hi;
    return sum_of(p, std::fma(x.hi, y.hi, -p) + (x.hi * y.lo + x.lo * y.hi));
}
static Two over(Two x, Two y) {
    const double q = x.hi / y.hi;
    if (!std::isfinite(q) || q == 0.0) return {q, 0.0};
    const Two r = plus(x, negative(times(y, {q, 0.0})));
    return sum_of(q, (r.hi + r.lo) / y.hi);
}
static Two power_of(Two x, int n) {
    Two r = {1.0, 0.0};
    for (; n; n >>= 1) {
        if (n & 1) r = times(r, x);
        x = times(x, x);
    }
    return r;
}
// theta^(-1 / n): a step of Newton's method from the double next to it.  (In two factors, as theta^-1 may leave a double's
// normal range; n = 1 is nobody's: a single pair turns by 1.)
static Two root_of_inverse(double theta, int n) {
    const Two y = {std::pow(theta, -1.0 / n), 0.0};
    if (n == 1) return y;
    const Two r = times(times({theta, 0.0}, power_of(y, n / 2)), power_of(y, n - n / 2));  // 1 + n times y's relative error
    const Two e = plus({1.0, 0.0}, negative(r));
    return plus(y, over(times(y, e), {(double)n, 0.0}));
}
// x turns modulo 1 (positions are whole, so whole turns drop out), in 2^-64 of one, rounded.
static uint64_t turns_of(Two x) {
    if (std::fabs(x.lo) >= 1.0) x.lo -= std::floor(x.lo);
    x = sum_of(x.hi - std::floor(x.hi), x.lo);
    if (x.hi < 0.0) x = plus(x, {1.0, 0.0});
    if (x.hi >= 1.0) x = plus(x, {-1.0, 0.0});
    const double top = std::ldexp(x.hi, 32), whole = std::floor(top);
    // (lo may be below 0, and the sum a whole turn: both are right modulo 2^64)
    return ((uint64_t)(int64_t)whole << 32) + (uint64_t)(int64_t)std::floor(std::ldexp(top - whole, 32) + std::ldexp(x.lo, 64) + 0.5);
}

}  // namespace kd

extern "C" {

kd_status kd_rope_plan(const kd_rope_config* c, kd_rope_table* out) {
    using namespace kd;
    const char* fn = "kd_rope_plan";
    if (!c || !out) return failf(KD_ERR_INVALID_ARG, "%s: null argument", fn);
    if (c->head_dim > KD_ROPE_MAX_DIM)
        return failf(KD_ERR_UNSUPPORTED, "%s: head_dim %d (at most %d)", fn, c->head_dim, KD_ROPE_MAX_DIM);
    if (c->rot_dim < 2 || c->rot_dim % 2 || c->rot_dim > c->head_dim)
        return failf(KD_ERR_INVALID_ARG, "%s: rot_dim %d of head_dim %d", fn, c->rot_dim, c->head_dim);
    if (c->layout != KD_ROPE_HALF && c->layout != KD_ROPE_PAIRS)
        return failf(KD_ERR_INVALID_ARG, "%s: layout %d", fn, c->layout);
    if (c->scaling < KD_ROPE_UNSCALED || c->scaling > KD_ROPE_RAMP)
        return failf(KD_ERR_INVALID_ARG, "%s: scaling %d", fn, c->scaling);
    if (c->reserved) return failf(KD_ERR_INVALID_ARG, "%s: reserved must be 0", fn);
    if (!(c->theta > 1.0) || !std::isfinite(c->theta)) return failf(KD_ERR_INVALID_ARG, "%s: theta %g", fn, c->theta);
    if (!std::isfinite((float)c->magnitude)) return failf(KD_ERR_INVALID_ARG, "%s: magnitude %g", fn, c->magnitude);
    const bool blends = c->scaling == KD_ROPE_BANDS || c->scaling == KD_ROPE_RAMP;
    if (c->scaling != KD_ROPE_UNSCALED && (!(c->factor > 0.0) || !std::isfinite(c->factor)))
        return failf(KD_ERR_INVALID_ARG, "%s: factor %g", fn, c->factor);
    if (blends && (c->original_ctx < 1 || !(c->low > 0.0) || !(c->high > c->low) || !std::isfinite(c->high)))
        return failf(KD_ERR_INVALID_ARG, "%s: original_ctx %d, low %g, high %g", fn, c->original_ctx, c->low, c->high);
    const double turn = 6.283185307179586476925286766559;
    const int n = c->rot_dim;
    double a = 0, b = 0;
    if (c->scaling == KD_ROPE_RAMP) {
        auto dim = [&](double turns) { return n * std::log(c->original_ctx / (turns * turn)) / (2 * std::log(c->theta)); };
        a = std::fmax(0.0, std::floor(dim(c->high)));
        b = std::fmin(n - 1.0, std::ceil(dim(c->low)));
    }
    kd_rope_table t = {};
    t.head_dim = c->head_dim;
    t.rot_dim = n;
    t.layout = c->layout;
    t.magnitude = c->magnitude;
    const Two one = {1.0, 0.0}, two_pi = {turn, 0x1.1a62633145c07p-52}, step = root_of_inverse(c->theta, n / 2);
    Two power = one;  // theta^(-2i / n)
    for (int i = 0; i < n / 2; ++i) {
        Two f = power;
        power = times(power, step);
        if (c->scaling == KD_ROPE_LINEAR) f = over(f, {c->factor, 0.0});
        if (blends) {
            Two slow;  // how much of the pair's pace is slowed
            if (c->scaling == KD_ROPE_BANDS)
                slow = over(plus({c->high, 0.0}, negative(over(times({(double)c->original_ctx, 0.0}, f), two_pi))), plus({c->high, 0.0}, {-c->low, 0.0}));
            else
                slow = over({i - a, 0.0}, {std::fmax(b - a, 0.001), 0.0});
            if (slow.hi <= 0.0) slow = {0.0, 0.0};
            if (slow.hi >= 1.0) slow = one;
            f = times(f, plus(plus(one, negative(slow)), over(slow, {c->factor, 0.0})));
        }
        if (!std::isfinite(f.hi)) return failf(KD_ERR_INVALID_ARG, "%s: factor %g leaves no finite frequency", fn, c->factor);
        t.turns[i] = turns_of(over(f, two_pi));
    }
    *out = t;
    return KD_OK;
}

kd_status kd_rope(const kd_rope_table* rope, const void* x, int32_t dtype, int64_t ld, const int32_t* positions,
                  int32_t n_tokens, int32_t n_heads, void* out, int64_t ld_out, kd_stream stream) {
    using kd::failf;
    const char* fn = "kd_rope";
    if (!rope || (n_tokens && (!x || !positions || !out))) return failf(KD_ERR_INVALID_ARG, "%s: null argument", fn);
    const kd_status st = kd::rope_table_check(fn, rope);
    if (st != KD_OK) return st;
    if (dtype < KD_F32 || dtype > KD_BF16) return failf(KD_ERR_INVALID_ARG, "%s: dtype %d", fn, dtype);
    if (n_tokens < 0 || n_heads < 1) return failf(KD_ERR_INVALID_ARG, "%s: %d tokens of %d heads", fn, n_tokens, n_heads);
    const int64_t row = (int64_t)n_heads * rope->head_dim;
    if (ld < row || ld_out < row || ld > INT64_MAX / 4 / ((int64_t)n_tokens + 1) || ld_out > INT64_MAX / 4 / ((int64_t)n_tokens + 1))
        return failf(KD_ERR_INVALID_ARG, "%s: ld %lld, ld_out %lld for rows of %lld", fn, (long long)ld, (long long)ld_out,
                     (long long)row);
    const uintptr_t mask = dtype == KD_F32 ? 3 : 1;
    if ((((uintptr_t)x | (uintptr_t)out) & mask) || ((uintptr_t)positions & 3))
        return failf(KD_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    if (n_tokens && x == out && ld != ld_out) return failf(KD_ERR_INVALID_ARG, "%s: in place, but ld %lld and ld_out %lld", fn, (long long)ld, (long long)ld_out);
    if ((int64_t)n_tokens * n_heads > 0x7fffffff) return failf(KD_ERR_UNSUPPORTED, "%s: %d tokens of %d heads", fn, n_tokens, n_heads);
    if (!n_tokens) return KD_OK;
    kd::RopeArgs a = {};
    a.x = x;
    a.out = out;
    a.pos = positions;
    a.ld = ld;
    a.ld_out = ld_out;
    a.tokens = n_tokens;
    a.heads = n_heads;
    a.hd = rope->head_dim;
    kd::rope_fill(a.r, *rope);
    cudaStream_t s = (cudaStream_t)stream;
    switch (dtype) {
        case KD_F32: KD_TRY(kd::launch_rope<float>(a, s)); break;
        case KD_F16: KD_TRY(kd::launch_rope<__half>(a, s)); break;
        default: KD_TRY(kd::launch_rope<__nv_bfloat16>(a, s));
    }
    return KD_OK;
}

}  // extern "C"
