// kd_rope.cuh -- rotary positions on the device: a position's angle as a whole
// number, and its cosine and sine.
//
// Pair i turns by turns[i] / 2^64 of a turn per position, so position p's angle is
// the low 64 bits of p * turns[i], off by |p| 2^-65 of a turn (2^-45 rad at 131072), where an fp32
// angle is off by 2e-3 at 32k positions and an fp64 one costs a range reduction on
// two units per SM.  The angle is the nearest 256th of a turn, whose cosine and sine
// come from a table of fp32 pairs, and a rest of at most pi / 256, whose sine and cosine
// are two terms of their series; the sum theorem joins them.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kd.h"
#include "kd_device.cuh"

namespace kd {

// cos(2 pi j / 256), j = 0..64, each as the sum of two fp32 values; the sine is the same read backwards.
constexpr int ROPE_TAB = 65;
static __device__ const float2 ROPE_COS[ROPE_TAB] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.ffd8860000000p-1f, 0x1.099a1a0000000p-30f}, {0x1.ff621e0000000p-1f, 0x1.bcb6be0000000p-28f},
    {0x1.fe9cda0000000p-1f, 0x1.a031080000000p-26f}, {0x1.fd88da0000000p-1f, 0x1.e892920000000p-28f}, {0x1.fc26480000000p-1f, -0x1.e3cc060000000p-26f},
    {0x1.fa75580000000p-1f, -0x1.eeb5d20000000p-30f}, {0x1.f876500000000p-1f, -0x1.63ad160000000p-27f}, {0x1.f6297c0000000p-1f, 0x1.feeb960000000p-26f},
    {0x1.f38f3a0000000p-1f, 0x1.8c9cb20000000p-26f}, {0x1.f0a7f00000000p-1f, -0x1.1b73ca0000000p-27f}, {0x1.ed740e0000000p-1f, 0x1.da12580000000p-27f},
    {0x1.e9f4160000000p-1f, -0x1.273a440000000p-26f}, {0x1.e6288e0000000p-1f, 0x1.891c220000000p-26f}, {0x1.e212100000000p-1f, 0x1.3da1ba0000000p-27f},
    {0x1.ddb13c0000000p-1f, -0x1.2667b80000000p-26f}, {0x1.d906bc0000000p-1f, 0x1.e651a80000000p-26f}, {0x1.d4134e0000000p-1f, -0x1.d646d80000000p-26f},
    {0x1.ced7b00000000p-1f, -0x1.7867120000000p-26f}, {0x1.c954b20000000p-1f, 0x1.3411f40000000p-29f}, {0x1.c38b300000000p-1f, -0x1.cfe84a0000000p-26f},
    {0x1.bd7c0a0000000p-1f, 0x1.8df2a60000000p-26f}, {0x1.b728340000000p-1f, 0x1.465b900000000p-27f}, {0x1.b090a60000000p-1f, -0x1.fabf800000000p-27f},
    {0x1.a9b6620000000p-1f, 0x1.21d4340000000p-26f}, {0x1.a29a7a0000000p-1f, 0x1.189e080000000p-31f}, {0x1.9b3e040000000p-1f, 0x1.fce1d00000000p-27f},
    {0x1.93a2240000000p-1f, 0x1.324c800000000p-26f}, {0x1.8bc8060000000p-1f, 0x1.62a2e80000000p-26f}, {0x1.83b0e00000000p-1f, 0x1.7ff2ee0000000p-26f},
    {0x1.7b5df20000000p-1f, 0x1.3557d80000000p-28f}, {0x1.72d0840000000p-1f, -0x1.02000e0000000p-26f}, {0x1.6a09e60000000p-1f, 0x1.9fcef40000000p-27f},
    {0x1.610b760000000p-1f, -0x1.5c5a640000000p-26f}, {0x1.57d6940000000p-1f, -0x1.6e626c0000000p-26f}, {0x1.4e6cac0000000p-1f, -0x1.0706860000000p-27f},
    {0x1.44cf320000000p-1f, 0x1.4247760000000p-27f}, {0x1.3affa20000000p-1f, 0x1.240a180000000p-26f}, {0x1.30ff800000000p-1f, -0x1.8f47e60000000p-28f},
    {0x1.26d0540000000p-1f, 0x1.9ba25c0000000p-26f}, {0x1.1c73b40000000p-1f, -0x1.9465ce0000000p-27f}, {0x1.11eb360000000p-1f, -0x1.7c969c0000000p-26f},
    {0x1.07387a0000000p-1f, -0x1.b740040000000p-27f}, {0x1.f8ba4e0000000p-2f, -0x1.01d9520000000p-28f}, {0x1.e2b5d40000000p-2f, -0x1.fe42720000000p-28f},
    {0x1.cc66ea0000000p-2f, -0x1.b38ee80000000p-28f}, {0x1.b5d1000000000p-2f, 0x1.3c2b980000000p-27f}, {0x1.9ef7940000000p-2f, 0x1.d476c60000000p-29f},
    {0x1.87de2a0000000p-2f, 0x1.abaa580000000p-28f}, {0x1.7088540000000p-2f, -0x1.e0b74c0000000p-27f}, {0x1.58f9a80000000p-2f, -0x1.4a9c040000000p-27f},
    {0x1.4135ca0000000p-2f, -0x1.7d13400000000p-27f}, {0x1.2940620000000p-2f, 0x1.dab3e00000000p-27f}, {0x1.111d260000000p-2f, 0x1.58fb3c0000000p-29f},
    {0x1.f19f980000000p-3f, -0x1.37a83a0000000p-29f}, {0x1.c0b8260000000p-3f, 0x1.4fc9ec0000000p-28f}, {0x1.8f8b840000000p-3f, -0x1.cb2cfa0000000p-30f},
    {0x1.5e21440000000p-3f, 0x1.22cff20000000p-29f}, {0x1.2c81060000000p-3f, 0x1.d1cc280000000p-28f}, {0x1.f564e60000000p-4f, -0x1.2ad19e0000000p-29f},
    {0x1.917a6c0000000p-4f, -0x1.eb25ea0000000p-31f}, {0x1.2d520a0000000p-4f, -0x1.a63cc20000000p-29f}, {0x1.91f6600000000p-5f, -0x1.de44fe0000000p-30f},
    {0x1.9215600000000p-6f, -0x1.0b93300000000p-31f}, {0x0.0p+0f, 0x0.0p+0f},
};

// A value in fp32.
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// x + y and x * y as fp32 pairs (the rounded result and what the rounding left out).
__device__ __forceinline__ float2 two_sum(float x, float y) {
    const float s = __fadd_rn(x, y), b = __fsub_rn(s, x);
    return make_float2(s, __fadd_rn(__fsub_rn(x, __fsub_rn(s, b)), __fsub_rn(y, b)));
}
__device__ __forceinline__ float2 two_prod(float x, float y) {
    const float p = __fmul_rn(x, y);
    return make_float2(p, __fmaf_rn(x, y, -p));
}

// Cosine and sine of `phase` / 2^64 turns as fp32 pairs.  EXACT: to about 2^-44, so that
// a rotation can be rounded to fp32 once; else the pairs' second parts are 0 and the first
// good to 2^-24.  tab: ROPE_COS in shared memory.
template <bool EXACT>
__device__ __forceinline__ void rope_cos_sin(uint64_t phase, const float2* tab, float2& c, float2& s) {
    const int j = (int)((phase + (1ull << 55)) >> 56);  // the nearest 256th of a turn
    const int64_t r = (int64_t)(phase - ((uint64_t)j << 56));
    const int rh = (int)(r >> 25);
    const float2 C = tab[j & 63], S = tab[64 - (j & 63)];
    // the rest in radians: xh + xl
    constexpr float PI2_HI = 0x1.921fb6p+2f, PI2_LO = -0x1.777a5cp-23f, UNIT = 0x1p-39f;
    const float a = (float)rh;
    float xh = __fmul_rn(a, PI2_HI * UNIT);
    const float x2 = __fmul_rn(xh, xh);
    const float third = __fmul_rn(xh, __fmul_rn(x2, __fmaf_rn(x2, 1.0f / 120.0f, -1.0f / 6.0f)));  // sin x - x
    float2 cc, ss;
    if constexpr (EXACT) {
        const float b = __fmaf_rn((float)((unsigned)r & 0x1ffffffu), 0x1p-25f, (float)(rh - (int)a));
        const float xl = __fadd_rn(__fmaf_rn(a, PI2_HI * UNIT, -xh), __fmaf_rn(a, PI2_LO * UNIT, __fmul_rn(b, PI2_HI * UNIT)));
        const float sl = __fadd_rn(xl, third);  // sin x = xh + sl
        // cos x - 1 = ch + cl
        const float ch = __fmul_rn(x2, -0.5f);
        const float x2l = __fmaf_rn(xh, xh, -x2);
        const float cl = __fmaf_rn(-0.5f, x2l, __fmaf_rn(-xh, xl, __fmul_rn(__fmul_rn(x2, x2), 1.0f / 24.0f)));
        auto join = [&](float2 A, float2 B, float sign) {  // A cos x + sign B sin x
            const float2 p = two_prod(B.x, __fmul_rn(sign, xh)), u = two_prod(A.x, ch);
            const float2 t = two_sum(A.x, p.x), w = two_sum(t.x, u.x);
            float lo = __fadd_rn(__fadd_rn(t.y, w.y), __fadd_rn(A.y, __fadd_rn(p.y, u.y)));
            lo = __fmaf_rn(A.x, cl, lo);
            lo = __fmaf_rn(__fmul_rn(sign, B.x), sl, lo);
            lo = __fmaf_rn(__fmul_rn(sign, B.y), xh, lo);
            const float h = __fadd_rn(w.x, lo);
            return make_float2(h, __fadd_rn(__fsub_rn(w.x, h), lo));
        };
        cc = join(C, S, -1.0f);
        ss = join(S, C, 1.0f);
    } else {
        xh = __fadd_rn(xh, third);
        const float ch = __fmul_rn(x2, __fmaf_rn(x2, 1.0f / 24.0f, -0.5f));
        cc = make_float2(__fadd_rn(C.x, __fmaf_rn(C.x, ch, __fmul_rn(-S.x, xh))), 0.0f);
        ss = make_float2(__fadd_rn(S.x, __fmaf_rn(S.x, ch, __fmul_rn(C.x, xh))), 0.0f);
    }
    // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
    const int q = (j >> 6) & 3;
    c = (q & 1) ? ss : cc;
    s = (q & 1) ? cc : ss;
    if (q == 1 || q == 2) c = make_float2(-c.x, -c.y);
    if (q >= 2) s = make_float2(-s.x, -s.y);
}

// Two results x c + y s at a time (the sign of the sine is the caller's); each of c and s the
// sum of its two parts.  EXACT: rounded to fp32 once, up to about 2^-44 (products and the sum with
// what their roundings left out, formed with their signs turned, as pairs of operations cannot turn an
// operand's); else to within two roundings, of the first parts alone.  nc, ns: -ch, -sh.
template <bool EXACT>
__device__ __forceinline__ float2 rope_turn2(float2 x, float2 y, float2 ch, float2 cl, float2 sh, float2 sl, float2 nc, float2 ns) {
    if constexpr (!EXACT) return f2_fma(x, ch, f2_mul(y, sh));
    const float2 p = f2_mul(x, nc), q = f2_mul(y, ns), t = f2_add(p, q);     // all negative
    const float2 left = f2_add(f2_fma(x, ch, p), f2_fma(y, sh, q));         // what the products left out
    const float2 minus = make_float2(-1.0f, -1.0f);
    const float2 b = f2_fma(p, minus, t);                                   // what of t is q, and what either is off by
    const float2 te = f2_add(f2_fma(f2_fma(b, minus, t), minus, p), f2_fma(b, minus, q));
    const float2 lo = f2_add(f2_fma(te, minus, left), f2_fma(x, cl, f2_mul(y, sl)));
    float2 v = f2_fma(t, minus, lo);
    if (!(fmaxf(fabsf(t.x), fabsf(t.y)) <= 3.402823466e38f)) {  // infinite: as the plain sum has it
        if (!(fabsf(t.x) <= 3.402823466e38f)) v.x = -t.x;
        if (!(fabsf(t.y) <= 3.402823466e38f)) v.y = -t.y;
    }
    return v;
}

// The table's entries for a launch: N of the plan's, and the magnitude as an fp32 pair.
template <int N>
struct RopeAngles {
    int rot, pairs;  // dims rotated; pairs: layout KD_ROPE_PAIRS
    float mh, ml;
    unsigned long long turns[N];
};
template <int N>
inline void rope_fill(RopeAngles<N>& a, const kd_rope_table& t) {
    a.rot = t.rot_dim;
    a.pairs = t.layout == KD_ROPE_PAIRS;
    a.mh = (float)t.magnitude;
    a.ml = (float)(t.magnitude - (double)a.mh);
    for (int i = 0; i < N; ++i) a.turns[i] = i < t.rot_dim / 2 ? t.turns[i] : 0;
}
template <bool EXACT>
__device__ __forceinline__ void rope_angle(uint64_t turns, int pos, float mh, float ml, const float2* tab, float2& c,
                                           float2& s) {
    rope_cos_sin<EXACT>((uint64_t)(int64_t)pos * turns, tab, c, s);
    if constexpr (EXACT) {
        auto scale = [&](float2 v) {
            const float2 p = two_prod(v.x, mh);
            return make_float2(p.x, __fadd_rn(p.y, __fmaf_rn(v.y, mh, __fmul_rn(v.x, ml))));
        };
        c = scale(c);
        s = scale(s);
    } else {
        c.x = __fmul_rn(c.x, mh);
        s.x = __fmul_rn(s.x, mh);
    }
}

}  // namespace kd
