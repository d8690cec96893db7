// kd_attn_paged.cu -- a decode step's attention over a paged cache of fp16 or Q8_0 rows: the
// part of each session's keys that it reads for itself, and the merge.
//
// Sessions differ in length by orders of magnitude, so the blocks of 128 keys of all
// (session, head)s are one sequence of which every CTA takes an equal share (kd_paged.h).
// A warp takes 32 keys of each of the CTA's blocks: 16-byte asynchronous copies into its
// own buffers, its next piece's keys fetched when this piece's scores are done and its
// next values when this piece's are; a running maximum and sum.  Pages are looked up two
// pieces ahead, one lane per 16 keys (a page is a multiple of 16).  At the end of a
// (session, head) the warps' sums are joined in shared memory and go out, divided, if
// no other CTA has a share of it, else to a record that the merge kernel reads.
//
// The products are m16n8k16 MMAs over transposed operands (keys are rows, the group's query
// heads columns), with queries and weights as fp16 pairs hi + lo: good to 2^-22 of a value, but no finer than half of
// fp16's least step, 2^-25, which a value from 2^-3 on does not notice.  Queries are split as they are, so one of 2^-10 keeps 15 bits
// (a power of two for each row of queries would keep them, and take queries beyond 65504: the merging of the rows' maxima cost shared prefixes
// 2 to 8 % and this kernel 1.4, and was not kept).  Weights are scaled up first (UP below).  The
// Q8_0 form scales each 32-dim block's partial scores by the key's block scale in fp32
// and multiplies the value scales into the weights, so neither cache is rounded again.
//
// Long sessions are bound by memory: 48 of 0 to 16384 keys (462 MB, 8 KV heads of 128) take 84 us with the merge, 5.8 TB/s
// without it (a CTA at its share of the rate would need 560 for one (session, head) of 16384).  Few keys are bound by
// latency: 37 of one session 3.6 us (launch, page, keys), 8 sessions of 1238 to 1365 13.7, 10.3 where the keys are in L2 (664
// blocks on 456 CTAs, merge 2.5).  The Q8_0 form is bound by instructions: the 48 sessions (246 MB) 73 us, issue 0.62.
//
// Nothing waits on an mbarrier, so nothing can run out.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "kd_attn_common.cuh"
#include "kd_host.h"
#include "kd_paged.h"

namespace kd {

template <int HD, bool Q8>
struct PagedSmem {
    static constexpr int NREG = Q8 ? 1 : HD / 64;         // 128-byte columns of a row
    static constexpr int COL = PAGED_KEYS * 128;          // one of a piece
    static constexpr int SCALES = NREG * COL;             // Q8_0: the scales, 8 bytes a row, behind the quants
    static constexpr int PART = SCALES + (Q8 ? PAGED_KEYS * 8 : 0);
    static constexpr int WARP = 2 * PART;
    // row r's 16-byte chunk c, placed as the 128-byte swizzle does
    static __device__ __forceinline__ uint32_t off(int row, int chunk) {
        return (uint32_t)((chunk >> 3) * COL + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
    }
    static constexpr int merge(int gq) { return PAGED_WARPS * gq * PAGED_REC(HD) * 4; }
    static constexpr int total(int gq) { return PAGED_WARPS * WARP + merge(gq); }
};
// CTAs per SM: as many as fill its shared memory and leave the warps the registers they need.
template <int HD, int GQ, bool Q8>
constexpr int paged_per_sm() {
    return Q8 ? (GQ == 8 ? 2 : 4) : GQ == 8 ? (HD == 64 ? 3 : 2) : HD == 64 ? 5 : 3;
}

__device__ __forceinline__ void paged_cp16(uint32_t dst, const void* src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void paged_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void paged_wait_but() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncwarp();
}

__device__ __forceinline__ float2 paged_h2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// Bytes 0 and 2, or 1 and 3, of v, each u = q + 128, as half2(q, q') exactly.
__device__ __forceinline__ uint32_t paged_u8(uint32_t v, uint32_t sel) {
    const uint32_t h = __byte_perm(v, 0x64646464u, sel);
    uint32_t r;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
    return r;
}

// A block of a (session, head), and the next ones in order.
struct PagedAt {
    int b, h, blk, nb;  // session, KV head, block of nb
    // Block x, the first of the CTA's.
    __device__ __forceinline__ void seek(const PagedArgs& a, int x) {
        b = a.hint[(int)blockIdx.x * PAGED_HINTS / a.ctas];
        while (x >= a.s[b + 1].first * a.nkv) ++b;
        nb = a.s[b + 1].first - a.s[b].first;
        const int r = x - a.s[b].first * a.nkv;
        h = r / nb;
        blk = r - h * nb;
    }
    __device__ __forceinline__ void next(const PagedArgs& a) {
        if (++blk < nb) return;
        blk = 0;
        if (++h < a.nkv) return;
        h = 0;
        do {
            if (++b >= a.B) {
                nb = 1;
                return;
            }
            nb = a.s[b + 1].first - a.s[b].first;
        } while (nb == 0);
    }
};

template <int HD, int GQ, bool Q8>
__global__ void __launch_bounds__(PAGED_WARPS * 32, paged_per_sm<HD, GQ, Q8>()) paged_kernel(const __grid_constant__ PagedArgs a) {
    using L = PagedSmem<HD, Q8>;
    constexpr int KT = PAGED_KEYS / 16;
    constexpr int KS = HD / 16, NU = HD / 8, CH = Q8 ? 8 : HD / 8;  // k-steps, 8-dim tiles, 16-byte chunks of a row
    constexpr int NQ = GQ > 4 ? GQ / 4 : 1;                         // N-tiles of heads
    constexpr int REC = PAGED_REC(HD);
    extern __shared__ __align__(1024) uint8_t paged_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const uint32_t kbase = smem_u32(paged_smem + warp * L::WARP), vbase = kbase + L::PART;
    float* joined = reinterpret_cast<float*>(paged_smem + PAGED_WARPS * L::WARP);  // [warp][GQ][REC]

    const int x0 = a.share.begin(blockIdx.x), x1 = a.share.begin(blockIdx.x + 1);
    int left = x1 - x0;  // blocks still to take
    PagedAt at;
    if (left > 0) at.seek(a, x0);
    pdl_launch_dependents();
    // Beside the prefix kernel: not its end is waited for, but that it has seen the end of all before it.  Its word, stored
    // after its own wait and loaded here in acquire order, makes visible what was visible there.  It is stored before this
    // kernel can start, or at most some instructions later; where it is not seen soon the wait is for the kernel's end.
    const bool beside = a.started != nullptr;
    bool seen = false;
    if (beside) {
        if (lane == 0)
            for (int i = 0; i < 256 && !seen; ++i) {
                unsigned long long x;
                asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(x) : "l"(a.started) : "memory");
                seen = x == a.call;
            }
        seen = __any_sync(FULL_MASK, seen);
    }
    if (!seen) pdl_wait();
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0 && !beside) *a.err = 0;
        for (int b = 0; a.empty && b < a.B; ++b)  // sessions without keys
            if (a.s[b].to == 0)
                for (int i = threadIdx.x; i < a.nh * HD; i += PAGED_WARPS * 32) a.out[(size_t)b * a.nh * HD + i] = __float2half_rn(0.0f);
    }
    if (left <= 0) {
        pdl_wait();  // (the only CTA)
        return;
    }

    // The warp's piece of a block: keys [key, key + n) of the session (n <= 0: none).
    auto first_key = [&](const PagedAt& t) { return a.s[t.b].from + (t.blk * PAGED_WARPS + warp) * PAGED_KEYS; };
    auto keys = [&](const PagedAt& t) { return min(PAGED_KEYS, a.s[t.b].to - first_key(t)); };
    // The page of 16 keys (lane 0 and 1: the piece's two runs); -1 where there is none.
    auto look_up = [&](const PagedAt& t, bool have) {
        int page = -1;
        const int key = first_key(t) + 16 * lane;
        if (have && lane < 2 && key < a.s[t.b].to) {
            page = a.table[(int64_t)(key < a.s[t.b].lead_keys ? a.s[t.b].lead : t.b) * a.table_ld + key / a.ps];
            if ((unsigned)page >= (unsigned)a.n_pages) {
                if (a.fault) *a.fault = 1;
                page = -1;
            }
        }
        return page;
    };
    // The lane's chunks of a piece: row j * ROWS + lane / CH, chunk lane % CH, j < CH; a
    // place repeats the swizzle every 8 rows.
    constexpr int ROWS = 32 / CH, PER = 8 / ROWS;
    uint32_t place[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) place[j] = L::off(j * ROWS + lane / CH, lane % CH);
    // Copy part 0 (K) or 1 (V) of the warp's piece, whose runs' pages lanes 0 and 1 hold.
    auto issue = [&](const PagedAt& t, int pages, bool have, int part) {
        const int n = have ? keys(t) : 0;
        if (n > 0) {
            const uint32_t dst = part ? vbase : kbase;
            int64_t row[KT];
            bool ok[KT];
#pragma unroll
            for (int i = 0; i < KT; ++i) {
                const int page = __shfl_sync(FULL_MASK, pages, i);
                ok[i] = page >= 0;
                row[i] = ok[i] ? ((int64_t)page * a.nkv + t.h) * a.ps + (first_key(t) + 16 * i) % a.ps : 0;
            }
            const uint8_t* base = (const uint8_t*)(part ? a.v : a.k) + (lane % CH) * 16;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int i = j * ROWS / 16, r = j * ROWS + lane / CH;
                const bool get = ok[i] && r < n;
                paged_cp16(dst + place[j % PER] + (j / PER) * 8 * 128,
                           base + (get ? (row[i] + (r & 15)) * (Q8 ? 128 : 2 * HD) : 0), get);
            }
            if constexpr (Q8) {
                if (lane < 16) {  // two rows' scales a lane
                    const int i = lane >> 3, r = 2 * lane;
                    const bool get = ok[i] && r < n;
                    paged_cp16(dst + L::SCALES + lane * 16, (const uint8_t*)(part ? a.vs : a.ks) + (get ? (row[i] + (r & 15)) * 8 : 0), get);
                }
            }
        }
        paged_commit();
    };

    PagedAt nxt = at, nn;
    nxt.next(a);
    nn = nxt;
    if (left > 1) nn.next(a);
    int pg = look_up(at, true);
    int pg_nxt = look_up(nxt, left > 1), pg_nn = look_up(nn, left > 2);
    issue(at, pg, true, 0);
    issue(at, pg, true, 1);

    // B fragments of Q^T: column 2h + part of N-tile j is head 4j + h, part 0 the fp16
    // rounding of q, part 1 what it left over.  Q8_0: per 32-dim block and 16-dim half
    // the k order is dims 4c .. 4c + 3, as the quants' operand has it.
    const int colh = g >> 1;
    const bool col_lo = (g & 1) != 0;
    uint32_t qb[NQ][KS][2];
    auto load_q = [&](const PagedAt& t) {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int h = 4 * j + colh;
            const bool on = h < GQ;
            const float* qp = a.q + ((size_t)t.b * a.nh + (size_t)t.h * GQ + (on ? h : 0)) * HD;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float2 u, w;
                if constexpr (Q8) {
                    const float4 f = *reinterpret_cast<const float4*>(qp + 16 * ks + 4 * c);
                    u = make_float2(f.x, f.y);
                    w = make_float2(f.z, f.w);
                } else {
                    u = *reinterpret_cast<const float2*>(qp + 16 * ks + 2 * c);
                    w = *reinterpret_cast<const float2*>(qp + 16 * ks + 2 * c + 8);
                }
                qb[j][ks][0] = !on ? 0u : (col_lo ? f2_lo(u.x, u.y) : f2_hi(u.x, u.y));
                qb[j][ks][1] = !on ? 0u : (col_lo ? f2_lo(w.x, w.y) : f2_hi(w.x, w.y));
            }
        }
    };
    // Weights are held as e^UP times their value, 403 times: a pair is then good to 2^-22 of a weight or 2^-33 of the
    // largest (one of 2^-14 of it keeps 19 bits, one of 2^-23 10; Q8_0 scales them with the value scales).
    constexpr float UP = Q8 ? 0.0f : 6.0f;
    // m: the running maximum of head 4j + c, l: the lane's part of its sum, o = sum p v
    // (Q8_0: times 2^oe, so that weights times scales stay in fp16's normal range).
    float m[NQ], l[NQ], o[NU / 2][NQ][4];
    int oe = 0;
    bool any = false;  // (Q8_0) oe is set
    auto start = [&]() {
        any = false;
        oe = 0;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            m[j] = -INFINITY;
            l[j] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < NU / 2; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][j][i] = 0.0f;
        }
    };
    load_q(at);
    start();

    for (;;) {
        const int n = keys(at);
        const bool more = left > 1;
        unsigned runs = 0;  // the 16-key runs that have a page
#pragma unroll
        for (int t = 0; t < KT; ++t) runs |= (__shfl_sync(FULL_MASK, pg, t) >= 0 ? 1u : 0u) << t;
        paged_wait_but<1>();  // the K part
        float sv[NQ][KT][2];
        if (n > 0) {
            float sacc[KT][NQ][4];
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int j = 0; j < NQ; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sacc[t][j][i] = 0.0f;
            if constexpr (!Q8) {
                uint32_t ka[2][KT][4];  // a k-step's keys, fetched a step ahead
                auto load_k = [&](int ks) {
#pragma unroll
                    for (int t = 0; t < KT; ++t) {
                        uint32_t(&k)[4] = ka[ks & 1][t];
                        ldsm_x4(kbase + L::off(16 * t + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * ks + (lane >> 4)), k[0], k[1], k[2], k[3]);
                    }
                };
                load_k(0);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    if (ks + 1 < KS) load_k(ks + 1);
#pragma unroll
                    for (int j = 0; j < NQ; ++j)
#pragma unroll
                        for (int t = 0; t < KT; ++t) {
                            const uint32_t(&k)[4] = ka[ks & 1][t];
                            mma_16816_acc(sacc[t][j], k[0], k[1], k[2], k[3], qb[j][ks][0], qb[j][ks][1]);
                        }
                }
            } else {
                const uint8_t* scales = paged_smem + warp * L::WARP + L::SCALES;
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    const uint2 s0 = *reinterpret_cast<const uint2*>(scales + (16 * t + g) * 8);
                    const uint2 s1 = *reinterpret_cast<const uint2*>(scales + (16 * t + g + 8) * 8);
                    const float2 d0p[2] = {paged_h2(s0.x), paged_h2(s0.y)}, d1p[2] = {paged_h2(s1.x), paged_h2(s1.y)};
#pragma unroll
                    for (int blk = 0; blk < 4; ++blk) {
                        uint32_t r0, r1, r2, r3;
                        ldsm_x4(kbase + L::off(16 * t + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * blk + (lane >> 4)), r0, r1, r2, r3);
                        const uint32_t a0 = u8x2_lo_to_half2(r0), a2 = u8x2_hi_to_half2(r0);
                        const uint32_t a1 = u8x2_lo_to_half2(r1), a3 = u8x2_hi_to_half2(r1);
                        const uint32_t e0 = u8x2_lo_to_half2(r2), e2 = u8x2_hi_to_half2(r2);
                        const uint32_t e1 = u8x2_lo_to_half2(r3), e3 = u8x2_hi_to_half2(r3);
                        const float d0 = (blk & 1) ? d0p[blk >> 1].y : d0p[blk >> 1].x;
                        const float d1 = (blk & 1) ? d1p[blk >> 1].y : d1p[blk >> 1].x;
#pragma unroll
                        for (int j = 0; j < NQ; ++j) {
                            float s[4];
                            mma_16816_zero(s, a0, a1, a2, a3, qb[j][2 * blk][0], qb[j][2 * blk][1]);
                            mma_16816_acc(s, e0, e1, e2, e3, qb[j][2 * blk + 1][0], qb[j][2 * blk + 1][1]);
                            sacc[t][j][0] = __fmaf_rn(d0, s[0], sacc[t][j][0]);
                            sacc[t][j][1] = __fmaf_rn(d0, s[1], sacc[t][j][1]);
                            sacc[t][j][2] = __fmaf_rn(d1, s[2], sacc[t][j][2]);
                            sacc[t][j][3] = __fmaf_rn(d1, s[3], sacc[t][j][3]);
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float sc = __fadd_rn(sacc[t][j][2 * e], sacc[t][j][2 * e + 1]);  // both parts
                        const bool seen = 16 * t + g + 8 * e < n && ((runs >> t) & 1);
                        sv[j][t][e] = seen ? __fmul_rn(sc, a.scale) : -INFINITY;
                    }
        }
        __syncwarp();
        issue(nxt, pg_nxt, more, 0);
        if (n > 0) {
            // Softmax of head 4j + c over keys 16t + g and 16t + g + 8; the weights are taken
            // against the new running maximum (0 while every score is -inf).
            float f[NQ];
            bool same = true;
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                float mx = m[j];
#pragma unroll
                for (int t = 0; t < KT; ++t) mx = fmaxf(mx, fmaxf(sv[j][t][0], sv[j][t][1]));
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, x));
                const float ref = mx == -INFINITY ? 0.0f : __fsub_rn(mx, UP);
                f[j] = m[j] == mx ? 1.0f : expf(__fsub_rn(m[j], mx == -INFINITY ? 0.0f : mx));
                same = same && f[j] == 1.0f;
                m[j] = mx;
                float s = 0.0f;
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool seen = 16 * t + g + 8 * e < n && ((runs >> t) & 1);
                        sv[j][t][e] = seen ? expf(__fsub_rn(sv[j][t][e], ref)) : 0.0f;
                        s = __fadd_rn(s, sv[j][t][e]);
                    }
                l[j] = __fmaf_rn(l[j], f[j], s);
            }
            paged_wait_but<1>();  // the V part
            float pscale = 1.0f;
            if constexpr (Q8) {
                // 2^oe from the largest value scale so far: p d 2^oe < 2^14
                const uint8_t* scales = paged_smem + warp * L::WARP + L::PART + L::SCALES;
                const uint2 w = *reinterpret_cast<const uint2*>(scales + lane * 8);
                float dm = 0.0f;
                if (lane < n && ((runs >> (lane >> 4)) & 1)) {
                    const float2 x = paged_h2(w.x), y = paged_h2(w.y);
                    dm = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y)));
                }
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) dm = fmaxf(dm, __shfl_xor_sync(FULL_MASK, dm, x));
                if (dm > 0.0f && dm <= 65504.0f) {
                    const int e = 140 - ((__float_as_int(dm) >> 23) & 0xff);  // within [-2, 37] for fp16 scales
                    if (!any) {
                        oe = e;  // o is still 0
                    } else if (e < oe) {
                        const float down = __int_as_float((127 + e - oe) << 23);
#pragma unroll
                        for (int j = 0; j < NQ; ++j) f[j] = __fmul_rn(f[j], down);
                        same = false;
                        oe = e;
                    }
                    any = true;
                }
                pscale = __int_as_float((127 + oe) << 23);
            }
            if (__any_sync(FULL_MASK, !same)) {
#pragma unroll
                for (int j = 0; j < NQ; ++j)
#pragma unroll
                    for (int mt = 0; mt < NU / 2; ++mt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[mt][j][i] = __fmul_rn(o[mt][j][i], f[j]);
            }
            const int src0 = (2 * c) * 4 + colh, src1 = src0 + 4;
#pragma unroll
            for (int js = 0; js < KT; ++js) {
                if (16 * js < n) {
                    float v[NQ][4];  // weights of keys 2c, 2c + 1, 2c + 8, 2c + 9 for the lane's column head
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        v[j][0] = __shfl_sync(FULL_MASK, sv[j][js][0], src0);
                        v[j][1] = __shfl_sync(FULL_MASK, sv[j][js][0], src1);
                        v[j][2] = __shfl_sync(FULL_MASK, sv[j][js][1], src0);
                        v[j][3] = __shfl_sync(FULL_MASK, sv[j][js][1], src1);
                    }
                    if constexpr (!Q8) {
                        uint32_t pb[NQ][2];
#pragma unroll
                        for (int j = 0; j < NQ; ++j) {
                            const bool on = 4 * j + colh < GQ;
                            pb[j][0] = !on ? 0u : (col_lo ? f2_lo(v[j][0], v[j][1]) : f2_hi(v[j][0], v[j][1]));
                            pb[j][1] = !on ? 0u : (col_lo ? f2_lo(v[j][2], v[j][3]) : f2_hi(v[j][2], v[j][3]));
                        }
                        constexpr int VB = 4;  // 16-dim tiles fetched at a time
                        uint32_t va[VB][4];
#pragma unroll
                        for (int mt0 = 0; mt0 < NU / 2; mt0 += VB) {
#pragma unroll
                            for (int u = 0; u < VB; ++u)
                                ldsm_x4_trans(vbase + L::off(16 * js + (lane >> 4) * 8 + (lane & 7), 2 * (mt0 + u) + ((lane >> 3) & 1)),
                                              va[u][0], va[u][1], va[u][2], va[u][3]);
#pragma unroll
                            for (int u = 0; u < VB; ++u)
#pragma unroll
                                for (int j = 0; j < NQ; ++j)
                                    mma_16816_acc(o[mt0 + u][j], va[u][0], va[u][1], va[u][2], va[u][3], pb[j][0], pb[j][1]);
                        }
                    } else {
                        // weights times their keys' block scales (0 where there is no key)
                        const uint8_t* scales = paged_smem + warp * L::WARP + L::PART + L::SCALES;
                        const int kb = 16 * js + 2 * c;
                        const uint4 wa = lds_v4(scales + kb * 8), wb = lds_v4(scales + (kb + 8) * 8);
                        const bool run = (runs >> js) & 1;
                        float2 dk[4][2];  // [key][blocks 0, 1 | 2, 3]
                        dk[0][0] = paged_h2(run && kb < n ? wa.x : 0u);
                        dk[0][1] = paged_h2(run && kb < n ? wa.y : 0u);
                        dk[1][0] = paged_h2(run && kb + 1 < n ? wa.z : 0u);
                        dk[1][1] = paged_h2(run && kb + 1 < n ? wa.w : 0u);
                        dk[2][0] = paged_h2(run && kb + 8 < n ? wb.x : 0u);
                        dk[2][1] = paged_h2(run && kb + 8 < n ? wb.y : 0u);
                        dk[3][0] = paged_h2(run && kb + 9 < n ? wb.z : 0u);
                        dk[3][1] = paged_h2(run && kb + 9 < n ? wb.w : 0u);
#pragma unroll
                        for (int blk = 0; blk < 4; ++blk) {
                            uint32_t r0, r1, r2, r3;
                            ldsm_x4_trans(vbase + L::off(16 * js + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * blk + (lane >> 4)), r0, r1, r2, r3);
                            // dims 2g of a 16-dim slice (MMA row g), then 2g + 1 (row g + 8)
                            const uint32_t s00 = paged_u8(r0, 0x4240), s01 = paged_u8(r0, 0x4341);
                            const uint32_t s02 = paged_u8(r1, 0x4240), s03 = paged_u8(r1, 0x4341);
                            const uint32_t s10 = paged_u8(r2, 0x4240), s11 = paged_u8(r2, 0x4341);
                            const uint32_t s12 = paged_u8(r3, 0x4240), s13 = paged_u8(r3, 0x4341);
#pragma unroll
                            for (int j = 0; j < NQ; ++j) {
                                float p[4];
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    p[r] = __fmul_rn(__fmul_rn(v[j][r], pscale), (blk & 1) ? dk[r][blk >> 1].y : dk[r][blk >> 1].x);
                                const bool on = 4 * j + colh < GQ;
                                const uint32_t b0 = !on ? 0u : (col_lo ? f2_lo(p[0], p[1]) : f2_hi(p[0], p[1]));
                                const uint32_t b1 = !on ? 0u : (col_lo ? f2_lo(p[2], p[3]) : f2_hi(p[2], p[3]));
                                mma_16816_acc(o[2 * blk][j], s00, s01, s02, s03, b0, b1);
                                mma_16816_acc(o[2 * blk + 1][j], s10, s11, s12, s13, b0, b1);
                            }
                        }
                    }
                }
            }
        } else {
            paged_wait_but<1>();
        }
        __syncwarp();
        issue(nxt, pg_nxt, more, 1);

        if (!more || nxt.b != at.b || nxt.h != at.h) {
            // The end of the (session, head), or of the CTA's share of it: join the warps.
            const float down = Q8 ? __int_as_float((127 - oe) << 23) : 1.0f;
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[j] = __fadd_rn(l[j], __shfl_xor_sync(FULL_MASK, l[j], x));
                const int h = 4 * j + c;
                if (h < GQ) {
                    float* dst = joined + (warp * GQ + h) * REC;
#pragma unroll
                    for (int mt = 0; mt < NU / 2; ++mt) {
                        const float lo = __fadd_rn(o[mt][j][0], o[mt][j][1]), hi = __fadd_rn(o[mt][j][2], o[mt][j][3]);
                        if constexpr (Q8) {
                            *reinterpret_cast<float2*>(dst + 16 * mt + 2 * g) = make_float2(__fmul_rn(lo, down), __fmul_rn(hi, down));
                        } else {
                            dst[16 * mt + g] = lo;
                            dst[16 * mt + g + 8] = hi;
                        }
                    }
                    if (g == 0) *reinterpret_cast<float2*>(dst + HD) = make_float2(__fsub_rn(m[j], UP), l[j]);
                }
            }
            __syncthreads();
            const int s0 = a.s[at.b].first * a.nkv + at.h * at.nb;  // the (session, head)'s blocks
            const bool whole = a.s[at.b].from == 0 && x0 <= s0 && s0 + at.nb <= x1;
            float* rec = a.part + ((size_t)blockIdx.x + (size_t)at.b * a.nkv + at.h) * GQ * REC;
            __half* out = a.out + ((size_t)at.b * a.nh + (size_t)at.h * GQ) * HD;
            for (int i = threadIdx.x; i < GQ * (HD / 4); i += PAGED_WARPS * 32) {
                const int h = i / (HD / 4), d = i % (HD / 4) * 4;
                float M = -INFINITY, w[PAGED_WARPS], den = 0.0f;
#pragma unroll
                for (int k = 0; k < PAGED_WARPS; ++k) M = fmaxf(M, joined[(k * GQ + h) * REC + HD]);
                const float ref = M == -INFINITY ? 0.0f : M;
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < PAGED_WARPS; ++k) {
                    const float* r = joined + (k * GQ + h) * REC;
                    w[k] = expf(__fsub_rn(r[HD], ref));
                    den = __fmaf_rn(w[k], r[HD + 1], den);
                    const float4 v = *reinterpret_cast<const float4*>(r + d);
                    acc.x = __fmaf_rn(w[k], v.x, acc.x);
                    acc.y = __fmaf_rn(w[k], v.y, acc.y);
                    acc.z = __fmaf_rn(w[k], v.z, acc.z);
                    acc.w = __fmaf_rn(w[k], v.w, acc.w);
                }
                if (whole) {
                    if (den == 0.0f) den = 1.0f;  // no key has a page
                    const __half2 lo = __floats2half2_rn(__fdiv_rn(acc.x, den), __fdiv_rn(acc.y, den));
                    const __half2 hi = __floats2half2_rn(__fdiv_rn(acc.z, den), __fdiv_rn(acc.w, den));
                    __half2* p = reinterpret_cast<__half2*>(out + h * HD + d);
                    p[0] = lo;
                    p[1] = hi;
                } else {
                    *reinterpret_cast<float4*>(rec + h * REC + d) = acc;
                    if (d == 0) *reinterpret_cast<float2*>(rec + h * REC + HD) = make_float2(M, den);
                }
            }
            __syncthreads();
            if (more) {
                load_q(nxt);
                start();
            }
        }
        if (!more) break;
        --left;
        at = nxt;
        nxt = nn;
        pg = pg_nxt;
        pg_nxt = pg_nn;
        if (left > 2) nn.next(a);
        pg_nn = look_up(nn, left > 2);
    }
    // One CTA sees to it that this kernel does not end before the one beside it; the others leave their place to the next.
    if (beside && blockIdx.x == gridDim.x - 1) pdl_wait();
}

// The merge of a (session, head) that several CTAs share: out = sum_i w_i o_i / sum_i w_i l_i
// over its records, w_i = e^{m_i - max m}: those of its own keys and those that the CTAs of
// its group's shared keys left.  A block per (session, query head): a warp takes every fourth record, eight
// of them in flight, with a running maximum, and the warps' sums are joined in order.
constexpr int PAGED_MERGE_WARPS = 4;
template <int HD>
__global__ void __launch_bounds__(PAGED_MERGE_WARPS * 32) paged_merge_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ SharedArgs sh) {
    constexpr int REC = PAGED_REC(HD), DIMS = HD / 32;  // a lane's dims
    __shared__ float sums[PAGED_MERGE_WARPS][HD];
    __shared__ float2 ends[PAGED_MERGE_WARPS];  // a warp's maximum and denominator
    const int qh = blockIdx.x, b = blockIdx.y, gq = a.nh / a.nkv, h = qh / gq, i = qh - h * gq;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nb = a.s[b + 1].first - a.s[b].first, g = a.s[b].group;
    // n records of its own keys, then one of each set of CTAs that has some of the shared keys
    const float *rec = nullptr, *shared = nullptr;
    int n = 0, sets = 0;
    size_t set_step = 0;
    if (nb) {
        const int s0 = a.s[b].first * a.nkv + h * nb, c0 = a.share.taker(s0);
        n = a.share.taker(s0 + nb - 1) - c0 + 1;
        rec = a.part + (((size_t)c0 + (size_t)b * a.nkv + h) * gq + i) * REC;
    }
    if (g != SHARED_NONE) {
        const int per = sh.tile_queries * sh.side, query = (b - sh.g[g].lead) * gq + i, pass = query / per, T = sh.tiles(g);
        const int s0 = sh.g[g].first * sh.nkv + (h * sh.passes(g) + pass) * T, c0 = sh.share.taker(s0);
        sets = sh.share.taker(s0 + T - 1) - c0 + 1;
        shared = sh.part + shared_row(sh, g, h, pass, c0, query - pass * per) * REC;
        set_step = (size_t)per * REC;
    }
    pdl_wait();
    if (sh.n_groups && qh == 0 && b == 0 && warp == PAGED_MERGE_WARPS - 1) {  // the call's fault word
        int bad = 0;
        for (int k = lane; k < sh.sets * sh.side; k += 32) bad |= sh.status[k];
        bad = __any_sync(FULL_MASK, bad != 0);
        if (lane == 0) {
            *a.err = bad ? ERR_WAIT_TIMEOUT : 0;
            *sh.started = 0;  // so that a graph's next run finds its word new
        }
    }
    const int total = n + sets;
    if (!total || (n == 1 && !sets)) return;  // no keys, or written by the CTA itself
    auto record = [&](int k) {
        return k < n ? rec + (size_t)k * gq * REC : shared + (k - n) * set_step;
    };
    float acc[DIMS], M = -INFINITY, den = 0.0f;
#pragma unroll
    for (int d = 0; d < DIMS; ++d) acc[d] = 0.0f;
    constexpr int U = 8;
    for (int k0 = warp; k0 < total; k0 += U * PAGED_MERGE_WARPS) {
        float v[U][DIMS];
        float2 ml[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * PAGED_MERGE_WARPS;
            ml[u] = make_float2(-INFINITY, 0.0f);
            if (k < total) {
                const float* r = record(k);
                ml[u] = *reinterpret_cast<const float2*>(r + HD);
                if constexpr (DIMS == 4) {
                    const float4 f = *reinterpret_cast<const float4*>(r + lane * DIMS);
                    v[u][0] = f.x, v[u][1] = f.y, v[u][2] = f.z, v[u][3] = f.w;
                } else {
                    const float2 f = *reinterpret_cast<const float2*>(r + lane * DIMS);
                    v[u][0] = f.x, v[u][1] = f.y;
                }
            }
        }
        float top = M;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
        const float ref = top == -INFINITY ? 0.0f : top, f = expf(__fsub_rn(M, ref));
        M = top;
        den = __fmul_rn(den, f);
#pragma unroll
        for (int d = 0; d < DIMS; ++d) acc[d] = __fmul_rn(acc[d], f);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (ml[u].x != -INFINITY || ml[u].y != 0.0f) {  // else there are no keys (without a maximum but with a sum: NaN)
                const float w = expf(__fsub_rn(ml[u].x, ref));
                den = __fmaf_rn(w, ml[u].y, den);
#pragma unroll
                for (int d = 0; d < DIMS; ++d) acc[d] = __fmaf_rn(w, v[u][d], acc[d]);
            }
    }
#pragma unroll
    for (int d = 0; d < DIMS; ++d) sums[warp][lane * DIMS + d] = acc[d];
    if (lane == 0) ends[warp] = make_float2(M, den);
    __syncthreads();
    for (int d = threadIdx.x; d < HD; d += PAGED_MERGE_WARPS * 32) {
        float all = -INFINITY, o = 0.0f, l = 0.0f;
#pragma unroll
        for (int k = 0; k < PAGED_MERGE_WARPS; ++k) all = fmaxf(all, ends[k].x);
        const float ref = all == -INFINITY ? 0.0f : all;
#pragma unroll
        for (int k = 0; k < PAGED_MERGE_WARPS; ++k) {
            const float w = expf(__fsub_rn(ends[k].x, ref));
            o = __fmaf_rn(w, sums[k][d], o);
            l = __fmaf_rn(w, ends[k].y, l);
        }
        a.out[((size_t)b * a.nh + qh) * HD + d] = __float2half_rn(l == 0.0f ? 0.0f : __fdiv_rn(o, l));  // 0: no key has a page
    }
    pdl_launch_dependents();
}

#define KD_PAGED_GROUPS(HD_, Q8_, MACRO)             \
    switch (group) {                                 \
        case 1: MACRO(HD_, 1, Q8_); break;           \
        case 2: MACRO(HD_, 2, Q8_); break;           \
        case 4: MACRO(HD_, 4, Q8_); break;           \
        case 8: MACRO(HD_, 8, Q8_); break;           \
    }
#define KD_PAGED_SHAPES(MACRO)                       \
    if (q8) {                                        \
        KD_PAGED_GROUPS(128, true, MACRO)            \
    } else if (hd == 64) {                           \
        KD_PAGED_GROUPS(64, false, MACRO)            \
    } else {                                         \
        KD_PAGED_GROUPS(128, false, MACRO)           \
    }

template <int HD, int GQ, bool Q8>
static cudaError_t paged_prepare(int dev, int* per_sm) {
    static OncePerDevice once;
    static std::atomic<int> fit{0};
    const cudaError_t e = once(dev, [] {
        cudaError_t r = cudaFuncSetAttribute(paged_kernel<HD, GQ, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             PagedSmem<HD, Q8>::total(GQ));
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(paged_kernel<HD, GQ, Q8>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        int n = 0;
        if (r == cudaSuccess)
            r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, paged_kernel<HD, GQ, Q8>, PAGED_WARPS * 32, PagedSmem<HD, Q8>::total(GQ));
        if (r == cudaSuccess) fit.store(n < 1 ? 1 : n, std::memory_order_relaxed);
        return r;
    });
    *per_sm = fit.load(std::memory_order_relaxed);
    return e;
}

int paged_slots(int hd, int group, bool q8, int dev, int num_sms, cudaError_t* e) {
    int per_sm = 0;
    *e = cudaErrorInvalidValue;
#define KD_PREPARE(HD_, GQ_, Q8_) *e = paged_prepare<HD_, GQ_, Q8_>(dev, &per_sm)
    KD_PAGED_SHAPES(KD_PREPARE)
#undef KD_PREPARE
    const int n = per_sm * num_sms;
    return *e != cudaSuccess ? 0 : n < PAGED_MAX_CTAS ? n : PAGED_MAX_CTAS;
}

static void paged_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = s;
}

cudaError_t launch_paged(const PagedArgs& a, int hd, bool q8, cudaStream_t s) {
    const int group = a.nh / a.nkv;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    paged_config(cfg, attr, s);
    cfg.gridDim = dim3(a.ctas);
    cfg.blockDim = dim3(PAGED_WARPS * 32);
#define KD_LAUNCH(HD_, GQ_, Q8_)                                   \
    cfg.dynamicSmemBytes = (PagedSmem<HD_, Q8_>::total(GQ_));      \
    return cudaLaunchKernelEx(&cfg, paged_kernel<HD_, GQ_, Q8_>, a)
    KD_PAGED_SHAPES(KD_LAUNCH)
#undef KD_LAUNCH
    return cudaErrorInvalidValue;
}

cudaError_t launch_paged_merge(const PagedArgs& a, const SharedArgs& sh, int hd, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    paged_config(cfg, attr, s);
    cfg.gridDim = dim3(a.nh, a.B);
    cfg.blockDim = dim3(PAGED_MERGE_WARPS * 32);
    return hd == 64 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<64>, a, sh) : cudaLaunchKernelEx(&cfg, paged_merge_kernel<128>, a, sh);
}

}  // namespace kd
