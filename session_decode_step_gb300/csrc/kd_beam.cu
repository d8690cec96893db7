// kd_beam.cu -- beam selection: each prompt's best continuations over its beams
// and the vocabulary, straight from the step's logits.
//
// Beam w of a group has the cumulative log probability score_w; continuing it
// with token v gives
//   s(w, v) = score_w + x_wv - L_w,   L_w = log sum_u e^{x_wu},
// and the group's K best pairs are wanted, larger s first, then lower w, then
// lower v.  Within a row the order is the logits' own, so one pass over the
// logits does everything that touches all of them: a CTA walks a segment of one
// row in blocks of 4096, leaves (m, sum e^{x-m}) of every block and the
// segment's K best logits, sorted.  A second kernel, one CTA per group, forms
// L_w, merges each row's lists, and merges the rows by s.
//
// The selection costs next to nothing once K candidates are known: a block whose
// largest logit does not exceed the K-th best so far is passed over, so a random
// row brings about K ln(blocks) late candidates.  The first block's are found
// through the threads' own maxima: the K-th largest of the 256 bounds the K-th
// largest logit from below, and few logits lie above it.  The warps keep their
// candidates apart and agree on a new bound after 4, 16 and 64 blocks.
//
// s decides between rows, where two candidates can lie as close as fp32 rounds:
// L_w's last steps and s are fp64 (a handful of operations per row); the sums of
// exponentials are fp32 inside a block, in an order that depends on nothing but
// the block, and exact 64-bit fixed point across blocks.  So a row's result does
// not depend on the segments, hence not on the rest of the batch.
#include <cuda_runtime.h>

#include <cmath>

#include "kd_device.cuh"
#include "kd_host.h"

namespace kd {

constexpr int BS_THREADS = 256;
constexpr int BS_WARPS = BS_THREADS / 32;
constexpr int BS_VPT = 16;                      // logits per thread and block
constexpr int BS_BLOCK = BS_THREADS * BS_VPT;   // logits per block
constexpr int BS_MAX_BLOCKS = 128;              // vocabulary up to 524288
constexpr int BS_MAX_SEGS = 32;                 // segments (lists) per row: one per lane of the merge
constexpr int BS_MAX_OUT = 32;
// A warp's candidates: up to 2 K kept, and at most all 512 of a block on top.
constexpr int BS_CAP = 2 * BS_MAX_OUT + 32 * BS_VPT;
static_assert(KD_BEAM_MAX_VOCAB == BS_BLOCK * BS_MAX_BLOCKS && KD_BEAM_MAX_OUT == BS_MAX_OUT, "kd.h limits");

// (x, index) as a 64-bit key whose unsigned order is: larger x, then lower index
// (-0 equals +0).  0 is no candidate.
__device__ __forceinline__ unsigned beam_ord(float x) {
    const unsigned u = __float_as_uint(x + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float beam_unord(unsigned ord) {
    return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7fffffffu) : ~ord);
}
__device__ __forceinline__ unsigned long long beam_key(float x, int i) {
    return ((unsigned long long)beam_ord(x) << 32) | (unsigned)~i;
}
__device__ __forceinline__ float beam_key_x(unsigned long long k) { return beam_unord((unsigned)(k >> 32)); }
__device__ __forceinline__ int beam_key_i(unsigned long long k) { return (int)~(unsigned)k; }

// The lanes holding the warp's largest key: by high words, then, among equals, low words.  0: no lane holds one.
__device__ __forceinline__ unsigned warp_best(unsigned long long k) {
    const unsigned hi = (unsigned)(k >> 32), mh = __reduce_max_sync(FULL_MASK, hi);
    if (mh == 0) return 0u;
    unsigned who = __ballot_sync(FULL_MASK, hi == mh);
    if (who & (who - 1)) {
        const unsigned ml = __reduce_max_sync(FULL_MASK, hi == mh ? (unsigned)k : 0u);
        who = __ballot_sync(FULL_MASK, hi == mh && (unsigned)k == ml);
    }
    return who;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float LOG2E = 1.44269504088896341f;
// Pairs of fp32 in a 64-bit register.
__device__ __forceinline__ unsigned long long pack2(float x, float y) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A beam's row is read only if the beam can continue: not finished, score > -inf (a NaN score is dead too).
__device__ __forceinline__ bool beam_live(const float* scores, const int* done, int r) {
    return (!scores || scores[r] > -INFINITY) && !(done && done[r]);
}

struct BeamArgs {
    const float* logits;  // [rows][ld]
    long ld;
    int V, W, K, nblk;    // vocabulary, beams per group, candidates kept, blocks per row
    int nseg, seg_blocks; // segments per row, blocks per segment
    const float* scores;  // [rows], or nullptr (zeros)
    const int* done;      // [rows], or nullptr
    int eos;
    float2* part;              // [rows][nblk] (m, sum e^{x - m})
    unsigned long long* keys;  // [rows][nseg][K] sorted, 0-padded
    int *parents, *tokens, *done_out;
    float* scores_out;
};

// Thread t's logits of a block: 4t .. 4t + 3 of each quarter.  VEC: 16-byte loads (every row 16-byte aligned).
template <bool VEC>
__device__ __forceinline__ void beam_load(const float* p, int n, int t, float (&x)[BS_VPT]) {
    if (VEC && n >= BS_BLOCK) {
#pragma unroll
        for (int i = 0; i < BS_VPT / 4; ++i) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(p + i * 4 * BS_THREADS + 4 * t));
            x[4 * i] = v.x;
            x[4 * i + 1] = v.y;
            x[4 * i + 2] = v.z;
            x[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < BS_VPT; ++i) {
            const int e = (i >> 2) * 4 * BS_THREADS + 4 * t + (i & 3);
            x[i] = e < n ? __ldg(p + e) : -INFINITY;
        }
    }
}

// The warp's candidates, sorted and cut to the K best, then zeros up to 32; returns their number.
__device__ __forceinline__ int beam_compact(unsigned long long* buf, unsigned long long* best, int n, int K, int lane) {
    __syncwarp();
    for (int q = lane; q < n; q += 32) {
        const unsigned long long k = buf[q];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += buf[j] > k ? 1 : 0;
        if (rank < K) best[rank] = k;
    }
    __syncwarp();
    const int c = min(n, K);
    buf[lane] = lane < c ? best[lane] : 0ull;
    __syncwarp();
    return c;
}

// Rank of key k, at place `lane` of its own warp's sorted 32, among all warps' lists (list w at lists + w * stride).
__device__ __forceinline__ int beam_rank(const unsigned long long* lists, int stride, unsigned long long k, int warp,
                                         int lane) {
    int rank = lane;
#pragma unroll
    for (int w = 0; w < BS_WARPS; ++w) {
        if (w == warp) continue;
        const unsigned long long* l = lists + w * stride;
        int c = 0;  // larger keys, found by halving
#pragma unroll
        for (int h = 16; h > 0; h >>= 1)
            if (l[c + h - 1] > k) c += h;
        rank += c + (l[c] > k ? 1 : 0);
    }
    return rank;
}

template <bool VEC>
__global__ void __launch_bounds__(BS_THREADS, 4) beam_scan_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ unsigned long long cand[BS_WARPS][BS_CAP];
    __shared__ unsigned long long best[BS_WARPS][BS_MAX_OUT];
    __shared__ float2 wpart[BS_MAX_BLOCKS][BS_WARPS];
    __shared__ int count[BS_WARPS];
    __shared__ unsigned long long bound;  // the K-th best key known to all warps (0: fewer than K)
    pdl_launch_dependents();
    const int r = blockIdx.y, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    if (!beam_live(a.scores, a.done, r)) return;
    const int K = a.K, b0 = blockIdx.x * a.seg_blocks, nb = min(a.seg_blocks, a.nblk - b0);
    const float* row = a.logits + (size_t)r * a.ld;
    unsigned long long* buf = cand[warp];
    int cnt = 0;
    float thr = -INFINITY;  // a K-th best: later equals lose to it (higher indices)
    float nx[BS_VPT];
    beam_load<VEC>(row + (size_t)b0 * BS_BLOCK, a.V - b0 * BS_BLOCK, t, nx);
    if (t == 0) bound = 0ull;
#pragma unroll 2
    for (int b = 0; b < nb; ++b) {
        const int e0 = (b0 + b) * BS_BLOCK;
        float x[BS_VPT];
#pragma unroll
        for (int i = 0; i < BS_VPT; ++i) x[i] = nx[i];
        if (b + 1 < nb) beam_load<VEC>(row + e0 + BS_BLOCK, a.V - e0 - BS_BLOCK, t, nx);
        float m = x[0];
#pragma unroll
        for (int i = 1; i < BS_VPT; ++i) m = fmaxf(m, x[i]);
        float s;
        {  // two logits per instruction (packed fp32 adds and products)
            const unsigned long long nm = pack2(-m, -m), l2 = pack2(LOG2E, LOG2E);
            unsigned long long acc = 0ull;
#pragma unroll
            for (int i = 0; i < BS_VPT; i += 2) {
                const float2 d = unpack2(mul2(add2(pack2(x[i], x[i + 1]), nm), l2));
                acc = add2(acc, pack2(ex2(d.x), ex2(d.y)));
            }
            const float2 v = unpack2(acc);
            s = v.x + v.y;
        }
        if (s != s) {  // a NaN, or the largest is infinite: NaN counts as -inf, x - m as 0 where x == m
            m = -INFINITY;
#pragma unroll
            for (int i = 0; i < BS_VPT; ++i) {
                x[i] = fmaxf(x[i], -INFINITY);
                m = fmaxf(m, x[i]);
            }
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < BS_VPT; ++i) s += x[i] == m ? 1.0f : ex2((x[i] - m) * LOG2E);
            if (m == -INFINITY) s = 0.0f;
        }
        const float mw = beam_unord(__reduce_max_sync(FULL_MASK, beam_ord(m)));
        s = m == mw ? s : s * ex2((m - mw) * LOG2E);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(FULL_MASK, s, o);
        if (lane == 0) wpart[b][warp] = make_float2(mw, s);

        unsigned long long floor_key = 0ull;  // candidates of the first block: keys no less than this
        if (b == 0) {
            // the thread's largest key and its place in the warp; the K-th largest of all threads'
            int at = BS_VPT - 1;
#pragma unroll
            for (int i = BS_VPT - 2; i >= 0; --i) at = x[i] == m ? i : at;
            const unsigned long long k =
                m > -INFINITY ? beam_key(m, e0 + (at >> 2) * 4 * BS_THREADS + 4 * t + (at & 3)) : 0ull;
            best[warp][lane] = k;
            __syncwarp();
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < 32; ++j) {
                const unsigned long long o = best[warp][j];
                rank += o > k || (o == k && j < lane) ? 1 : 0;
            }
            __syncwarp();
            best[warp][rank] = k;
            __syncwarp();
            const unsigned long long sk = best[warp][lane];
            __syncthreads();
            if (sk && beam_rank(best[0], BS_MAX_OUT, sk, warp, lane) == K - 1) bound = sk;
            __syncthreads();
            floor_key = bound;
            thr = floor_key ? beam_key_x(floor_key) : -INFINITY;
        }
        const unsigned hot = __ballot_sync(FULL_MASK, floor_key ? m >= thr : m > thr);
        if (hot) {
            // x >= lo: x > thr, by the next value above; in the first block x >= thr
            float lo = floor_key ? thr : beam_unord(beam_ord(thr) + 1u);
            if (b > 0 && __popc(hot) >= K) {  // at least K logits are no less than the K-th largest lane maximum
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < 32; ++j) {
                    const float o = __shfl_sync(FULL_MASK, m, j);
                    rank += o > m || (o == m && j < lane) ? 1 : 0;
                }
                lo = __shfl_sync(FULL_MASK, m, __ffs(__ballot_sync(FULL_MASK, rank == K - 1)) - 1);
            }
#pragma unroll
            for (int i = 0; i < BS_VPT; ++i) {
                if (!__any_sync(FULL_MASK, x[i] >= lo)) continue;
                const unsigned long long k = beam_key(x[i], e0 + (i >> 2) * 4 * BS_THREADS + 4 * t + (i & 3));
                const bool in = x[i] >= lo && k >= floor_key;
                const unsigned who = __ballot_sync(FULL_MASK, in);
                if (in) buf[cnt + __popc(who & ((1u << lane) - 1u))] = k;
                cnt += __popc(who);
            }
            if (cnt > K + 24) {
                cnt = beam_compact(buf, best[warp], cnt, K, lane);
                thr = fmaxf(thr, beam_key_x(buf[K - 1]));
            }
        }
        if ((b == 3 || b == 15 || b == 63) && b + 1 < nb) {  // a new common bound after 4, 16, 64 blocks
            cnt = beam_compact(buf, best[warp], cnt, K, lane);
            __syncthreads();
            const unsigned long long k = buf[lane];
            if (k && beam_rank(cand[0], BS_CAP, k, warp, lane) == K - 1) bound = k;
            __syncthreads();
            if (bound) thr = fmaxf(thr, beam_key_x(bound));
        }
    }
    cnt = beam_compact(buf, best[warp], cnt, K, lane);
    if (lane == 0) count[warp] = cnt;
    __syncthreads();
    // the warps' sorted lists into the segment's
    unsigned long long* out = a.keys + ((size_t)r * a.nseg + blockIdx.x) * K;
    if (lane < cnt) {
        const unsigned long long k = buf[lane];
        const int rank = beam_rank(cand[0], BS_CAP, k, warp, lane);
        if (rank < K) out[rank] = k;
    }
    int total = 0;
#pragma unroll
    for (int w = 0; w < BS_WARPS; ++w) total += count[w];
    if (t < K && t >= total) out[t] = 0ull;
    if (t < nb) {  // the blocks' sums, warps in order
        float mb = -INFINITY, sb = 0.0f;
#pragma unroll
        for (int w = 0; w < BS_WARPS; ++w) mb = fmaxf(mb, wpart[t][w].x);
#pragma unroll
        for (int w = 0; w < BS_WARPS; ++w) {
            const float2 p = wpart[t][w];
            sb += p.x == mb ? p.y : p.y * ex2((p.x - mb) * LOG2E);
        }
        a.part[(size_t)r * a.nblk + b0 + t] = make_float2(mb, mb > -INFINITY ? sb : 0.0f);
    }
}

// One CTA per group: warps 0 .. W - 1 merge the rows' lists while warps W .. 2W - 1
// form the rows' log sums; then warp 0 merges the rows.
__global__ void __launch_bounds__(64 * KD_BEAM_MAX_BEAMS) beam_merge_kernel(const __grid_constant__ BeamArgs a) {
    extern __shared__ unsigned long long staged[];  // [W][nseg][K] the rows' lists
    __shared__ unsigned long long row_key[KD_BEAM_MAX_BEAMS][BS_MAX_OUT];
    __shared__ double row_s[KD_BEAM_MAX_BEAMS][BS_MAX_OUT];
    __shared__ unsigned long long row_o[KD_BEAM_MAX_BEAMS][BS_MAX_OUT + 2];  // row_s as order-preserving keys, 0-padded
    __shared__ double row_lg[KD_BEAM_MAX_BEAMS];
    __shared__ float row_m[KD_BEAM_MAX_BEAMS];
    __shared__ int row_n[KD_BEAM_MAX_BEAMS];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp < a.W ? warp : warp - a.W;
    const int g = blockIdx.x, r = g * a.W + w, K = a.K;
    const bool live = beam_live(a.scores, a.done, r);
    const float score = a.scores ? a.scores[r] : 0.0f;
    if (warp >= a.W) {
        // L = M + log sum_b s_b e^{m_b - M}; the sum in units of 2^-40 (a block's is at most 4096, the largest's at least 1)
        if (live) {
            const float2* part = a.part + (size_t)r * a.nblk;
            float2 p[BS_MAX_BLOCKS / 32];
            float M = -INFINITY;
#pragma unroll
            for (int q = 0; q < BS_MAX_BLOCKS / 32; ++q) {
                const int b = lane + 32 * q;
                p[q] = b < a.nblk ? __ldcg(part + b) : make_float2(-INFINITY, 0.0f);
                M = fmaxf(M, p[q].x);
            }
            M = beam_unord(__reduce_max_sync(FULL_MASK, beam_ord(M)));
            long long sum = 0;
#pragma unroll
            for (int q = 0; q < BS_MAX_BLOCKS / 32; ++q)
                sum += __float2ll_rn((p[q].x == M ? p[q].y : p[q].y * expf(p[q].x - M)) * 0x1p40f);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
            const double lg = log((double)sum * 0x1p-40);
            if (lane == 0) {
                row_lg[w] = lg;
                row_m[w] = M;
            }
        }
    } else if (live) {
        const unsigned long long* lists = a.keys + (size_t)r * a.nseg * K;
        unsigned long long* st = staged + (size_t)w * a.nseg * K;
        for (int i = lane; i < a.nseg * K; i += 32) st[i] = __ldcg(lists + i);
        __syncwarp();
        // lane l holds the head of list l and the entry after it
        const unsigned long long* at = st + lane * K;
        const int have = lane < a.nseg ? K : 0;
        unsigned long long head = have > 0 ? at[0] : 0ull, after = have > 1 ? at[1] : 0ull;
        int n = 0, next = 2;
        for (; n < K; ++n) {
            const unsigned who = warp_best(head);
            if (!who) break;
            if ((who >> lane) & 1u) {
                row_key[w][n] = head;
                head = after;
                after = next < have ? at[next] : 0ull;
                ++next;
            }
        }
        if (lane == 0) row_n[w] = n;
    } else if (lane == 0) {  // a finished beam stands for itself; a dead one offers nothing
        const bool fin = a.done && a.done[r] && score > -INFINITY;
        row_n[w] = fin ? 1 : 0;
        row_key[w][0] = (unsigned)~a.eos;
        row_s[w][0] = (double)score;
    }
    __syncthreads();
    if (warp < a.W) {
        unsigned long long o = 0ull;
        if (lane < row_n[w]) {
            if (live) {
                const float xv = beam_key_x(row_key[w][lane]), M = row_m[w];
                // x == M first: M may be infinite
                row_s[w][lane] = (double)score + ((xv == M ? 0.0 : (double)xv - (double)M) - row_lg[w]);
            }
            const double v = row_s[w][lane] + 0.0;  // -inf and NaN never win
            const unsigned long long u = (unsigned long long)__double_as_longlong(v);
            o = !(v > -INFINITY) ? 0ull : (u >> 63) ? ~u : (u | 0x8000000000000000ull);
        }
        row_o[w][lane] = o;
        if (lane < 2) row_o[w][BS_MAX_OUT + lane] = 0ull;
    }
    __syncthreads();
    if (warp) return;
    // Lane w holds the head of beam w's list; larger s first, then the lower beam.
    const unsigned long long* mine_o = row_o[lane < a.W ? lane : 0];
    unsigned long long key = lane < a.W ? mine_o[0] : 0ull, after = lane < a.W ? mine_o[1] : 0ull;
    int pos = 0, mine = -1;  // mine: the winner (beam, place) of output `lane`
    for (int j = 0; j < K; ++j) {
        const unsigned who = warp_best(key);
        if (!who) break;
        const int win = __ffs(who) - 1, wp = __shfl_sync(FULL_MASK, pos, win);
        if (lane == j) mine = win * BS_MAX_OUT + wp;
        if (lane == win) {
            key = after;
            ++pos;
            after = mine_o[min(pos + 1, BS_MAX_OUT + 1)];
        }
    }
    if (lane < K) {
        const int o = g * K + lane;
        if (mine < 0) {
            a.parents[o] = -1;
            a.tokens[o] = -1;
            a.scores_out[o] = -INFINITY;
            if (a.done_out) a.done_out[o] = 0;
        } else {
            const int bw = mine / BS_MAX_OUT, tok = beam_key_i(row_key[bw][mine % BS_MAX_OUT]);
            a.parents[o] = bw;
            a.tokens[o] = tok;
            a.scores_out[o] = (float)row_s[bw][mine % BS_MAX_OUT];
            if (a.done_out) a.done_out[o] = tok == a.eos || (a.done && a.done[r + bw]) ? 1 : 0;
        }
    }
}

constexpr int BS_MERGE_SMEM = KD_BEAM_MAX_BEAMS * BS_MAX_SEGS * BS_MAX_OUT * 8;
cudaError_t beam_init_attributes() {
    cudaError_t e = cudaSuccess;
    for (const void* f : {(const void*)beam_scan_kernel<true>, (const void*)beam_scan_kernel<false>,
                          (const void*)beam_merge_kernel})
        if ((e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout,
                                      cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
            return e;
    return cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BS_MERGE_SMEM);
}

}  // namespace kd

extern "C" {

size_t kd_beam_workspace_bytes(int32_t n_groups, int32_t n_beams, int32_t V, int32_t n_out) {
    if (n_groups < 1 || n_beams < 1 || V < 1 || n_out < 1) return 0;
    const size_t nblk = ((size_t)V + kd::BS_BLOCK - 1) / kd::BS_BLOCK;
    return 256 + (size_t)n_groups * n_beams * nblk * (8 + 8 * (size_t)n_out);
}

kd_status kd_beam_select(const float* logits, int64_t ld, int32_t n_groups, int32_t n_beams, int32_t V,
                         const float* scores, const int32_t* done, int32_t eos, int32_t n_out, int32_t* parents_out,
                         int32_t* tokens_out, float* scores_out, int32_t* done_out, void* workspace,
                         size_t workspace_bytes, kd_stream stream) {
    using namespace kd;
    if (!logits || !parents_out || !tokens_out || !scores_out || !workspace)
        return failf(KD_ERR_INVALID_ARG, "kd_beam_select: null argument");
    if (n_groups < 1 || n_beams < 1 || n_beams > KD_BEAM_MAX_BEAMS || (int64_t)n_groups * n_beams > 65535)
        return failf(KD_ERR_BATCH, "kd_beam_select: %d groups of %d beams (at most %d beams, 65535 rows)", n_groups,
                     n_beams, KD_BEAM_MAX_BEAMS);
    if (n_out < 1 || n_out > KD_BEAM_MAX_OUT)
        return failf(KD_ERR_INVALID_ARG, "kd_beam_select: n_out=%d outside [1, %d]", n_out, KD_BEAM_MAX_OUT);
    if (V < 1 || ld < V) return failf(KD_ERR_INVALID_ARG, "kd_beam_select: V=%d, ld=%lld", V, (long long)ld);
    if (V > KD_BEAM_MAX_VOCAB)
        return failf(KD_ERR_UNSUPPORTED, "kd_beam_select: V=%d exceeds %d", V, KD_BEAM_MAX_VOCAB);
    if (eos >= V || (done && eos < 0))
        return failf(KD_ERR_INVALID_ARG, "kd_beam_select: eos=%d (finished beams need one in [0, %d))", eos, V);
    if (workspace_bytes < kd_beam_workspace_bytes(n_groups, n_beams, V, n_out))
        return failf(KD_ERR_INVALID_ARG, "kd_beam_select: workspace too small");
    if ((reinterpret_cast<uintptr_t>(workspace) & 15) || (reinterpret_cast<uintptr_t>(logits) & 3))
        return failf(KD_ERR_INVALID_ARG, "kd_beam_select: the workspace must be 16-byte aligned, logits 4-byte");
    BeamArgs a{};
    const int rows = n_groups * n_beams;
    a.logits = logits;
    a.ld = ld;
    a.V = V;
    a.W = n_beams;
    a.K = n_out;
    a.nblk = (V + BS_BLOCK - 1) / BS_BLOCK;
    a.scores = scores;
    a.done = done;
    a.eos = eos < 0 ? -1 : eos;
    a.parents = parents_out;
    a.tokens = tokens_out;
    a.scores_out = scores_out;
    a.done_out = done_out;
    cudaStream_t s = (cudaStream_t)stream;
    int dev = 0;
    KD_TRY(cudaGetDevice(&dev));
    KD_TRY(ensure_device_attributes(dev));
    // Segments: as many per row as fill the GPU with four CTAs on every SM, at most
    // 32 (the merge's lanes) and one block each; more rows than that, one segment.
    int sms = 0;
    KD_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    int nseg = 4 * sms / rows;
    nseg = nseg < 1 ? 1 : nseg > BS_MAX_SEGS ? BS_MAX_SEGS : nseg;
    a.seg_blocks = (a.nblk + nseg - 1) / nseg;
    a.nseg = (a.nblk + a.seg_blocks - 1) / a.seg_blocks;
    a.keys = reinterpret_cast<unsigned long long*>(workspace);
    a.part = reinterpret_cast<float2*>(a.keys + (size_t)rows * a.nseg * n_out);
    const dim3 grid(a.nseg, rows);
    if (ld % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0)
        beam_scan_kernel<true><<<grid, BS_THREADS, 0, s>>>(a);
    else
        beam_scan_kernel<false><<<grid, BS_THREADS, 0, s>>>(a);
    KD_TRY(cudaGetLastError());
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(n_groups);
    cfg.blockDim = dim3(64 * n_beams);
    cfg.dynamicSmemBytes = (size_t)n_beams * a.nseg * n_out * 8;
    cfg.stream = s;
    KD_TRY(cudaLaunchKernelEx(&cfg, beam_merge_kernel, a));
    return KD_OK;
}

}  // extern "C"
