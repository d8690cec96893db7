// kd_beam.cu -- beam selection: each prompt's best continuations over its beams
// and the vocabulary, straight from the step's logits.
//
// Beam w of a group has the cumulative log probability score_w; continuing it
// with token v gives
//   s(w, v) = score_w + x_wv - L_w,   L_w = log sum_u e^{x_wu},
// and the group's n_out best pairs are wanted, larger s first, then lower w, then
// lower v.  Within a row the order is the logits' own, so one pass over the
// logits does everything that touches all of them: a block takes 4096 logits of
// one row, leaves (m, sum e^{x-m}) and its n_out best logits, sorted.  A second
// kernel, one CTA per group and one warp per beam, forms L_w, merges the row's
// lists, and merges the rows by s.
//
// s decides between rows, where two candidates can lie as close as fp32 rounds:
// L_w's last steps and s are fp64 (a handful of operations per row), the sums of
// exponentials fp32 inside a warp and exact 64-bit fixed point across blocks, so
// the order of blocks never matters and a row's result does not depend on the
// rest of the batch.
#include <cuda_runtime.h>

#include <cmath>

#include "kd_device.cuh"
#include "kd_host.h"

namespace kd {

constexpr int BS_THREADS = 256;
constexpr int BS_WARPS = BS_THREADS / 32;
constexpr int BS_VPT = 16;                      // logits per thread
constexpr int BS_BLOCK = BS_THREADS * BS_VPT;   // logits per block
constexpr int BS_MAX_BLOCKS = 128;              // vocabulary up to 524288
constexpr int BS_MAX_OUT = 32;
constexpr int BS_CAP = 512;                     // candidates a block ranks at once
constexpr int BS_AHEAD = 4;                     // list entries the merge stages in shared memory
static_assert(KD_BEAM_MAX_VOCAB == BS_BLOCK * BS_MAX_BLOCKS && KD_BEAM_MAX_OUT == BS_MAX_OUT, "kd.h limits");

// (x, index) as a 64-bit key whose unsigned order is: larger x, then lower index
// (-0 equals +0).  0 is no candidate.
__device__ __forceinline__ unsigned long long beam_key(float x, int i) {
    const unsigned u = __float_as_uint(x + 0.0f);
    const unsigned ord = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((unsigned long long)ord << 32) | (unsigned)~i;
}
__device__ __forceinline__ float beam_key_x(unsigned long long k) {
    const unsigned ord = (unsigned)(k >> 32);
    return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7fffffffu) : ~ord);
}
__device__ __forceinline__ int beam_key_i(unsigned long long k) { return (int)~(unsigned)k; }

// Warp maximum / minimum of 64-bit keys, high words first.
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long k) {
    const unsigned hi = (unsigned)(k >> 32), mh = __reduce_max_sync(FULL_MASK, hi);
    const unsigned ml = __reduce_max_sync(FULL_MASK, hi == mh ? (unsigned)k : 0u);
    return ((unsigned long long)mh << 32) | ml;
}
__device__ __forceinline__ unsigned long long warp_min_u64(unsigned long long k) {
    const unsigned hi = (unsigned)(k >> 32), mh = __reduce_min_sync(FULL_MASK, hi);
    const unsigned ml = __reduce_min_sync(FULL_MASK, hi == mh ? (unsigned)k : 0xffffffffu);
    return ((unsigned long long)mh << 32) | ml;
}

// A beam's row is read only if the beam can continue: not finished, score > -inf (a NaN score is dead too).
__device__ __forceinline__ bool beam_live(const float* scores, const int* done, int r) {
    return (!scores || scores[r] > -INFINITY) && !(done && done[r]);
}

struct BeamArgs {
    const float* logits;  // [rows][ld]
    long ld;
    int V, W, K, nblk;    // vocabulary, beams per group, candidates kept, blocks per row
    const float* scores;  // [rows], or nullptr (zeros)
    const int* done;      // [rows], or nullptr
    int eos;
    float2* part;              // [rows][nblk] (m, sum e^{x - m})
    unsigned long long* keys;  // [rows][nblk][K] sorted, 0-padded
    int *parents, *tokens, *done_out;
    float* scores_out;
};

__global__ void __launch_bounds__(BS_THREADS) beam_scan_kernel(const BeamArgs a) {
    __shared__ unsigned long long cand[BS_CAP];
    __shared__ unsigned long long subset[32];
    __shared__ float wm[BS_WARPS], wsum[BS_WARPS];
    __shared__ int cnt;
    pdl_launch_dependents();
    const int r = blockIdx.y, blk = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    if (!beam_live(a.scores, a.done, r)) return;
    const float* p = a.logits + (size_t)r * a.ld + (size_t)blk * BS_BLOCK;
    const int n = min(BS_BLOCK, a.V - blk * BS_BLOCK);
    float x[BS_VPT];
#pragma unroll
    for (int i = 0; i < BS_VPT; ++i) x[i] = i * BS_THREADS + t < n ? __ldg(p + i * BS_THREADS + t) : -INFINITY;
    // NaN counts as -inf; the thread's largest value and its first place
    float m = -INFINITY;
    int at = 0;
#pragma unroll
    for (int i = 0; i < BS_VPT; ++i) {
        x[i] = fmaxf(x[i], -INFINITY);
        if (x[i] > m) {
            m = x[i];
            at = i;
        }
    }
    float s = 0.0f;
    if (m == INFINITY) {  // x - m taken as 0 where x == m
#pragma unroll
        for (int i = 0; i < BS_VPT; ++i) s += x[i] == INFINITY ? 1.0f : 0.0f;
    } else if (m > -INFINITY) {
#pragma unroll
        for (int i = 0; i < BS_VPT; ++i) s += exp2f((x[i] - m) * 1.44269504088896341f);
    }
    const unsigned long long best = m > -INFINITY ? beam_key(m, blk * BS_BLOCK + at * BS_THREADS + t) : 0ull;
    // The warp's (m, sum), and the largest key of each subset of 8 threads: 32
    // subsets, so at least 32 logits are no less than the smallest of these.
    float mw = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mw = fmaxf(mw, __shfl_xor_sync(FULL_MASK, mw, o));
    s = m == mw ? s : s * expf(m - mw);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(FULL_MASK, s, o);
    unsigned long long k8 = best;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) k8 = max(k8, __shfl_xor_sync(FULL_MASK, k8, o));
    if ((lane & 7) == 0) subset[t >> 3] = k8;
    if (lane == 0) {
        wm[warp] = mw;
        wsum[warp] = mw > -INFINITY ? s : 0.0f;
    }
    if (t == 0) cnt = 0;
    __syncthreads();
    const unsigned long long thr = warp_min_u64(subset[lane]);
    if (t == 0) {
        float mb = wm[0], sb = 0.0f;
        for (int w = 1; w < BS_WARPS; ++w) mb = fmaxf(mb, wm[w]);
        for (int w = 0; w < BS_WARPS; ++w) sb += wm[w] == mb ? wsum[w] : wsum[w] * expf(wm[w] - mb);
        a.part[(size_t)r * a.nblk + blk] = make_float2(mb, mb > -INFINITY ? sb : 0.0f);
    }
    const float tv = thr ? beam_key_x(thr) : -INFINITY;
#pragma unroll
    for (int i = 0; i < BS_VPT; ++i)
        if (x[i] >= tv && x[i] > -INFINITY) {
            const unsigned long long k = beam_key(x[i], blk * BS_BLOCK + i * BS_THREADS + t);
            if (k >= thr) {
                const int j = atomicAdd(&cnt, 1);
                if (j < BS_CAP) cand[j] = k;
            }
        }
    __syncthreads();
    unsigned long long* out = a.keys + ((size_t)r * a.nblk + blk) * a.K;
    const int c = cnt;
    if (c <= BS_CAP) {
        for (int j = t; j < c; j += BS_THREADS) {
            const unsigned long long k = cand[j];
            int rank = 0;
            for (int i = 0; i < c; ++i) rank += cand[i] > k ? 1 : 0;
            if (rank < a.K) out[rank] = k;
        }
        for (int j = c + t; j < a.K; j += BS_THREADS) out[j] = 0ull;
    } else {  // too many to rank (a subset without a value): one block maximum per candidate
        unsigned long long last = ~0ull;
        for (int j = 0; j < a.K; ++j) {
            unsigned long long b = 0ull;
#pragma unroll
            for (int i = 0; i < BS_VPT; ++i)
                if (x[i] > -INFINITY) {
                    const unsigned long long k = beam_key(x[i], blk * BS_BLOCK + i * BS_THREADS + t);
                    if (k < last) b = max(b, k);
                }
            b = warp_max_u64(b);
            __syncthreads();
            if (lane == 0) subset[warp] = b;
            __syncthreads();
            last = warp_max_u64(lane < BS_WARPS ? subset[lane] : 0ull);
            if (t == 0) out[j] = last;
        }
    }
}

// One CTA per group, one warp per beam.
__global__ void __launch_bounds__(32 * KD_BEAM_MAX_BEAMS) beam_merge_kernel(const BeamArgs a) {
    extern __shared__ unsigned long long staged[];  // [W][nblk][ahead] the lists' first entries
    __shared__ double row_s[KD_BEAM_MAX_BEAMS][BS_MAX_OUT];
    __shared__ int row_v[KD_BEAM_MAX_BEAMS][BS_MAX_OUT];
    __shared__ int row_n[KD_BEAM_MAX_BEAMS];
    pdl_wait();
    const int g = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5, r = g * a.W + w;
    const int ahead = min(a.K, BS_AHEAD);
    const float score = a.scores ? a.scores[r] : 0.0f;
    if (!beam_live(a.scores, a.done, r)) {
        if (lane == 0) {  // a finished beam stands for itself; a dead one offers nothing
            const bool fin = a.done && a.done[r] && score > -INFINITY;
            row_n[w] = fin ? 1 : 0;
            row_s[w][0] = (double)score;
            row_v[w][0] = a.eos;
        }
    } else {
        const unsigned long long* lists = a.keys + (size_t)r * a.nblk * a.K;
        unsigned long long* st = staged + (size_t)w * a.nblk * ahead;
        for (int i = lane; i < a.nblk * ahead; i += 32) st[i] = __ldcg(lists + (size_t)(i / ahead) * a.K + i % ahead);
        // L = M + log sum_b s_b e^{m_b - M}; the sum in units of 2^-40 (each term at most 4096, the largest at least 1)
        const float2* part = a.part + (size_t)r * a.nblk;
        float M = -INFINITY;
        for (int b = lane; b < a.nblk; b += 32) M = fmaxf(M, __ldcg(part + b).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
        long long sum = 0;
        for (int b = lane; b < a.nblk; b += 32) {
            const float2 ms = __ldcg(part + b);
            const float f = ms.x == M ? ms.y : ms.y * expf(ms.x - M);
            sum += __float2ll_rn(f * 0x1p40f);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
        const double lg = log((double)sum * 0x1p-40);
        __syncwarp();
        // The row's K best: lane l holds the heads of lists l, l + 32, ...
        unsigned long long head[BS_MAX_BLOCKS / 32];
        int next[BS_MAX_BLOCKS / 32];
#pragma unroll
        for (int q = 0; q < BS_MAX_BLOCKS / 32; ++q) {
            const int b = lane + 32 * q;
            head[q] = b < a.nblk ? st[b * ahead] : 0ull;
            next[q] = 1;
        }
        int n = 0;
        for (; n < a.K; ++n) {
            unsigned long long best = head[0];
#pragma unroll
            for (int q = 1; q < BS_MAX_BLOCKS / 32; ++q) best = max(best, head[q]);
            const unsigned long long k = warp_max_u64(best);
            if (!k) break;
#pragma unroll
            for (int q = 0; q < BS_MAX_BLOCKS / 32; ++q)
                if (head[q] == k) {
                    const int b = lane + 32 * q, e = next[q]++;
                    head[q] = e >= a.K ? 0ull : e < ahead ? st[b * ahead + e] : __ldcg(lists + (size_t)b * a.K + e);
                }
            if (lane == 0) {
                const float xv = beam_key_x(k);
                // x == M first: M may be +inf
                row_s[w][n] = (double)score + ((xv == M ? 0.0 : (double)xv - (double)M) - lg);
                row_v[w][n] = beam_key_i(k);
            }
        }
        if (lane == 0) row_n[w] = n;
    }
    __syncthreads();
    if (w) return;
    // The group's K best: lane w holds the head of beam w's list (larger s, then the lower beam).
    const int cnt = lane < a.W ? row_n[lane] : 0;
    int pos = 0;
    double hs = cnt ? row_s[lane][0] : -INFINITY;
    for (int j = 0; j < a.K; ++j) {
        const double v = hs + 0.0;
        const unsigned long long u = (unsigned long long)__double_as_longlong(v);
        // -inf and NaN never win; an order-preserving key of s otherwise
        const unsigned long long key = !(v > -INFINITY) ? 0ull : (u >> 63) ? ~u : (u | 0x8000000000000000ull);
        const unsigned long long k = warp_max_u64(key);
        const int o = g * a.K + j;
        if (!k) {
            if (lane == 0) {
                a.parents[o] = -1;
                a.tokens[o] = -1;
                a.scores_out[o] = -INFINITY;
                if (a.done_out) a.done_out[o] = 0;
            }
            continue;
        }
        const int win = __ffs(__ballot_sync(FULL_MASK, key == k)) - 1;
        if (lane == win) {
            const int tok = row_v[lane][pos];
            a.parents[o] = lane;
            a.tokens[o] = tok;
            a.scores_out[o] = (float)hs;
            if (a.done_out) a.done_out[o] = (a.eos >= 0 && tok == a.eos) || (a.done && a.done[r + lane]) ? 1 : 0;
            hs = ++pos < cnt ? row_s[lane][pos] : -INFINITY;
        }
    }
}

constexpr int BS_MERGE_SMEM = KD_BEAM_MAX_BEAMS * BS_MAX_BLOCKS * BS_AHEAD * 8;
cudaError_t beam_init_attributes() {
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
    a.keys = reinterpret_cast<unsigned long long*>(workspace);
    a.part = reinterpret_cast<float2*>(a.keys + (size_t)rows * a.nblk * n_out);
    a.parents = parents_out;
    a.tokens = tokens_out;
    a.scores_out = scores_out;
    a.done_out = done_out;
    cudaStream_t s = (cudaStream_t)stream;
    int dev = 0;
    KD_TRY(cudaGetDevice(&dev));
    KD_TRY(ensure_device_attributes(dev));
    beam_scan_kernel<<<dim3(a.nblk, rows), BS_THREADS, 0, s>>>(a);
    KD_TRY(cudaGetLastError());
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(n_groups);
    cfg.blockDim = dim3(32 * n_beams);
    cfg.dynamicSmemBytes = (size_t)n_beams * a.nblk * (n_out < BS_AHEAD ? n_out : BS_AHEAD) * 8;
    cfg.stream = s;
    KD_TRY(cudaLaunchKernelEx(&cfg, beam_merge_kernel, a));
    return KD_OK;
}

}  // extern "C"
