// kd_beam.cu -- beam selection: each prompt's best continuations over its beams
// and the vocabulary, straight from the step's logits.
//
// Beam w of a group has the cumulative log probability score_w; continuing it
// with token v gives
//   s(w, v) = score_w + x_wv - L_w,   L_w = log sum_u e^{x_wu},
// and the group's K best pairs are wanted, larger s first, then lower w, then
// lower v.  Within a row the order is the logits' own, so one pass over the
// logits does everything that touches all of them: a CTA walks a segment of one
// row 4096 logits at a time, and leaves (m, sum e^{x-m}) of every block (one or two
// such steps) and the segment's K best logits, sorted.  A second kernel, one CTA per
// group, forms L_w, merges each row's lists, and merges the rows by s.
//
// The selection costs next to nothing once K candidates are known: a block whose
// largest logit does not exceed the K-th best so far is passed over, so a random
// row brings about K ln(blocks) late candidates.  The first block's are found
// through the maxima of 32 or 64 subsets of it: the K-th largest of them bounds
// the K-th largest logit from below, and few logits lie above it (K = 4: 4.3 of
// 4096 on average, 8: 9, 32: 45).  The same of the 4, 16 and 64 blocks seen renews the
// bound; the warps keep their candidates apart to the end.
//
// s decides between rows, where two candidates can lie as close as fp32 rounds:
// L_w's last steps and s are pairs of fp32 whose sum carries about 48 bits (fp64
// instructions are so slow here that three of them per candidate took 20000
// cycles of a CTA).  The sums of exponentials are fp32 inside a block, in an order
// that depends on nothing but the block, and exact 64-bit fixed point across
// blocks.  So a row's result does not depend on the segments, hence not on the
// rest of the batch.
//
// What bounds it (device time of both kernels): 512 rows of 128256 logits 45.5 us, 5.8
// TB/s; 256 rows 28.2 us, 4.7 TB/s, where a CTA's 16 steps of about 0.9 us (the copies'
// latency, 15 dependent operations and the shared pipes) do not overlap with another
// CTA's as well as with four; 4 rows of 32000, 5.9 us: launch, one load's latency, one
// block's candidates, the merge.
#include <cuda_runtime.h>

#include <cmath>

#include "kd_device.cuh"
#include "kd_host.h"

namespace kd {

constexpr int BS_THREADS = 256;
constexpr int BS_WARPS = BS_THREADS / 32;
constexpr int BS_VPT = 16;                      // logits per thread and step
constexpr int BS_STEP = BS_THREADS * BS_VPT;    // logits per step
// Steps per block, the unit that sums are kept for: two where rows are long (a
// block's reduction costs a quarter of a step).  By the vocabulary alone, so that
// a row's sums do not depend on the batch.
constexpr int beam_block_shift(int V) { return V > 65536 ? 1 : 0; }
constexpr int BS_MAX_BLOCKS = 64;               // vocabulary up to 524288
constexpr int BS_MAX_SEGS = 32;                 // segments (lists) per row: one per lane of the merge
constexpr int BS_MAX_OUT = 32;
constexpr int BS_CAP = 128;                     // a warp's candidates between cuts to the K best
// Short lists are merged by counting, for each candidate, those above it: few keys wait less
// so than for the merge networks' exchanges (4 x 128256, best 4: 6.4 us against 7.6; 8 x 151936,
// best 8: 8.7, 10.1; 48 x 32003, best 32: 11.9, 13.5).  Networks where more keys would be left:
// 8 rows of 8 in the merge 14.5 us counted, 14.0 by networks; 8 lists of 32 a row 13.0, 11.9.
constexpr int BS_COUNT_OUT = 128;  // candidates of a segment, by a CTA
constexpr int BS_COUNT_KEYS = 64;  // keys of a row's segments, by a warp
constexpr int BS_COUNT_PICK = 16;  // best of more keys than those
constexpr int BS_COUNT_ROWS = 64;  // rows x candidates x (rows / 4, the warps that share an issue slot)
constexpr int BS_STAGES = 2;                    // steps in flight behind the one being worked on
static_assert(KD_BEAM_MAX_VOCAB == (BS_STEP << beam_block_shift(KD_BEAM_MAX_VOCAB)) * BS_MAX_BLOCKS && KD_BEAM_MAX_OUT == BS_MAX_OUT, "kd.h limits");

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

// The 32 largest of two descending lists held a key per lane, descending: the larger
// of a[i] and b[31 - i] are those 32, a bitonic sequence that five exchanges sort.
__device__ __forceinline__ unsigned long long warp_merge(unsigned long long a, unsigned long long b, int lane) {
    unsigned long long c = max(a, __shfl_sync(FULL_MASK, b, 31 - lane));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long p = __shfl_xor_sync(FULL_MASK, c, o);
        c = (lane & o) ? min(c, p) : max(c, p);
    }
    return c;
}
// The 32 largest of the first n of eight lists (the others empty), merged in a tree:
// merges of one level overlap.
__device__ __forceinline__ unsigned long long warp_merge8(unsigned long long (&v)[8], int n, int lane) {
#pragma unroll
    for (int h = 4; h > 0; h >>= 1)
        if (n > h) {
#pragma unroll
            for (int i = 0; i < h; ++i) v[i] = warp_merge(v[i], v[i + h], lane);
        }
    return v[0];
}

// ---- pairs of fp32: hi + lo, hi = fp32(hi + lo) ---------------------------------
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {  // a + b exactly (Knuth)
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// log(sum 2^-40) for 2^40 <= sum < 2^63, within 3e-11.  sum 2^-40 = 2^n m, m in
// [1, 2) in two parts; m c = 1 + u with an 8-bit c near 1 / m from the table, so
// |u| < 1/59 (0.01685 at most): log = n log 2 - log c + u - u^2/2 + ... - u^6/6, whose
// next term is below 6e-14.  A table-driven logarithm (Tang, 1990).
__device__ const float LOG_TAB[32][3] = {  // c, and -log c in two parts
    {0.984375f, 1.574835740e-02f, -4.321589475e-10f}, {0.95703125f, 4.391923547e-02f, -1.533075222e-09f},
    {0.92578125f, 7.711730152e-02f, 1.820745776e-09f}, {0.90234375f, 1.027597338e-01f, 1.616492495e-10f},
    {0.875f, 1.335313916e-01f, 1.003886640e-09f}, {0.8515625f, 1.606823802e-01f, 1.491041068e-09f},
    {0.83203125f, 1.838852763e-01f, 2.452540837e-09f}, {0.80859375f, 2.124586552e-01f, -4.023958056e-09f},
    {0.7890625f, 2.369097471e-01f, -4.536054865e-11f}, {0.76953125f, 2.619737089e-01f, 6.873547065e-09f},
    {0.75390625f, 2.824872434e-01f, 1.216075152e-08f}, {0.734375f, 3.087354898e-01f, -8.195662815e-09f},
    {0.71875f, 3.302416801e-01f, 6.725313195e-09f}, {0.703125f, 3.522205949e-01f, -1.293612995e-09f},
    {0.6875f, 3.746934533e-01f, -3.870509246e-09f}, {0.671875f, 3.976829648e-01f, 2.864321225e-09f},
    {0.66015625f, 4.152787328e-01f, -3.220152811e-09f}, {0.64453125f, 4.392319620e-01f, 8.613421087e-09f},
    {0.6328125f, 4.575811028e-01f, 6.399125230e-09f}, {0.62109375f, 4.762732387e-01f, 3.600425957e-09f},
    {0.609375f, 4.953214228e-01f, 1.441470232e-08f}, {0.59765625f, 5.147395134e-01f, 9.689910208e-09f},
    {0.5859375f, 5.345421433e-01f, 7.038427619e-09f}, {0.578125f, 5.479651690e-01f, 1.762505475e-09f},
    {0.56640625f, 5.684437156e-01f, -1.351336909e-08f}, {0.5546875f, 5.893504024e-01f, -1.547689266e-08f},
    {0.546875f, 6.035349965e-01f, 2.536070554e-08f}, {0.5390625f, 6.179237366e-01f, 2.275009159e-08f},
    {0.52734375f, 6.399026513e-01f, 1.473116562e-08f}, {0.51953125f, 6.548283100e-01f, 6.244991191e-09f},
    {0.51171875f, 6.699801087e-01f, 1.254046555e-08f}, {0.50390625f, 6.853650212e-01f, 1.888910006e-08f}
};
struct LogEntry {  // an entry per lane, loaded ahead of the sum
    float c, hi, lo;
};
__device__ __forceinline__ LogEntry log_entry(int lane) { return {LOG_TAB[lane][0], LOG_TAB[lane][1], LOG_TAB[lane][2]}; }
__device__ __forceinline__ Pair pair_log(unsigned long long sum, const LogEntry& tab) {  // sum the same in all lanes
    const int k = 63 - __clzll((long long)sum);
    const unsigned long long m = sum << (63 - k);
    const unsigned top = (unsigned)(m >> 40);  // 24 bits
    const float mh = (float)top * 0x1p-23f, ml = (float)((unsigned)(m >> 16) & 0xffffffu) * 0x1p-47f;
    const int at = (top >> 18) & 31u;
    const float c = __shfl_sync(FULL_MASK, tab.c, at), chi = __shfl_sync(FULL_MASK, tab.hi, at),
                clo = __shfl_sync(FULL_MASK, tab.lo, at), p = __fmul_rn(mh, c);
    const float u0 = __fsub_rn(p, 1.0f), u1 = __fmaf_rn(ml, c, __fmaf_rn(mh, c, -p)), u = __fadd_rn(u0, u1);
    float q = __fmaf_rn(u, -1.0f / 6, 1.0f / 5);
    q = __fmaf_rn(u, q, -0.25f);
    q = __fmaf_rn(u, q, 1.0f / 3);
    q = __fmaf_rn(u, q, -0.5f);
    q = __fmul_rn(__fmul_rn(u, u), q);
    const float n = (float)(k - 40);  // log 2 in two parts, the first of 16 bits: its product with n is exact
    const Pair a = two_sum(__fmul_rn(n, 0.693145751953125f), chi), b = two_sum(a.hi, u0);
    const float lo = __fadd_rn(__fadd_rn(__fadd_rn(__fmaf_rn(n, 1.428606765330187e-06f, clo), u1), q),
                               __fadd_rn(a.lo, b.lo));
    return two_sum(b.hi, lo);
}
// x + y of pairs; not finite: the sum alone.
__device__ __forceinline__ Pair pair_add(Pair x, Pair y) {
    const Pair s = two_sum(x.hi, y.hi);
    if (!(fabsf(s.hi) < INFINITY)) return {s.hi, 0.0f};
    return two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(x.lo, y.lo)));
}
// Order-preserving key of a pair; 0 for -inf and NaN.
__device__ __forceinline__ unsigned long long pair_key(Pair s) {
    return s.hi > -INFINITY ? ((unsigned long long)beam_ord(s.hi) << 32) | beam_ord(s.lo) : 0ull;
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
    int block_shift;      // log2 of the steps per block
    const float* scores;  // [rows], or nullptr (zeros)
    const int* done;      // [rows], or nullptr
    int eos;
    float2* part;              // [rows][nblk] (m, sum e^{x - m})
    unsigned long long* keys;  // [rows][nseg][K] sorted, 0-padded
    int *parents, *tokens, *done_out;
    float* scores_out;
};

// A step's logits on their way through shared memory: thread t reads elements 4t .. 4t + 3 of
// each quarter.  Rows on 16-byte boundaries (ALIGNED) are copied by 16 bytes, by the threads that
// read them, so none waits for another.  Others, which start `off` elements past one: where rows
// are long (SHIFTED), a warp's 128 elements of a quarter are in 33 aligned pieces, which its
// lanes copy for one another; else (SINGLY) an element at a time, which is less code to run once
// (144 rows of 164879 33 us against 36; 76 of 645 6.2, 5.7).  Only what lies in the row is read.
enum BeamRows : int { BEAM_ALIGNED, BEAM_SHIFTED, BEAM_SINGLY };
constexpr int BS_SHIFTED_VOCAB = 32768;
constexpr int BS_PIECES = 33 * 4;  // floats of a warp's quarter in pieces
template <int ROWS>
constexpr int BS_QUARTER = ROWS == BEAM_SHIFTED ? BS_WARPS * BS_PIECES : 4 * BS_THREADS;
template <int ROWS>
constexpr int BS_STAGE = BS_VPT / 4 * BS_QUARTER<ROWS>;
// Where a thread's elements of the first quarter are in a stage (SHIFTED: `off` further).
template <int ROWS>
__device__ __forceinline__ int beam_place(int t) {
    return ROWS == BEAM_SHIFTED ? (t >> 5) * BS_PIECES + 4 * (t & 31) : 4 * t;
}
__device__ __forceinline__ void beam_copy4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void beam_copy16(uint32_t dst, const float* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int ROWS>
__device__ __forceinline__ void beam_fetch(float* stage, const float* row, int e0, int V, int off, int t) {
    constexpr bool SHIFTED = ROWS == BEAM_SHIFTED;
    const int lane = t & 31, warp = t >> 5;
    const uint32_t dst = smem_u32(stage + beam_place<ROWS>(t));
    if (ROWS != BEAM_SINGLY && e0 + BS_STEP + (SHIFTED ? 4 : 0) <= V) {
        const int e = e0 + 4 * t - off;
        if (!SHIFTED || e >= 0)
            beam_copy16(dst, row + e);
        else  // the row's first piece
            for (int j = off; j < 4; ++j) beam_copy4(dst + 4 * j, row + e + j);
#pragma unroll
        for (int i = 1; i < BS_VPT / 4; ++i) beam_copy16(dst + 4 * i * BS_QUARTER<ROWS>, row + e + i * 4 * BS_THREADS);
        if (SHIFTED && lane < BS_VPT / 4)  // the 33rd pieces, one per quarter
            beam_copy16(smem_u32(stage + lane * BS_QUARTER<ROWS> + warp * BS_PIECES + 128),
                        row + e0 + lane * 4 * BS_THREADS + 128 * (warp + 1) - off);
    } else {  // the row's end, an element at a time
        const int left = V - e0 - 4 * t;
        const float* p = row + e0 + 4 * t;
#pragma unroll
        for (int i = 0; i < BS_VPT; ++i) {
            const int o = (i >> 2) * 4 * BS_THREADS + (i & 3);
            if (o < left) beam_copy4(dst + 4 * ((i >> 2) * BS_QUARTER<ROWS> + (i & 3) + off), p + o);
        }
    }
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// At most 32 candidates of the warp, sorted and cut to the K best, then zeros up to 32; returns their number.
__device__ __forceinline__ int beam_sort(unsigned long long* buf, int n, int K, int lane) {
    __syncwarp();
    const unsigned long long k = lane < n ? buf[lane] : 0ull;
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += buf[j] > k ? 1 : 0;
    __syncwarp();
    const int c = min(n, K);
    if (lane < n) buf[rank] = k;
    __syncwarp();
    if (lane >= c) buf[lane] = 0ull;
    __syncwarp();
    return c;
}
// Any number of them.  Out of line: inlined at its call sites it made the kernel several times as
// long, and a CTA that passes through its code once waits for instructions more than for anything else.
__device__ __noinline__ int beam_cut(unsigned long long* buf, unsigned long long* best, int n, int K, int lane) {
    if (n <= 32) return beam_sort(buf, n, K, lane);
    __syncwarp();
    unsigned long long k[BS_CAP / 32];
    int rank[BS_CAP / 32] = {};
#pragma unroll
    for (int q = 0; q < BS_CAP / 32; ++q) k[q] = lane + 32 * q < n ? buf[lane + 32 * q] : 0ull;
    for (int j = 0; j < n; ++j) {
        const unsigned long long o = buf[j];
#pragma unroll
        for (int q = 0; q < BS_CAP / 32; ++q) rank[q] += o > k[q] ? 1 : 0;
    }
#pragma unroll
    for (int q = 0; q < BS_CAP / 32; ++q)
        if (k[q] && rank[q] < K) best[rank[q]] = k[q];
    __syncwarp();
    buf[lane] = lane < K ? best[lane] : 0ull;  // n > 32 >= K
    __syncwarp();
    return K;
}

// How many of the first n (even) keys of a list lie above k.
__device__ __forceinline__ int beam_above(const unsigned long long* list, int n, unsigned long long k) {
    int c = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 2) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(list + j);
        c += (o.x > k ? 1 : 0) + (o.y > k ? 1 : 0);
    }
    return c;
}

// Warp 0: the 32 best of the warps' lists (each sorted, 0-padded to 32).
__device__ __forceinline__ unsigned long long beam_merge_lists(const unsigned long long (*lists)[BS_CAP], int lane) {
    static_assert(BS_WARPS == 8, "merged in a tree of eight");
    unsigned long long v[8];
#pragma unroll
    for (int w = 0; w < 8; ++w) v[w] = lists[w][lane];
    return warp_merge8(v, 8, lane);
}

template <int ROWS>
__global__ void __launch_bounds__(BS_THREADS, 4) beam_scan_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ __align__(16) unsigned long long cand[BS_WARPS][BS_CAP];
    __shared__ __align__(16) unsigned long long best[BS_WARPS][BS_MAX_OUT];
    __shared__ int counts[BS_WARPS];
    __shared__ unsigned low[BS_WARPS];
    // [stages][BS_STEP] logits, then the blocks' sums by warp; off a 128-byte line the copies take 5% longer
    extern __shared__ __align__(128) float beam_smem[];
    __shared__ __align__(16) float subset[4][64];  // maxima by 8 or 4 threads of the blocks seen, at each renewal of the bound
    pdl_launch_dependents();
    const int r = blockIdx.y, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int K = a.K, c0 = blockIdx.x * a.seg_blocks, nc = min(a.seg_blocks, a.nblk - c0);  // the segment's blocks
    const int e_end = min(a.V, ((c0 + nc) << a.block_shift) * BS_STEP), e_begin = (c0 << a.block_shift) * BS_STEP;
    const int nb = (e_end - e_begin + BS_STEP - 1) / BS_STEP;  // its steps
    const float* row = a.logits + (size_t)r * a.ld;
    const int off = ROWS != BEAM_SHIFTED ? 0 : (int)(reinterpret_cast<uintptr_t>(row) >> 2 & 3);
    unsigned long long* buf = cand[warp];
    int cnt = 0;
    float thr = -INFINITY;  // K logits seen are no less: later equals lose to them (higher indices)
    float mrun = -INFINITY; // the thread's largest so far
    float mt = -INFINITY, st = 0.0f;  // the thread's (m, sum) of the block
    float2(*wpart)[BS_WARPS] = reinterpret_cast<float2(*)[BS_WARPS]>(beam_smem + BS_STAGES * BS_STAGE<ROWS>);
    auto fetch = [&](int b) {
        const int e0 = e_begin + b * BS_STEP;
        if (ROWS == BEAM_SHIFTED) __syncwarp();  // the stage is read
        if (b < nb) beam_fetch<ROWS>(beam_smem + (b % BS_STAGES) * BS_STAGE<ROWS>, row, e0, a.V, off, t);
        cp_async_commit();
    };
    pdl_wait();
    fetch(0);  // in flight while the beam's state is read
    if (!beam_live(a.scores, a.done, r)) {
        cp_async_wait<0>();
        return;
    }
#pragma unroll
    for (int b = 1; b < BS_STAGES; ++b) fetch(b);
    for (int b = 0; b < nb; ++b) {
        const int e0 = e_begin + b * BS_STEP;
        const float* stage = beam_smem + (b % BS_STAGES) * BS_STAGE<ROWS> + beam_place<ROWS>(t);
        float x[BS_VPT];
        cp_async_wait<BS_STAGES - 1>();
        if (ROWS == BEAM_SHIFTED) __syncwarp();
#pragma unroll
        for (int i = 0; i < BS_VPT / 4; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(stage + i * BS_QUARTER<ROWS>);
            x[4 * i] = v.x;
            x[4 * i + 1] = v.y;
            x[4 * i + 2] = v.z;
            x[4 * i + 3] = v.w;
        }
        if (ROWS == BEAM_SHIFTED && off) {
#pragma unroll
            for (int i = 0; i < BS_VPT / 4; ++i) {
                const float4 n = *reinterpret_cast<const float4*>(stage + i * BS_QUARTER<ROWS> + 4);
                float* y = x + 4 * i;
                if (off == 1) {
                    y[0] = y[1]; y[1] = y[2]; y[2] = y[3]; y[3] = n.x;
                } else if (off == 2) {
                    y[0] = y[2]; y[1] = y[3]; y[2] = n.x; y[3] = n.y;
                } else {
                    y[0] = y[3]; y[1] = n.x; y[2] = n.y; y[3] = n.z;
                }
            }
        }
        if (a.V - e0 < BS_STEP) {
            const int left = a.V - e0 - 4 * t;
#pragma unroll
            for (int i = 0; i < BS_VPT; ++i)
                if ((i >> 2) * 4 * BS_THREADS + (i & 3) >= left) x[i] = -INFINITY;
        }
        float m = x[0];
#pragma unroll
        for (int i = 1; i < BS_VPT; ++i) m = fmaxf(m, x[i]);
        // Candidates are logits >= lo: those above thr (the next value up).  A warp without
        // any is done with the stage once it holds the logits, and refills it at once.
        float lo = beam_unord(beam_ord(thr) + 1u);
        const bool renew = b == 0 || b == 3 || b == 15 || b == 63;
        const bool none = !renew && !__any_sync(FULL_MASK, m >= lo);
        if (none) fetch(b + BS_STAGES);
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
        {  // into the block's
            const float mn = fmaxf(mt, m);
            st = (mt == mn ? st : st * ex2((mt - mn) * LOG2E)) + (m == mn ? s : s * ex2((m - mn) * LOG2E));
            mt = mn;
        }
        const int c = b >> a.block_shift;
        if (b + 1 == nb || b + 1 == (c + 1) << a.block_shift) {  // the block is complete
            const float mw = beam_unord(__reduce_max_sync(FULL_MASK, beam_ord(mt)));
            st = mt == mw ? st : st * ex2((mt - mw) * LOG2E);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) st += __shfl_xor_sync(FULL_MASK, st, o);
            if (lane == 0) wpart[c][warp] = make_float2(mw, st);
            mt = -INFINITY;
            st = 0.0f;
        }

        mrun = fmaxf(mrun, m);
        if (none) continue;
        if (renew) {  // and no less than the K-th largest subset maximum of the blocks seen, this one included
            float* sub = subset[b == 0 ? 0 : b == 3 ? 1 : b == 15 ? 2 : 3];
            float m8 = mrun;
            m8 = fmaxf(m8, __shfl_xor_sync(FULL_MASK, m8, 1));
            m8 = fmaxf(m8, __shfl_xor_sync(FULL_MASK, m8, 2));
            // the least of those with fewer than K above them: at least K subsets reach it
            unsigned least = 0xffffffffu;
            if (K <= 12) {
                m8 = fmaxf(m8, __shfl_xor_sync(FULL_MASK, m8, 4));
                if ((lane & 7) == 0) sub[t >> 3] = m8;
                __syncthreads();
                const float v = sub[lane];
                int rank = 0;  // subsets with a larger maximum
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 o = *reinterpret_cast<const float4*>(sub + j);
                    rank += (o.x > v ? 1 : 0) + (o.y > v ? 1 : 0) + (o.z > v ? 1 : 0) + (o.w > v ? 1 : 0);
                }
                if (rank < K) least = beam_ord(v);
            } else {
                if ((lane & 3) == 0) sub[t >> 2] = m8;
                __syncthreads();
                // eight of the 64 per warp, four lanes each
                const float v = sub[8 * warp + (lane >> 2)];
                const float* part = sub + 16 * (lane & 3);
                int rank = 0;
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 o = *reinterpret_cast<const float4*>(part + j);
                    rank += (o.x > v ? 1 : 0) + (o.y > v ? 1 : 0) + (o.z > v ? 1 : 0) + (o.w > v ? 1 : 0);
                }
                rank += __shfl_xor_sync(FULL_MASK, rank, 1);
                rank += __shfl_xor_sync(FULL_MASK, rank, 2);
                const unsigned mine = __reduce_min_sync(FULL_MASK, rank < K ? beam_ord(v) : 0xffffffffu);
                if (lane == 0) low[warp] = mine;
                __syncthreads();
                least = low[lane & 7];
            }
            const float kth = beam_unord(__reduce_min_sync(FULL_MASK, least));
            lo = fmaxf(lo, kth);
            thr = fmaxf(thr, kth);
        }
        if (__any_sync(FULL_MASK, m >= lo)) {
            unsigned mine = 0;
#pragma unroll
            for (int i = 0; i < BS_VPT; ++i) mine |= x[i] >= lo ? 1u << i : 0u;
            int quarter = 0;
            for (unsigned bits = __reduce_or_sync(FULL_MASK, mine); bits; bits &= bits - 1) {
                const int i = __ffs(bits) - 1;
                if (b == 0 && i >> 2 != quarter) {
                    quarter = i >> 2;
                    if (cnt >= K) {
                        // indices grow from quarter to quarter: what only equals a K-th best now loses to it
                        cnt = beam_cut(buf, best[warp], cnt, K, lane);
                        lo = fmaxf(lo, beam_unord(beam_ord(beam_key_x(buf[K - 1])) + 1u));
                    }
                }
                const float v = stage[(i >> 2) * BS_QUARTER<ROWS> + (i & 3) + off];
                const bool in = (mine >> i & 1u) && v >= lo;
                const unsigned who = __ballot_sync(FULL_MASK, in);
                if (cnt + __popc(who) > BS_CAP) cnt = beam_cut(buf, best[warp], cnt, K, lane);
                if (in) buf[cnt + __popc(who & ((1u << lane) - 1u))] = beam_key(v, e0 + (i >> 2) * 4 * BS_THREADS + (i & 3) + 4 * t);
                cnt += __popc(who);
            }
            if (cnt > K + 8) {
                cnt = beam_cut(buf, best[warp], cnt, K, lane);
                thr = fmaxf(thr, beam_key_x(buf[K - 1]));
            }
        }
        fetch(b + BS_STAGES);  // into the stage just read
    }
    // The segment's list: as long as few candidates are left, a thread each, which counts those above it.
    unsigned long long* list = a.keys + ((size_t)r * a.nseg + blockIdx.x) * K;
    if (lane == 0) counts[warp] = cnt;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < BS_WARPS; ++w) {
        if (w == warp) before = total;
        total += counts[w];
    }
    if (total <= BS_COUNT_OUT) {
        unsigned long long* all = best[0];
        static_assert(BS_COUNT_OUT < BS_WARPS * BS_MAX_OUT && BS_COUNT_OUT <= BS_THREADS, "they fit, a thread each");
        for (int i = lane; i < cnt; i += 32) all[before + i] = buf[i];
        if (t == 0) all[total] = 0ull;
        __syncthreads();
        if (t < total) {
            const unsigned long long k = all[t];
            const int rank = beam_above(all, (total + 1) & ~1, k);
            if (rank < K) list[rank] = k;
        } else if (t < K) {
            list[t] = 0ull;
        }
    } else {
        if (cnt > 32) cnt = beam_cut(buf, best[warp], cnt, K, lane);
        beam_sort(buf, cnt, K, lane);
        __syncthreads();
        if (warp == 0) {
            const unsigned long long k = beam_merge_lists(cand, lane);
            if (lane < K) list[lane] = k;
        }
    }
    const int b = t - BS_THREADS / 2;  // the blocks' sums, warps in order
    if (b >= 0 && b < nc) {
        float mb = -INFINITY, sb = 0.0f;
#pragma unroll
        for (int w = 0; w < BS_WARPS; ++w) mb = fmaxf(mb, wpart[b][w].x);
#pragma unroll
        for (int w = 0; w < BS_WARPS; ++w) {
            const float2 p = wpart[b][w];
            sb += p.x == mb ? p.y : p.y * ex2((p.x - mb) * LOG2E);
        }
        a.part[(size_t)r * a.nblk + c0 + b] = make_float2(mb, mb > -INFINITY ? sb : 0.0f);
    }
}
static_assert(BS_THREADS / 2 >= BS_MAX_BLOCKS, "a thread per block of a segment");

// One CTA per group: warps 0 .. W - 1 merge the rows' lists while warps W .. 2W - 1
// form the rows' log sums; then the rows are merged in a tree of warps.  Lists are
// held a key per lane throughout.
__global__ void __launch_bounds__(64 * KD_BEAM_MAX_BEAMS) beam_merge_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ __align__(16) unsigned long long xkey[KD_BEAM_MAX_BEAMS][BS_COUNT_KEYS];  // lists on their way to another warp
    __shared__ int xfrom[KD_BEAM_MAX_BEAMS][32];
    __shared__ int row_v[KD_BEAM_MAX_BEAMS][32];  // the rows' tokens
    __shared__ Pair row_lg[KD_BEAM_MAX_BEAMS];
    __shared__ float row_m[KD_BEAM_MAX_BEAMS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp < a.W ? warp : warp - a.W;
    const int g = blockIdx.x, r = g * a.W + w, K = a.K;
    const LogEntry tab = log_entry(lane);
    pdl_launch_dependents();
    pdl_wait();
    const bool live = beam_live(a.scores, a.done, r);
    const float score = a.scores ? a.scores[r] : 0.0f;
    unsigned long long x = 0ull;  // warps < W: the row's 32 best logits
    if (warp >= a.W) {
        // L = M + log sum_b s_b e^{m_b - M}; the sum in units of 2^-40 (a block's is at most 8192, the largest's at least 1)
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
            unsigned long long sum = 0;
#pragma unroll
            for (int q = 0; q < BS_MAX_BLOCKS / 32; ++q)
                if (32 * q < a.nblk)
                    sum += __float2ull_rn((p[q].x == M ? p[q].y : p[q].y * expf(p[q].x - M)) * 0x1p40f);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
            const Pair lg = pair_log(sum ? sum : 1ull, tab);  // 0: nothing in the row, no candidates either
            if (lane == 0) {
                row_lg[w] = lg;
                row_m[w] = M;
            }
        }
    } else if (live) {
        const unsigned long long* lists = a.keys + (size_t)r * a.nseg * K + lane;
        const int n = a.nseg * K;
        if (a.nseg == 1) {
            x = lane < K ? __ldcg(lists) : 0ull;
        } else {
            // All keys, or, of more than BS_COUNT_KEYS, those that can be among the K best: where m
            // lists reach a value with their p-th keys, m p >= K keys do.  Then by counting.
            static_assert(BS_COUNT_KEYS == 64, "two keys per lane");
            unsigned long long* row = xkey[w];
            int left = n;
            if (n > BS_COUNT_KEYS && K > BS_COUNT_PICK) {
                // more would be left than pay
            } else if (n <= BS_COUNT_KEYS) {
                row[lane] = lane < n ? __ldcg(lists) : 0ull;
                row[lane + 32] = lane + 32 < n ? __ldcg(lists + 32) : 0ull;
            } else {
                const int p = min(K, 2 * ((K + a.nseg - 1) / a.nseg)), m = (K + p - 1) / p;
                const unsigned pth = lane < a.nseg ? (unsigned)(__ldcg(lists - lane + (size_t)lane * K + p - 1) >> 32) : 0u;
                int rank = 0;
                for (int l = 0; l < a.nseg; ++l) rank += __shfl_sync(FULL_MASK, pth, l) > pth ? 1 : 0;
                const unsigned bound = max(1u, __reduce_min_sync(FULL_MASK, lane < a.nseg && rank < m ? pth : 0xffffffffu));
                row[lane] = 0ull;
                row[lane + 32] = 0ull;
                __syncwarp();
                left = 0;
                for (int l = 0; l < a.nseg; l += 8) {
                    unsigned long long v[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] = lane < K && l + q < a.nseg ? __ldcg(lists + (size_t)(l + q) * K) : 0ull;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const bool in = (unsigned)(v[q] >> 32) >= bound;
                        const unsigned who = __ballot_sync(FULL_MASK, in);
                        const int at = left + __popc(who & ((1u << lane) - 1u));
                        if (in && at < BS_COUNT_KEYS) row[at] = v[q];
                        left += __popc(who);
                    }
                }
            }
            __syncwarp();
            if (left <= BS_COUNT_KEYS) {
                const unsigned long long k0 = row[lane], k1 = row[lane + 32];
                const int even = (left + 1) & ~1, r0 = beam_above(row, even, k0);
                const int r1 = left > 32 ? beam_above(row, even, k1) : 32;
                __syncwarp();
                row[lane] = 0ull;
                __syncwarp();
                if (k0 && r0 < 32) row[r0] = k0;
                if (k1 && r1 < 32) row[r1] = k1;
                __syncwarp();
                x = row[lane];
            } else {
                for (int l = 0; l < a.nseg; l += 8) {
                    unsigned long long v[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] = lane < K && l + q < a.nseg ? __ldcg(lists + (size_t)(l + q) * K) : 0ull;
                    const unsigned long long y = warp_merge8(v, a.nseg - l, lane);
                    x = l ? warp_merge(x, y, lane) : y;
                }
            }
        }
        row_v[w][lane] = beam_key_i(x);
    } else if (lane == 0) {
        row_v[w][0] = a.eos;
    }
    __syncthreads();
    // s of every candidate, as a key; from: its beam and place, which order equals
    unsigned long long key = 0ull;
    int from = w * 32 + lane;
    if (warp < a.W) {
        if (live && x) {
            const float xv = beam_key_x(x), M = row_m[w];
            const Pair lg = row_lg[w], c = pair_add({score, 0.0f}, {-lg.hi, -lg.lo});
            key = pair_key(pair_add(xv == M ? Pair{0.0f, 0.0f} : two_sum(xv, -M), c));  // x == M first: M may be infinite
        } else if (!live && lane == 0 && a.done && a.done[r]) {
            key = pair_key({score, 0.0f});  // a finished beam stands for itself; a dead one offers nothing
        }
        // The merges below rank a row's candidates by their lanes, so its keys must fall with the lane.  A pair's
        // sum rounds the low parts first, and two logits whose s differ by less than its last bit can come out the
        // other way round (where x - M passes the middle between two fp32 values, as 2^-17 and the next value under
        // M = 250 with 2% of all scores): such a key takes the least of those before it, and the lane decides.
        const unsigned long long up = __shfl_up_sync(FULL_MASK, key, 1);
        if (__any_sync(FULL_MASK, lane > 0 && key > up)) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long b = __shfl_up_sync(FULL_MASK, key, o);
                if (lane >= o) key = min(key, b);
            }
        }
    }
    auto put = [&](int place, int beam, int tok, unsigned long long k) {
        const int o = g * K + place;
        a.parents[o] = k ? beam : -1;
        a.tokens[o] = k ? tok : -1;
        a.scores_out[o] = k ? beam_unord((unsigned)(k >> 32)) : -INFINITY;
        if (a.done_out) a.done_out[o] = k && (tok == a.eos || (a.done && a.done[g * a.W + beam])) ? 1 : 0;
    };
    if ((a.W + 3) / 4 * a.W * K <= BS_COUNT_ROWS) {  // each candidate counts those before it: of lower beams also its equals
        if (warp < a.W) xkey[warp][lane] = key;
        const int have = __syncthreads_count(warp < a.W && key != 0ull);
        if (warp < a.W && key) {
            int place = lane;
            for (int o = 0; o < a.W; ++o)
                if (o != warp) place += beam_above(xkey[o], (K + 1) & ~1, o < warp ? key - 1 : key);
            if (place < K) put(place, warp, row_v[warp][lane], key);
        }
        if ((int)threadIdx.x >= have && (int)threadIdx.x < K) put(threadIdx.x, 0, -1, 0ull);
        return;
    }
    for (int h = 1; h < a.W; h *= 2) {
        const bool give = warp < a.W && (warp & (2 * h - 1)) == h, take = (warp & (2 * h - 1)) == 0 && warp + h < a.W;
        if (give) {
            xkey[warp][lane] = key;
            xfrom[warp][lane] = from;
        }
        __syncthreads();
        if (take) {
            const unsigned long long k = xkey[warp + h][31 - lane];
            const int f = xfrom[warp + h][31 - lane];
            auto before = [](unsigned long long k1, int f1, unsigned long long k2, int f2) {
                return k1 > k2 || (k1 == k2 && f1 < f2);
            };
            if (before(k, f, key, from)) {
                key = k;
                from = f;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const unsigned long long pk = __shfl_xor_sync(FULL_MASK, key, o);
                const int pf = __shfl_xor_sync(FULL_MASK, from, o);
                if (before(pk, pf, key, from) == !(lane & o)) {
                    key = pk;
                    from = pf;
                }
            }
        }
    }
    if (warp == 0 && lane < K) put(lane, from / 32, key ? row_v[from / 32][from % 32] : -1, key);
}

// stages, and a warp's (m, sum) per block of a segment
static int beam_scan_smem(int blocks, bool shifted) {
    return BS_STAGES * (shifted ? BS_STAGE<BEAM_SHIFTED> : BS_STAGE<BEAM_ALIGNED>) * 4 + blocks * BS_WARPS * 8;
}
static cudaError_t beam_init_attributes() {
    cudaError_t e = cudaSuccess;
    for (const void* f : {(const void*)beam_scan_kernel<BEAM_ALIGNED>, (const void*)beam_scan_kernel<BEAM_SHIFTED>,
                          (const void*)beam_scan_kernel<BEAM_SINGLY>, (const void*)beam_merge_kernel})
        if ((e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout,
                                      cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
            return e;
    for (const void* f : {(const void*)beam_scan_kernel<BEAM_ALIGNED>, (const void*)beam_scan_kernel<BEAM_SHIFTED>,
                          (const void*)beam_scan_kernel<BEAM_SINGLY>})
        if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, beam_scan_smem(BS_MAX_BLOCKS, true))) !=
            cudaSuccess)
            return e;
    return cudaSuccess;
}

}  // namespace kd

extern "C" {

size_t kd_beam_workspace_bytes(int32_t n_groups, int32_t n_beams, int32_t V, int32_t n_out) {
    if (n_groups < 1 || n_beams < 1 || V < 1 || n_out < 1) return 0;
    const size_t nblk = ((size_t)V + kd::BS_STEP - 1) / kd::BS_STEP;
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
    uintptr_t words = 0;
    for (const void* p : {(const void*)logits, (const void*)scores, (const void*)done, (const void*)parents_out,
                          (const void*)tokens_out, (const void*)scores_out, (const void*)done_out})
        words |= reinterpret_cast<uintptr_t>(p);
    if ((reinterpret_cast<uintptr_t>(workspace) & 15) || (words & 3))
        return failf(KD_ERR_INVALID_ARG, "kd_beam_select: the workspace must be 16-byte aligned, the other buffers 4-byte");
    BeamArgs a{};
    const int rows = n_groups * n_beams;
    a.logits = logits;
    a.ld = ld;
    a.V = V;
    a.W = n_beams;
    a.K = n_out;
    a.block_shift = beam_block_shift(V);
    a.nblk = (V + (BS_STEP << a.block_shift) - 1) / (BS_STEP << a.block_shift);
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
    static OncePerDevice once;
    KD_TRY(once(dev, beam_init_attributes));
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
    const bool aligned = ld % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0, shifted = !aligned && V >= BS_SHIFTED_VOCAB;
    const int smem = beam_scan_smem(a.seg_blocks, shifted);
    // Both launches may start while the kernel before them ends; they wait for it first.
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(BS_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    if (aligned)
        KD_TRY(cudaLaunchKernelEx(&cfg, beam_scan_kernel<BEAM_ALIGNED>, a));
    else if (shifted)
        KD_TRY(cudaLaunchKernelEx(&cfg, beam_scan_kernel<BEAM_SHIFTED>, a));
    else
        KD_TRY(cudaLaunchKernelEx(&cfg, beam_scan_kernel<BEAM_SINGLY>, a));
    cfg.gridDim = dim3(n_groups);
    cfg.blockDim = dim3(64 * n_beams);
    cfg.dynamicSmemBytes = 0;
    KD_TRY(cudaLaunchKernelEx(&cfg, beam_merge_kernel, a));
    return KD_OK;
}

}  // extern "C"
