// kd_attn_shared.cu -- attention of a group of sessions over the prefix that they share, on
// the fifth-generation tensor cores: every key and value is read once for up to 128
// queries (64 on Q8_0 caches), the sessions' heads of one KV head.
//
// S = Q K^T and O += P V with tcgen05.mma, the queries as the 128 rows, keys 128 at a
// time.  K and V come by TMA (boxes of a page's rows, 128-byte swizzle, six buffers); the queries
// and the weights are the products' operands in tensor memory, which leaves shared memory's
// rate (one operand of 4 KB a product of 64 cycles takes half of it) to K and V; scores of two tiles are there
// in turn, so that one's products run under the other's exponentials.  Four threads hold a query's row, a quarter of
// the tile's keys each, and tell each other their maxima.  The sums are rescaled only when the
// maximum has grown by 2^8 or more.
//
// Queries and weights are fp16 pairs hi + lo, as in the kernel of the sessions' own
// keys (kd_attn_paged.cu: what pairs are good to; weights are held as 2^7 times their value, at most 2^15 with what the maximum
// has grown, which leaves room for the rounding of the maximum's product with the scale while scores are below 10^7), two products each: 4 x 2 x 128^3 flops a tile of 128 keys and 128 queries, 2048 cycles, 1.1 us
// at the SM's share of the bf16 rate, while its 64 KB take 1.4 us of the SM's share of the memory's.
// Q8_0 rows become such pairs, too (three products each), made by eight warps of their own.  A row that holds a scale of
// 512 or more, whose values may leave fp16's range, is divided by a power of two; K's goes back to the scores, V's to the
// weights, whose maximum such a tile always moves (to look for such rows costs 1 to 2 us of the 97 below).
//
// Two groups of 32 sessions behind 16384 and 15383 keys, 8 KV heads of 128, take 61 us with the sessions' own 91 MB and the
// merge, 392 where each reads its prefix; a tile takes 3300 cycles then: neither memory nor the tensor core (active 0.44) bounds it, but the chain of
// scores, maximum, exchange, weights and products, of which two tiles are in turn.  Three
// groups of 8 on Q8_0 caches behind 26 k keys: 97 us, 311 where each reads, 4400 cycles a tile: shared memory's rate (512 cycles
// to write a part's pairs, 768 for three products to read them, 270 for the codes, of 2200 a part).
//
// CTAs share the tiles of all (group, KV head)s equally (kd_paged.h); what one finds of a
// (group, head) goes to a record that the merge reads.  Groups of more queries are taken by
// CTAs side by side, one tile of queries each, that read the same keys at the same time.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kd_attn_common.cuh"
#include "kd_host.h"
#include "kd_paged.h"

namespace kd {

// ---- tcgen05 ---------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// D (tensor memory) += or = A B: A in tensor memory, B by descriptor in shared memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((int)add)
        : "memory");
}
// 32 columns of the warp's 32 rows, a row per lane.
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
// The loads before have arrived; v is theirs, so that no use of it is moved up.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// 8 columns of 16 rows: a lane has columns 2 (lane % 4) and the next of row lane / 4 (v0, v1) and of
// the row 8 below (v2, v3).  Where rows lie apart in memory, four lanes read or write 32 bytes or more of one.
__device__ __forceinline__ void tc_st_16x8(uint32_t addr, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v0), "r"(v1), "r"(v2), "r"(v3) : "memory");
}
__device__ __forceinline__ void tc_ld_16x8(uint32_t addr, uint32_t (&v)[4]) {  // (to be waited for)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t* v) {  // and waits
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 2^x to 2^-22, 0 below fp32's normal range.
__device__ __forceinline__ float tc_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A shared-memory operand in 128-byte swizzled rows, 8 of them 1024 bytes: sbo from 8 rows
// to the next 8, lbo (operands whose rows run along K) from 64 columns to the next 64.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// fp16 operands, fp32 sums, M = 128; b_cols: B's rows run along K (its columns are contiguous).
__device__ __forceinline__ constexpr uint32_t tc_idesc(int n, bool b_cols) {
    return 1u << 4 | (b_cols ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// ---- the kernel ---------------------------------------------------------------
constexpr int SH_SOFT = 16;  // softmax warps (Q8_0: four, and eight that make K and V)
constexpr int SH_COPY = SH_SOFT, SH_SCORES = SH_SOFT + 1, SH_VALUES = SH_SOFT + 2;  // the copies' and the products' warps
constexpr int SH_THREADS = (SH_SOFT + 3) * 32;
constexpr float SH_UP = 7.0f;

template <int HD, bool Q8>
struct SharedSmem {
    static constexpr int QUERIES = shared_queries(Q8);
    static constexpr int SHARE = Q8 ? 2 : 4;           // threads (warps) of a row
    static constexpr int WEIGH = SHARE * QUERIES / 32; // softmax warps
    static constexpr int COLS = HD / 64;               // 128-byte columns of a row
    static constexpr int COL = SHARED_TILE * 128;      // one of a tile
    static constexpr int TILE = COLS * COL;            // K or V of a tile
    static constexpr int SLOTS = HD == 64 ? 8 : 6;
    static constexpr int RING = 0, BARS = SLOTS * TILE;
    static constexpr int MAXIMA = BARS + 320;          // [2][share][row]: what the warps of a row tell each other
    static constexpr int CODES = MAXIMA + 2 * SHARE * QUERIES * 4;  // Q8_0: a part's codes, by thread, and scales, by warp, on their way
    static constexpr int EARLY = CODES + 256 * 4 * 16 + 8 * 128;  // [tile % 2]: V's scales, with K on their way, by warp
    static constexpr int UPS = EARLY + 2 * 8 * 128;        // [tile % 8][K, V][row]: what rows whose scales are large were divided by
    static constexpr int LARGE = UPS + 8 * 2 * SHARED_TILE * 4;  // [tile % 8][warp]: 1 where there is such a row, else the warp leaves no divisors
    static constexpr int TOTAL = Q8 ? LARGE + 8 * 8 : CODES;
    static_assert(TOTAL <= 227 * 1024, "opt-in shared memory");
};
// Columns of tensor memory: scores, then weights, of two tiles in turn (128 each); the sums; the queries, hi and lo.
constexpr uint32_t TM_SUMS = 256, TM_QUERIES = 384;

// Q8_0: the first of the two places, counted on round the buffers, of K (part 0) or V (1) of a CTA's tile t: in
// the order K0 K1 V0 K2 V1 K3 V2 ..., as V is made when its tile has been weighed, and then the K after next.
__device__ __forceinline__ uint32_t shared_place(uint32_t t, int part) { return 2 * (part ? 2 * t + 2 : t ? 2 * t - 1 : 0); }

// Four block scales of a Q8_0 row in fp16: a power of two, 1 to 2^7, by which 128 times each of them is divided
// into fp16's range (65504 is 128 times 511.75, so 1 for scales below 512).
__device__ __forceinline__ bool shared_large(uint32_t x, uint32_t y) {
    return ((((x & (x << 1)) | (y & (y << 1))) & 0x40004000u) != 0);  // an exponent of 2^9 or more
}
__device__ __forceinline__ int shared_down(uint32_t x, uint32_t y) {
    const uint32_t e = __vmaxu2(__vmaxu2(x & 0x7c007c00u, y & 0x7c007c00u), 0x5c005c00u);
    return min((int)(max(e & 0xffffu, e >> 16) >> 10) - 23, 7);
}

// A CTA's next tiles of one (group, KV head, pass).
struct SharedSeg {
    int g = 0, h, pass, tile, n;  // tiles [tile, tile + n)
    // from x on, at most `left` of them; g: a group at or before x's
    __device__ __forceinline__ void at(const SharedArgs& a, int x, int left) {
        while (x >= a.g[g + 1].first * a.nkv) ++g;
        const int r = x - a.g[g].first * a.nkv, T = a.tiles(g), u = r / T;
        tile = r - u * T;
        h = u;
        pass = 0;
        if (a.passes(g) > 1) {
            h = u / a.passes(g);
            pass = u - h * a.passes(g);
        }
        n = min(T - tile, left);
    }
};

template <int HD, bool Q8>
__global__ void __launch_bounds__(SH_THREADS, 1)
    shared_kernel(const __grid_constant__ SharedArgs a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using L = SharedSmem<HD, Q8>;
    constexpr int NS = L::SLOTS;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BARS);
    uint64_t *empty = full + NS, *s_full = empty + NS, *p_full = s_full + 2, *pv_done = p_full + 2, *q_full = pv_done + 2, *q_free = q_full + 1, *pair = q_free + 1, *drained = pair + 4;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 2);
    volatile int* failed = reinterpret_cast<volatile int*>(tmem_at + 1);
    // The last tiles' 16-key runs that have a page, by tile: an entry is written again after 8 tiles, when the
    // buffers (at most 8, two a tile) have gone round past its tile's values, so past its softmax.
    volatile uint8_t* runs = reinterpret_cast<volatile uint8_t*>(tmem_at + 2);
    static_assert(NS <= 8, "tiles in the buffers");
    static_assert((2 * NS + 14) * 8 + 16 <= 320, "barriers and words");

    if (smem_u32(smem) & 1023) {  // the swizzle counts on it, and there is no room to move up
        pdl_wait();
        if (threadIdx.x == 0) a.status[blockIdx.x] = 1;
        return;
    }
    if (warp == SH_COPY) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_at)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, Q8 ? SH_SOFT / 2 : 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(drained + i, 1);
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, L::WEIGH);
            mbar_init(pv_done + i, 1);
        }
        mbar_init(q_full, L::WEIGH);
        mbar_init(q_free, L::WEIGH);
        for (int i = 0; i < 4; ++i) mbar_init(pair + i, L::SHARE);
        mbar_init_fence();
        // debug fault hook: the first tile's K or V waits for bytes that nothing delivers
        if (a.inject && blockIdx.x == 0) mbar_expect_tx(full + (Q8 ? shared_place(0, a.inject - 1) % NS : a.inject - 1), 16);
        *failed = 0;
        if (!Q8) {
            prefetch_tmap(&tmk);
            prefetch_tmap(&tmv);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    const int set = blockIdx.x / a.side, mine = blockIdx.x - set * a.side;  // of the CTAs side by side
    const int x0 = a.share.begin(set), x1 = a.share.begin(set + 1);
    SharedSeg head;  // the CTA's first segment
    head.at(a, x0, x1 - x0);
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == SH_VALUES * 32)  // the kernel behind this one reads what was written before both
        asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(a.started), "l"(a.call) : "memory");
    pdl_launch_dependents();  // after the wait, so that no CTA of that kernel starts before it
    const int box = a.box_runs;  // 16-key runs of a copy's box
    // The first of the CTA's queries in a segment's group, and how many (<= 0: none).
    auto first_query = [&](const SharedSeg& s) { return (s.pass * a.side + mine) * L::QUERIES; };
    auto n_queries = [&](const SharedSeg& s) { return min(L::QUERIES, a.g[s.g].queries - first_query(s)); };

    if (warp == SH_COPY) {
        if constexpr (!Q8) {
        // ---- copies: K and V of each tile, boxes of whole 16-key runs within a page
        uint32_t slot = 0, phase = 0, tiles = 0;
        bool ok = true;
        SharedSeg s = head;
        for (int x = x0; x < x1 && ok;) {
            if (x != x0) s.at(a, x, x1 - x);
            x += s.n;
            if (n_queries(s) <= 0) continue;
            const int keys = a.g[s.g].keys;
            const int* row = a.table + (int64_t)a.g[s.g].lead * a.table_ld;
            auto look_up = [&](int t) {  // lane i: the page of the tile's run i
                const int key = t * SHARED_TILE + 16 * lane;
                return lane < SHARED_TILE / 16 && key < keys ? row[key / a.ps] : -1;
            };
            int page = look_up(s.tile);
            for (int t = s.tile; t < s.tile + s.n && ok; ++t, ++tiles) {
                const int key = t * SHARED_TILE + 16 * lane;
                const int here = min(SHARED_TILE, keys - t * SHARED_TILE) / 16;  // runs
                const bool good = lane < here && (unsigned)page < (unsigned)a.n_pages;
                if (lane < here && !good && a.fault) *a.fault = 1;
                const unsigned mask = __ballot_sync(FULL_MASK, good) & 0xffu;
                // a page that does not exist: rows behind the last one, which read as zeros
                const int y = good ? (page * a.nkv + s.h) * a.ps + key % a.ps : a.rows;
                if (t + 1 < s.tile + s.n) page = look_up(t + 1);
                for (int part = 0; part < 2 && ok; ++part) {
                    if (lane == 0) ok = mbar_wait_bounded(empty + slot, phase ^ 1);
                    ok = __shfl_sync(FULL_MASK, ok, 0);
                    if (!ok) break;
                    if (lane == 0) {
                        if (!part) runs[tiles & 7] = (uint8_t)mask;
                        mbar_arrive_expect_tx(full + slot, (uint32_t)(here * 16 * HD * 2));
                    }
                    __syncwarp();
                    if (lane < here && lane % box == 0) {
                        uint8_t* dst = smem + L::RING + slot * L::TILE + lane * 16 * 128;
#pragma unroll
                        for (int c = 0; c < L::COLS; ++c) tma_load_2d(dst + c * L::COL, part ? &tmv : &tmk, 64 * c, y, full + slot);
                    }
                    __syncwarp();
                    if (++slot == NS) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        if (!ok && lane == 0) *failed = 1;
        }
    } else if (warp == SH_SCORES || warp == SH_VALUES) {
        // ---- products, S = Q K^T and O += P V by a thread each: one that has issued products
        // goes on only when the tensor core has taken them (1200 cycles for a tile's), and the other's
        // should be ready then.  K parts are in the buffers' even places of a round, V parts in the odd ones.
        if (lane == 0) {
            const bool values = warp == SH_VALUES;
            // buffers of a tile's K or V: one, or with Q8_0 the two parts of the pairs
            constexpr int PARTS = Q8 ? 2 : 1;
            uint32_t place = values, tile = 0, q_phase = 0;
            unsigned turn_phase = 0;  // of p_full (values) or pv_done (scores), a bit for even and odd tiles
            bool ok = true;
            const uint32_t ring = smem_u32(smem + L::RING);
            SharedSeg s = head;
            for (int x = x0; x < x1 && ok;) {
                if (x != x0) s.at(a, x, x1 - x);
                x += s.n;
                if (n_queries(s) <= 0) continue;
                const int keys = a.g[s.g].keys;
                if (!values) {
                    ok = mbar_wait_bounded(q_full, q_phase);  // the segment before is done with then, too
                    q_phase ^= 1;
                }
                for (int j = 0; j < s.n && ok; ++j) {
                    const int w = j & 1, n = min(SHARED_TILE, keys - (s.tile + j) * SHARED_TILE);
                    // weights that are there; or, for scores, weights in their place that are done with
                    if (values || j >= 2) ok = mbar_wait_bounded((values ? p_full : pv_done) + w, (turn_phase >> w) & 1);
                    if constexpr (Q8) place = shared_place(tile++, values);
                    uint32_t slot[PARTS];
                    slot[0] = place % NS;
                    if constexpr (Q8) slot[1] = slot[0] + 1;  // places are even, and so is the number of buffers
                    ok = ok && mbar_wait_bounded(full + slot[0], (place / NS) & 1);
                    place += 2;  // fp16: K and V parts lie in turn
                    if (!ok) break;
                    if (values || j >= 2) turn_phase ^= 1u << w;
                    tc_fence_after();
                    // lo hi, hi lo, hi hi: the small ones first, so that the scores' sums are rounded at their
                    // own size in the last 8 products only (what is left out is 2^-22 of a product)
                    if (!values) {
                        const uint32_t id = tc_idesc(n, false);
#pragma unroll
                        for (int part = 0; part < 1 + PARTS; ++part)
#pragma unroll
                            for (int k = 0; k < HD / 16; ++k) {
                                const uint32_t off = (k / 4) * L::COL + (k % 4) * 32;
                                const uint64_t kd = tc_desc(ring + slot[Q8 && part == 1 ? PARTS - 1 : 0] * L::TILE + off, 0);
                                tc_mma_ts(tmem + w * 128, tmem + TM_QUERIES + (part == 0 ? HD / 2 : 0) + 8 * k, kd, id, part || k);
                            }
                        tc_commit(s_full + w);
                    } else {
                        const uint32_t id = tc_idesc(HD, true);
                        for (int k = 0; k < n / 16; ++k)
#pragma unroll
                            for (int part = 0; part < 1 + PARTS; ++part)
                                tc_mma_ts(tmem + TM_SUMS, tmem + w * 128 + 32 * (k / 2) + (part == 1 ? 16 : 0) + 8 * (k & 1),
                                          tc_desc(ring + slot[part / 2] * L::TILE + k * 2048, L::COL), id, part || k || j);
                        tc_commit(pv_done + w);
                    }
                    tc_commit(empty + slot[0]);
                }
                // The last products of even and odd tiles are not waited for here: keep their count.
                if (!values) turn_phase ^= (s.n > 0 ? 1u : 0u) | (s.n > 1 ? 2u : 0u);
            }
            if (!ok) *failed = 1;
            // Products that are still under way, and what they signal, before the memory is given up.
            tc_commit(drained + values);
            if (!mbar_wait_bounded(drained + values, 0)) *failed = 1;
        }
        __syncwarp();
    } else {
        // ---- softmax: SHARE threads have a query's row, an equal part of the tile's keys (then of the head's dims) each
        constexpr int KEYS = SHARED_TILE / L::SHARE, DIMS = HD / L::SHARE;
        const int part = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);
        const uint32_t ot = lane_base + TM_SUMS + part * DIMS;
        float* maxima = reinterpret_cast<float*>(smem + L::MAXIMA);
        unsigned s_phase = 0, t_phase = 0, met = 0;  // scores seen and tiles weighed, a bit for even and odd ones; meetings of a row's warps
        uint32_t tiles = 0, segs = 0;
        bool ok = true;
        const float c = a.scale * 1.4426950408889634f;
        // Tell the row's other threads x and have all of theirs joined.  (In turn in two places: who writes again
        // has met them in between, so they have read.)
        auto exchange = [&](float x, auto join) {
            float* at = maxima + (met & 1) * L::SHARE * L::QUERIES + r;
            at[part * L::QUERIES] = x;
            __syncwarp();
            if (lane == 0) mbar_arrive(pair + (warp & 3));
            ok = __all_sync(FULL_MASK, mbar_wait_bounded(pair + (warp & 3), met++ & 1));
            float v = at[0];
#pragma unroll
            for (int i = 1; i < L::SHARE; ++i) v = join(v, at[i * L::QUERIES]);
            return v;
        };
        SharedSeg s = head;
        // Q8_0: warps 8 .. 15 make K (part 0) and V (1) of tile j of the segment, codes times scales as fp16
        // pairs hi + lo (19 bits, so exactly): a thread takes 16 codes of rows trow + 32 i.
        const bool makes = Q8 && warp >= 8;
        const int t = threadIdx.x & 255;
        // 8 lanes write 4 chunks of two rows, which the swizzle puts into different banks
        const int chunk = (lane & 3) | ((lane >> 4) << 2), trow = (t >> 5) * 4 + ((lane >> 2) & 3);
        struct Codes {
            uint4 v[4];
            __half d[4];
        };
        // The thread's codes and scales of a part, to its own place in shared memory: loads to registers would be
        // waited for together with those of the part after.
        const uint32_t mine_at = smem_u32(smem + L::CODES) + t * 16;
        const uint32_t scales_at = smem_u32(smem + L::CODES) + 256 * 4 * 16 + (t >> 5) * 128;  // the warp's: 4 rows of each i, 8 bytes each
        const uint32_t early_at = smem_u32(smem + L::EARLY) + (t >> 5) * 128;
        auto fetch = [&](int rows, int part, uint32_t T) {
            const uint8_t* codes = (part ? a.vq : a.kq) + (trow & 15) * 128 + 16 * chunk;
            const unsigned have = __ballot_sync(FULL_MASK, rows >= 0);
            if (!part && t == 0) runs[T & 7] = (uint8_t)have;
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // the warp's rows of i are of one run
                const int first = __shfl_sync(FULL_MASK, rows, 2 * i + (t >> 7));
                // else zeros: a scale of 0, whatever the codes
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(mine_at + i * 256 * 16), "l"(codes + (int64_t)max(first, 0) * 128),
                             "r"(first >= 0 ? 16 : 0)
                             : "memory");
            }
            const int first = __shfl_sync(FULL_MASK, rows, (lane & 6) + (t >> 7));
            if (lane < 8) {  // two rows' scales of i = lane / 2
                const uint8_t* scales = (const uint8_t*)(part ? a.vs : a.ks) + ((t >> 5) & 3) * 32 + (lane & 1) * 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(scales_at + lane * 16), "l"(scales + (int64_t)max(first, 0) * 8),
                             "r"(first >= 0 ? 16 : 0)
                             : "memory");
                // V's, too: its tile's weights are formed before it is made
                if (!part)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(early_at + (T & 1) * 1024 + lane * 16),
                                 "l"((const uint8_t*)a.vs + ((t >> 5) & 3) * 32 + (lane & 1) * 16 + (int64_t)max(first, 0) * 8), "r"(first >= 0 ? 16 : 0)
                                 : "memory");
            }
        };
        auto landed = [&](Codes& f) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                unsigned short d;
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(f.v[i].x), "=r"(f.v[i].y), "=r"(f.v[i].z), "=r"(f.v[i].w)
                             : "r"(mine_at + i * 256 * 16)
                             : "memory");
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(d) : "r"(scales_at + i * 32 + (trow & 3) * 8 + (chunk >> 1) * 2) : "memory");
                f.d[i] = __ushort_as_half(d);
            }
            // read before the next part's copies are issued
#pragma unroll
            for (int i = 0; i < 4; ++i) asm volatile("" : "+r"(f.v[i].x), "+r"(f.v[i].y), "+r"(f.v[i].z), "+r"(f.v[i].w)::"memory");
            __syncwarp();
        };
        unsigned v_large = 0;  // a bit for even and odd tiles
        auto make = [&](int part, uint32_t T, const Codes& f) {
            // Rows of the warp's with large scales: with K looked for in the thread's own scales and in V's; all else only where there are any.
            const uint8_t* early = smem + L::EARLY + (T & 1) * 1024 + (t >> 5) * 128;
            bool large = (v_large >> (T & 1)) & 1;
            if (!part) {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) top = max(top, (uint32_t)__half_as_ushort(f.d[i]) & 0x7fffu);
                uint4 of_v = make_uint4(0, 0, 0, 0);
                if (lane < 8) of_v = lds_v4(early + lane * 16);
                large = __any_sync(FULL_MASK, top >= 0x6000u || shared_large(of_v.x, of_v.y) || shared_large(of_v.z, of_v.w));
                v_large = (v_large & ~(1u << (T & 1))) | (large ? 1u << (T & 1) : 0u);
                if (lane == 0) smem[L::LARGE + (T & 7) * 8 + (t >> 5)] = large;
                if (large && lane < 8) {  // V's divisors, for the warps that weigh
                    float* up = reinterpret_cast<float*>(smem + L::UPS) + ((T & 7) * 2 + 1) * SHARED_TILE + 32 * (lane >> 1) + 4 * (t >> 5) + 2 * (lane & 1);
                    *reinterpret_cast<float2*>(up) = make_float2((float)(1 << shared_down(of_v.x, of_v.y)), (float)(1 << shared_down(of_v.z, of_v.w)));
                }
            }
            const uint32_t place = shared_place(T, part), s0 = place % NS, s1 = s0 + 1;
            if (!__all_sync(FULL_MASK, mbar_wait_bounded(empty + s0, ((place / NS) & 1) ^ 1))) return false;
            uint8_t* dst = smem + L::RING + (chunk >> 2) * L::COL + trow * 128;
            const uint32_t c0 = ((2 * (chunk & 3)) ^ (trow & 7)) << 4;  // the second 8 dims are 16 bytes away in it
            auto pairs = [&](auto divided) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2 dd = __half2half2(f.d[i]);
                    const uint32_t w[4] = {f.v[i].x, f.v[i].y, f.v[i].z, f.v[i].w};
                    __half2 div = dd;
                    if constexpr (decltype(divided)::value) {  // codes are divided, exactly, before the product: a smaller scale of the row keeps its bits
                        uint32_t d = (uint32_t)__half_as_ushort(f.d[i]) & 0x7fffu;  // the largest of the row's four
                        d = max(d, __shfl_xor_sync(FULL_MASK, d, 2));
                        d = max(d, __shfl_xor_sync(FULL_MASK, d, 16));
                        const float up = (float)(1 << shared_down(d, 0));
                        if (!part && (lane & 19) == 0) reinterpret_cast<float*>(smem + L::UPS)[(T & 7) * 2 * SHARED_TILE + 32 * i + trow] = up;
                        div = __float2half2_rn(1.0f / up);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t q = (e & 1) ? u8x2_hi_to_half2(w[2 * k + (e >> 1)]) : u8x2_lo_to_half2(w[2 * k + (e >> 1)]);
                            __half2 c = *reinterpret_cast<const __half2*>(&q);
                            if constexpr (decltype(divided)::value) c = __hmul2_rn(c, div);
                            const __half2 h = __hmul2_rn(c, dd), l = __hfma2(c, dd, __hneg2(h));
                            hi[e] = *reinterpret_cast<const uint32_t*>(&h);
                            lo[e] = *reinterpret_cast<const uint32_t*>(&l);
                        }
                        uint8_t* at = dst + i * 32 * 128 + (c0 ^ (k << 4));
                        *reinterpret_cast<uint4*>(at + s0 * L::TILE) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(at + s1 * L::TILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            };
            if (large) pairs(std::true_type{});
            else pairs(std::false_type{});
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(full + s0);
            return true;
        };
        if (makes) {
            // the parts in the order of their places, K0 [K1] V0 K2 V1 .., a part's codes fetched while the one before is made
            const int tile_pages = SHARED_TILE / a.ps, tile_rest = SHARED_TILE - tile_pages * a.ps;
            for (int x = x0; x < x1 && ok;) {
                if (x != x0) s.at(a, x, x1 - x);
                x += s.n;
                if (n_queries(s) <= 0) continue;
                const int keys = a.g[s.g].keys;
                // Lane i < 8: run i of the next K's tile, its place in the table and in its page, and the page's number
                // (-1: no run), which is not looked at before that K is fetched.
                const int* row = a.table + (int64_t)a.g[s.g].lead * a.table_ld;
                int key = s.tile * SHARED_TILE + 16 * lane, in_table = key / a.ps, in_page = key - in_table * a.ps, page;
                auto look_up = [&] { page = lane < 8 && key < keys ? row[in_table] : -1; };
                look_up();
                int nk = 0, nv = 0, rows = -1, before = -1;  // K and V parts fetched; the cache rows of the last K's runs, and the one's before
                auto fetch_k = [&] {
                    before = rows;
                    const bool good = (unsigned)page < (unsigned)a.n_pages;
                    if (!good && lane < 8 && key < keys && a.fault) *a.fault = 1;
                    rows = good ? (page * a.nkv + s.h) * a.ps + in_page : -1;
                    fetch(rows, 0, tiles + nk);
                    if (++nk < s.n) {
                        key += SHARED_TILE;
                        in_table += tile_pages;
                        in_page += tile_rest;
                        if (in_page >= a.ps) {
                            in_page -= a.ps;
                            ++in_table;
                        }
                        look_up();
                    }
                };
                fetch_k();
                for (int part = 0, k = 0; k < 2 * s.n && ok; ++k) {
                    Codes f;
                    landed(f);
                    const int j = part ? nv - 1 : nk - 1, now = part;
                    if (k + 1 < 2 * s.n) {
                        part = part ? nk == s.n : s.n == 1 || nk > 1;
                        if (!part) {
                            fetch_k();
                        } else {
                            fetch(nk - 1 > nv ? before : rows, 1, tiles + nv);
                            ++nv;
                        }
                    }
                    ok = make(now, tiles + j, f);
                }
                tiles += s.n;
            }
        }
        const bool weighs = (warp & 3) * 32 < L::QUERIES && part < L::SHARE;
        for (int x = weighs ? x0 : x1; x < x1 && ok;) {
            if (x != x0) s.at(a, x, x1 - x);
            x += s.n;
            const int nq = n_queries(s), q0 = first_query(s);
            if (nq <= 0) continue;
            const int keys = a.g[s.g].keys;
            {  // the queries, hi and lo: the warp's dims of its 32 rows, 16 dims of 16 rows at a time
                const uint32_t qt = lane_base + TM_QUERIES + part * (DIMS / 2);
                const int lg = 31 - __clz(a.gq);  // a power of two
                float4 u[4][DIMS / 16];           // rows 8 apart, all on their way at once
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = (warp & 3) * 32 + 8 * e + (lane >> 2), qi = q0 + row;
                    const float* src = a.q + ((size_t)(a.g[s.g].lead + (qi >> lg)) * a.nh + (size_t)(s.h << lg) + (qi & (a.gq - 1))) * HD + part * DIMS + 4 * (lane & 3);
#pragma unroll
                    for (int k = 0; k < DIMS / 16; ++k) {
                        u[e][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (row < nq) u[e][k] = *reinterpret_cast<const float4*>(src + 16 * k);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2)
#pragma unroll
                    for (int k = 0; k < DIMS / 16; ++k) {
                        const float4 x = u[e][k], y = u[e + 1][k];
                        const uint32_t at = qt + ((uint32_t)(8 * e) << 16) + 8 * k;
                        tc_st_16x8(at, f2_hi(x.x, x.y), f2_hi(x.z, x.w), f2_hi(y.x, y.y), f2_hi(y.z, y.w));
                        tc_st_16x8(at + HD / 2, f2_lo(x.x, x.y), f2_lo(x.z, x.w), f2_lo(y.x, y.y), f2_lo(y.z, y.w));
                    }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            const bool idle = (warp & 3) * 32 >= nq;  // no query in the warp's rows: what its weights hold does not matter
            float m = -INFINITY;                      // the maximum that the weights are taken against, in units of 1 / c
            float2 l = make_float2(0.0f, 0.0f);
            // The product P V of tile j, the last weighed of the even or odd ones, is done.
            auto values_done = [&](int j) { return __all_sync(FULL_MASK, mbar_wait_bounded(pv_done + (j & 1), ((t_phase >> (j & 1)) & 1) ^ 1)); };
            for (int j = 0; j < s.n && ok; ++j) {
                const int b = j & 1;
                const uint32_t st = lane_base + b * 128 + part * KEYS;
                const int n = min(KEYS, keys - (s.tile + j) * SHARED_TILE - part * KEYS);  // the thread's keys of the tile
                ok = __all_sync(FULL_MASK, mbar_wait_bounded(s_full + b, (s_phase >> b) & 1));
                s_phase ^= 1u << b;
                if (!ok) break;
                tc_fence_after();
                const unsigned have = runs[(tiles + j) & 7] >> (part * (KEYS / 16));  // their 16-key runs that have a page
                // (Q8_0) Rows that were divided, and by what: a warp that makes has 4 of 32 rows in a row, and a byte here.
                uint2 large = make_uint2(0, 0);
                const float* ups = nullptr;
                if constexpr (Q8) {
                    large = *reinterpret_cast<const uint2*>(smem + L::LARGE + ((tiles + j) & 7) * 8);
                    ups = reinterpret_cast<const float*>(smem + L::UPS) + ((tiles + j) & 7) * 2 * SHARED_TILE + part * KEYS;
                }
                const bool any_large = (large.x | large.y) != 0;
                auto divisors = [&](int v, int i) {  // of K's or V's rows i .. i + 3
                    return ((i & 16 ? large.y : large.x) >> (2 * (i & 12))) & 0xff ? *reinterpret_cast<const float4*>(ups + v * SHARED_TILE + i) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                };
                if (!idle) {
                    constexpr int STEPS = KEYS / 32;
                    const bool all = n == KEYS && (have & ((1u << (KEYS / 16)) - 1)) == (1u << (KEYS / 16)) - 1;
                    uint32_t v[32];  // 32 keys' scores
                    auto load = [&](int k) {
                        tc_ld32(st + 32 * k, v);
                        tc_wait_ld(v);
                        if (!all) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(32 * k + i < n && ((have >> (2 * k + (i >> 4))) & 1))) v[i] = __float_as_uint(-INFINITY);
                        }
                    };
                    if (Q8 && any_large) {  // scores times K's divisors, in their place
#pragma unroll 1
                        for (int k = 0; 32 * k < n; ++k) {
                            tc_ld32(st + 32 * k, v);
                            tc_wait_ld(v);
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 u = divisors(0, 32 * k + i);
                                v[i] = __float_as_uint(__uint_as_float(v[i]) * u.x);
                                v[i + 1] = __float_as_uint(__uint_as_float(v[i + 1]) * u.y);
                                v[i + 2] = __float_as_uint(__uint_as_float(v[i + 2]) * u.z);
                                v[i + 3] = __float_as_uint(__uint_as_float(v[i + 3]) * u.w);
                            }
                            tc_st32(st + 32 * k, v);
                        }
                        tc_wait_st();
                    }
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < STEPS; ++k)
                        if (32 * k < n) {
                            load(k);
#pragma unroll
                            for (int i = 0; i < 32; ++i) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(v[i]));
                        }
                    const float mx = exchange(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), [](float x, float y) { return fmaxf(x, y); });
                    if (!ok) break;
                    float f = 1.0f;
                    if (m == -INFINITY) {
                        m = mx;
                        f = 0.0f;
                    } else if ((mx - m) * c > (Q8 && any_large ? 0.0f : 8.0f)) {  // weights of divided rows have their factor to hold, too
                        f = tc_exp2((m - mx) * c);
                        m = mx;
                    }
                    if (j && __any_sync(FULL_MASK, f != 1.0f)) {
                        ok = values_done(j - 1);
                        if (!ok) break;
                        tc_fence_after();
                        l.x *= f;
                        l.y *= f;
#pragma unroll 1
                        for (int k = 0; k < DIMS / 16; ++k) {
                            uint32_t o[16];
                            tc_ld16(ot + 16 * k, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tc_st16(ot + 16 * k, o);
                        }
                    }
                    // 2^SH_UP times the weights, up to 2^15 with what the maximum has grown: so that small ones keep
                    // more bits (2^(-inf) where no key is seen)
                    const float mc = m == -INFINITY ? 0.0f : m * c - SH_UP;
#pragma unroll
                    for (int k = STEPS - 1; k >= 0; --k) {  // the last are still here
                        if (32 * k < n) {
                            if (STEPS > 1 && k == 0 && n > 32) load(0);
                            uint32_t p[32];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 t = f2_fma(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])),
                                                      make_float2(c, c), make_float2(-mc, -mc));
                                const float2 e = make_float2(tc_exp2(t.x), tc_exp2(t.y));
                                l = f2_add(l, e);
                                p[i] = f2_hi(e.x, e.y);
                                const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
                                const float2 lo = f2_fma(hi, make_float2(-1.0f, -1.0f), e);
                                p[16 + i] = f2_hi(lo.x, lo.y);
                            }
                            tc_st32(st + 32 * k, p);  // the weights in the scores' place: 16 columns hi, 16 lo
                        }
                    }
                    tc_wait_st();
                    if (Q8 && any_large) {  // weights times V's divisors: at most 2^14
#pragma unroll 1
                        for (int k = 0; 32 * k < n; ++k) {
                            tc_ld32(st + 32 * k, v);
                            tc_wait_ld(v);
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float4 u = divisors(1, 32 * k + 2 * i);
                                const __half2 u0 = __floats2half2_rn(u.x, u.y), u1 = __floats2half2_rn(u.z, u.w);
#pragma unroll
                                for (int w = i; w < 32; w += 16) {
                                    const __half2 h0 = __hmul2(*reinterpret_cast<const __half2*>(&v[w]), u0), h1 = __hmul2(*reinterpret_cast<const __half2*>(&v[w + 1]), u1);
                                    v[w] = *reinterpret_cast<const uint32_t*>(&h0);
                                    v[w + 1] = *reinterpret_cast<const uint32_t*>(&h1);
                                }
                            }
                            tc_st32(st + 32 * k, v);
                        }
                        tc_wait_st();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + b);
                t_phase ^= 1u << b;
            }
            tiles += s.n;
            // ---- the record of the segment's tiles
            if (ok) {
                ok = values_done(s.n - 1);
                tc_fence_after();
            }
            if (ok && !idle) {
                float* rec = a.part + shared_row(a, s.g, s.h, s.pass, set, q0 - s.pass * a.side * L::QUERIES) * PAGED_REC(HD);
                const float sum = exchange(l.x + l.y, [](float x, float y) { return x + y; });
#pragma unroll
                for (int rh = 0; rh < 2; ++rh) {
                    const int row = (warp & 3) * 32 + 16 * rh + (lane >> 2);
                    float* to = rec + (size_t)row * PAGED_REC(HD) + part * DIMS + 2 * (lane & 3);
#pragma unroll 4
                    for (int k = 0; k < DIMS / 8; ++k) {
                        uint32_t v[4];
                        tc_ld_16x8(ot + ((uint32_t)(16 * rh) << 16) + 8 * k, v);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3])::"memory");
                        if (row < nq) *reinterpret_cast<uint2*>(to + 8 * k) = make_uint2(v[0], v[1]);
                        if (row + 8 < nq) *reinterpret_cast<uint2*>(to + 8 * PAGED_REC(HD) + 8 * k) = make_uint2(v[2], v[3]);
                    }
                }
                if (r < nq && !part) *reinterpret_cast<float2*>(rec + (size_t)r * PAGED_REC(HD) + HD) = make_float2(m * a.scale - SH_UP * 0.6931471806f, sum);
            }
            tc_fence_before();
            // All are done with the queries and with tensor memory.
            __syncwarp();
            if (lane == 0) mbar_arrive(q_free);
            ok = ok && __all_sync(FULL_MASK, mbar_wait_bounded(q_free, segs++ & 1));
        }
        if (!ok) *failed = 1;
        if constexpr (Q8) asm volatile("cp.async.wait_all;" ::: "memory");  // (a warp that gave up has some on their way)
        tc_fence_before();
    }
    __syncthreads();
    if (warp == SH_COPY) {
        if (!Q8 && *failed) {  // copies may be in flight: give them their time before the memory is given up
            if (lane < NS)
                for (int i = 0; i < 2; ++i) (void)mbar_wait_bounded(full + lane, i);
            __syncwarp();
        }
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
        if (lane == 0) a.status[blockIdx.x] = *failed;
    }
}

// ---- launch ----------------------------------------------------------------------
cudaError_t encode_fp16_2d(CUtensorMap* out, const void* base, long inner, long rows, int box_inner, int box_rows);

template <int HD, bool Q8>
static cudaError_t launch_shared_as(const SharedArgs& a, const void* k, const void* v, int dev, cudaStream_t s) {
    static OncePerDevice once;
    cudaError_t e = once(dev, [] {
        return cudaFuncSetAttribute(shared_kernel<HD, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, SharedSmem<HD, Q8>::TOTAL);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap mk = {}, mv = {};
    if (!Q8) {
        if ((e = encode_fp16_2d(&mk, k, HD, a.rows, 64, a.box_runs * 16)) != cudaSuccess) return e;
        if ((e = encode_fp16_2d(&mv, v, HD, a.rows, 64, a.box_runs * 16)) != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(a.sets * a.side);
    cfg.blockDim = dim3(SH_THREADS);
    cfg.dynamicSmemBytes = SharedSmem<HD, Q8>::TOTAL;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, shared_kernel<HD, Q8>, a, mk, mv);
}

cudaError_t launch_shared(const SharedArgs& a, int hd, bool q8, const void* k, const void* v, int dev, cudaStream_t s) {
    if (q8) return launch_shared_as<128, true>(a, k, v, dev, s);
    return hd == 64 ? launch_shared_as<64, false>(a, k, v, dev, s) : launch_shared_as<128, false>(a, k, v, dev, s);
}

}  // namespace kd
