// kd_attn_chain.cu -- windowed attention over fp16 rows in one launch: KV append,
// attention and merge, with few or no partial results in memory.
//
// A row's visible keys of one KV head -- the leading ones, then the window, as one
// sequence -- are cut into pieces of 32; piece p belongs to chain p mod CHAINS, a
// running maximum and sum over its pieces in order, and the chains are merged in a
// fixed order.  Pieces, chains and the merge depend on the row's own position and on
// the slot's capacity, window and sinks, so the result does not depend on the batch:
// the chains of a (row, KV head) are taken by one CTA, each warp one after another,
// or by a cluster of 2, 4 or 8 where that many fit the GPU at once, down to a chain
// per warp; a cluster merges through distributed shared memory.
//
// Chains: 24 for capacities of up to WIN_CHAIN_ITEMS * 64 visible keys, 48 beyond (16
// and 32 for groups of 8 heads, whose accumulators leave room for 8 warps).  More make
// one row faster and many rows slower, as each ends in a record.  8192 keys of 8 KV
// heads of 128, 1 / 4 / 16 rows: 24 chains 15.5 / 25.6 / 80.8 us, 48 chains 11.1 / 25.0 /
// 84.9, 96 chains 10.8 / 25.1 / 91; at 2000 keys 24 chains 8.3 / 8.5 / 24.9, 48 chains
// 8.5 / 9.2 / 27.2.  64-key splits with a record each and a second launch that merges
// them: 12.2 / 26.9 / 95.1 and 6.9 / 11.1 / 27.5.
//
// Each warp copies its own pieces with 16-byte asynchronous copies into its own
// buffers (a K and a V part each; CTAs with fewer warps keep several pieces in flight),
// placed as the 128-byte swizzle does, so the products are the split kernel's.
// Rows that do not exist are filled with zeros and never read.  No mbarrier is
// waited on, so nothing can run out and the call's fault word is only cleared.
//
// What bounds it: with many rows HBM (16 rows over 8192 + 64 keys, 543 MB: 84.9 us,
// 6.4 TB/s; 8 rows over 20000 keys 6.7), of which an SM holds 192 KB in flight (128 KB in
// groups of 8; half of these for heads of 64); with few the chain's latency, about 1 us a
// piece (copy, scores, softmax, values), after 4 us of launch, first copies and merge.
// A deal that leaves a last round part empty costs as much as a full one: 8 rows of 24
// pieces 9.9 us, 25 11.7, 33 11.5, 48 13.1.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "kd_attn_common.cuh"
#include "kd_host.h"

namespace kd {

constexpr int CH_KEYS = 32;          // keys per piece
constexpr int CH_KT = CH_KEYS / 16;  // 16-key MMA tiles of a piece

// Chains (warps) per CTA: as many as 192 KB of buffers (heads of 128) and the registers of a group of 8 allow.
__host__ __device__ constexpr int chain_warps(int gq) { return gq == 8 ? 8 : 12; }

template <int HD>
struct ChainSmem {
    static constexpr int NREG = HD / 64;               // 64-dim halves of a row
    static constexpr int HALF_BYTES = CH_KEYS * 128;   // one half of a piece
    static constexpr int PART = NREG * HALF_BYTES;     // K or V of a piece
    static constexpr int WARP = 2 * PART;
    static __device__ __forceinline__ uint32_t off(int row, int chunk) {
        return (uint32_t)((chunk >> 3) * HALF_BYTES + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
    }
};

// 16 bytes from global to shared memory, or 16 zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N committed groups have landed, for every lane of the warp.
template <int N>
__device__ __forceinline__ void cp_wait_but() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncwarp();
}

// Another CTA of the cluster: its shared memory at the same offset, and a barrier of all.
__device__ __forceinline__ float4 ld_other4(uint32_t addr, uint32_t rank) {
    uint32_t ra;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(ra)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_other2(uint32_t addr, uint32_t rank) {
    uint32_t ra;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(ra) : "memory");
    return v;
}
__device__ __forceinline__ float ld_other(uint32_t addr, uint32_t rank) {
    uint32_t ra;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ra) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Bytes of a chain's record (its o by head, and m and l).
template <int HD>
__host__ __device__ constexpr int chain_record(int gq) { return gq * (HD + 4) * 4; }
// R chains per warp of a full CTA (chain_warps), shared by a cluster of CS: a CTA's warps,
// the chains that each takes one after another, and the pieces that it has in flight.
__host__ __device__ constexpr int chain_cta_warps(int gq, int r, int cs) { return cs > r ? chain_warps(gq) * r / cs : chain_warps(gq); }
__host__ __device__ constexpr int chain_turns(int r, int cs) { return cs > r ? 1 : r / cs; }
__host__ __device__ constexpr int chain_depth(int r, int cs) { return cs > r ? cs / r : 1; }
// The buffers, and behind them the records of the first turn while the buffers serve the others.
template <int HD>
constexpr int chain_smem_bytes(int gq, int r, int cs) {
    return chain_warps(gq) * (ChainSmem<HD>::WARP + (chain_turns(r, cs) > 1 ? chain_record<HD>(gq) : 0));
}

template <int HD, int GQ, int R, int CS>
__global__ void __launch_bounds__(chain_cta_warps(GQ, R, CS) * 32, 1)
    attn_chain_kernel(const __grid_constant__ AttnWinArgs a) {
    using L = ChainSmem<HD>;
    constexpr int NW = chain_cta_warps(GQ, R, CS), P = chain_turns(R, CS), D = chain_depth(R, CS);
    constexpr int CHAINS = R * chain_warps(GQ), AREA = D * L::WARP;
    static_assert(P == 1 || D == 1, "one or the other");
    constexpr int KS = HD / 16, NU = HD / 8, CH = HD / 8;  // k-steps, 8-dim tiles, 16-byte chunks of a row
    constexpr int NQ = GQ > 4 ? GQ / 4 : 1;                // N-tiles of heads
    extern __shared__ __align__(1024) uint8_t chain_smem[];
    tl_entry(a.tl);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int kvh = blockIdx.x / CS, b = blockIdx.y, rank = blockIdx.x % CS;
    uint8_t* mine = chain_smem + warp * AREA;
    const uint32_t kbase = smem_u32(mine), vbase = kbase + L::PART;

    const int pos = a.slot ? a.pos[b] : a.vpos[b], slot = a.slot ? a.slot[b] : a.vslot[b];
    // visible key v of nvis is row v (a leading key) or v + gap (the window's)
    const int lo = pos + 1 > a.window ? pos + 1 - a.window : 0, lead = min(a.sinks, lo), gap = lo - lead;
    const int nvis = pos + 1 - gap, n_items = (nvis + CH_KEYS - 1) / CH_KEYS;
    const size_t row0 = ((size_t)slot * a.nkv + kvh) * a.cap;
    const __half* kc = a.kc + row0 * HD;
    const __half* vc = a.vc + row0 * HD;
    const bool append = a.k_new != nullptr;
    const int nread = nvis - (append ? 1 : 0);  // the new row does not come from the cache
    // The lane's chunks of a piece: row j * ROWS + lane / CH, chunk lane % CH, j < CH.
    // Its place repeats the swizzle every 8 rows.
    constexpr int ROWS = 32 / CH, PER = 8 / ROWS;
    uint32_t place[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) place[j] = L::off(j * ROWS + lane / CH, lane % CH);
    auto issue = [&](int item, int part, int slot) {
        if (item < n_items) {
            const uint32_t dst = (part ? vbase : kbase) + slot * L::WARP;
            const int v0 = item * CH_KEYS;
            const __half* src = (part ? vc : kc) + (lane % CH) * 8;
            if (v0 >= lead && v0 + CH_KEYS <= nread) {  // 32 rows of the window: consecutive
                src += (size_t)(v0 + gap + lane / CH) * HD;
#pragma unroll
                for (int j = 0; j < CH; ++j)
                    cp_async16(dst + place[j % PER] + (j / PER) * 8 * 128, src + j * ROWS * HD, true);
            } else {
#pragma unroll 4
                for (int j = 0; j < CH; ++j) {
                    const int v = v0 + j * ROWS + lane / CH;
                    const bool have = v < nread;
                    cp_async16(dst + place[j % PER] + (j / PER) * 8 * 128,
                               src + (have ? (size_t)(v < lead ? v : v + gap) * HD : 0), have);
                }
            }
        }
        cp_commit();
    };
    // Piece p belongs to chain p mod CHAINS; the warp's chains are first, first + NW, ...
    const int first = rank * P * NW + warp;
    // In the step the kernel before writes the new row and nothing else of the cache:
    // pieces without that row are fetched before the wait.
    const bool early = !append && (first + (D - 1) * CHAINS + 1) * CH_KEYS < nvis;
    pdl_launch_dependents();
    if (!early) pdl_wait();
#pragma unroll
    for (int d = 0; d < D; ++d) {
        issue(first + d * CHAINS, 0, d);
        issue(first + d * CHAINS, 1, d);
    }
    if (early) pdl_wait();
    tl_waited(a.tl);
    if (a.clear_err && b == 0 && blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;

    // B fragments of Q^T, as in the split kernel: column 2h + part of N-tile j is head
    // 4j + h, part 0 the fp16 rounding of q, part 1 what it left over.
    const int colh = g >> 1;
    const bool col_lo = (g & 1) != 0;
    uint32_t qb[NQ][KS][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int h = 4 * j + colh;
        const bool on = h < GQ;
        const float* qp = a.q + ((size_t)b * a.nh + (size_t)kvh * GQ + (on ? h : 0)) * HD + 2 * c;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const float2 u = *reinterpret_cast<const float2*>(qp + 16 * ks), w = *reinterpret_cast<const float2*>(qp + 16 * ks + 8);
            qb[j][ks][0] = !on ? 0u : (col_lo ? f2_lo(u.x, u.y) : f2_hi(u.x, u.y));
            qb[j][ks][1] = !on ? 0u : (col_lo ? f2_lo(w.x, w.y) : f2_hi(w.x, w.y));
        }
    }
    // The chain: m the running maximum of head 4j + c, l the lane's part of its sum, o = sum p v.
    float m[NQ], l[NQ], o[NU / 2][NQ][4];
    auto start = [&]() {
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
    start();
    // The chain's o, heads HD + 4 floats apart, and its (m, l) behind it or to ml.
    constexpr int REC = HD + 4, RECORDS = chain_record<HD>(GQ);
    auto finish = [&](float* rec, float2* ml) {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[j] = __fadd_rn(l[j], __shfl_xor_sync(FULL_MASK, l[j], x));
            const int h = 4 * j + c;
            if (h < GQ) {
                float* dst = rec + h * REC;
#pragma unroll
                for (int mt = 0; mt < NU / 2; ++mt) {
                    dst[16 * mt + g] = __fadd_rn(o[mt][j][0], o[mt][j][1]);
                    dst[16 * mt + g + 8] = __fadd_rn(o[mt][j][2], o[mt][j][3]);
                }
                if (g == 0) *(ml ? ml + h : reinterpret_cast<float2*>(dst + HD)) = make_float2(m[j], l[j]);
            }
        }
    };
    // The records of a turn, and the floats from warp to warp: the last in the buffers' place
    // (with R == 2 at the CTA's rank, as the merge copies the others' there), the first
    // behind the buffers, the others in the workspace, which has 24 records a head.
    __shared__ float2 chain_ml[R > 2 ? CHAINS * GQ : 1];
    auto records = [&](int turn, int& stride) -> float* {
        if (turn == P - 1) {
            stride = AREA / 4;
            return reinterpret_cast<float*>(chain_smem + (R == 2 ? rank * RECORDS : 0));
        }
        stride = GQ * REC;
        if (turn == 0) return reinterpret_cast<float*>(chain_smem + NW * AREA);
        return a.part + (((size_t)b * a.nh + (size_t)kvh * GQ) * a.max_splits + (size_t)(turn - 1) * NW * GQ) * REC;
    };
    auto store = [&](int turn) {
        int stride;
        float* rec = records(turn, stride);
        finish(rec + warp * stride, R > 2 ? chain_ml + ((rank * P + turn) * NW + warp) * GQ : nullptr);
    };
    // the new row: converted, into the cache and into the warp's piece
    auto put_new = [&](int item, int part, int slot) {
        if (lane < CH) {
            const float* src = (part ? a.v_new : a.k_new) + ((size_t)b * a.nkv + kvh) * HD + 8 * lane;
            const uint4 w = make_uint4(f2_hi(src[0], src[1]), f2_hi(src[2], src[3]), f2_hi(src[4], src[5]), f2_hi(src[6], src[7]));
            *reinterpret_cast<uint4*>((__half*)(part ? a.v_dst : a.k_dst) + (row0 + pos) * HD + 8 * lane) = w;
            *reinterpret_cast<uint4*>(mine + slot * L::WARP + part * L::PART + L::off(nvis - 1 - item * CH_KEYS, lane)) = w;
        }
        __syncwarp();
    };

    int turn = 0;
    for (int item = first, nx, slot = 0; item < n_items; item = nx, slot = D > 1 ? (slot + 1) % D : 0) {
        nx = item + CHAINS;
        const bool ends = P > 1 && turn + 1 < P && nx >= n_items;  // a chain before the warp's last
        if (ends) nx = first + (turn + 1) * NW;
        const int fetch = D > 1 ? item + D * CHAINS : nx;  // the piece that takes this one's place
        const uint32_t kb = kbase + slot * L::WARP, vb = vbase + slot * L::WARP;
        const int n = min(CH_KEYS, nvis - item * CH_KEYS);
        const bool has_new = append && item == n_items - 1;
        cp_wait_but<2 * D - 1>();  // the K part
        if (has_new) put_new(item, 0, slot);
        float sacc[CH_KT][NQ][4];
#pragma unroll
        for (int t = 0; t < CH_KT; ++t)
#pragma unroll
            for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) sacc[t][j][i] = 0.0f;
        uint32_t ka[2][CH_KT][4];  // a k-step's keys, fetched a step ahead
        auto load_k = [&](int ks) {
#pragma unroll
            for (int t = 0; t < CH_KT; ++t) {
                uint32_t(&k)[4] = ka[ks & 1][t];
                ldsm_x4(kb + L::off(16 * t + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * ks + (lane >> 4)), k[0], k[1], k[2], k[3]);
            }
        };
        load_k(0);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks + 1 < KS) load_k(ks + 1);
#pragma unroll
            for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int t = 0; t < CH_KT; ++t) {
                    const uint32_t(&k)[4] = ka[ks & 1][t];
                    mma_16816_acc(sacc[t][j], k[0], k[1], k[2], k[3], qb[j][ks][0], qb[j][ks][1]);
                }
        }
        __syncwarp();
        issue(fetch, 0, slot);
        // Softmax of head 4j + c over keys 16t + g and 16t + g + 8; the weights are taken
        // against the new running maximum (0 while every score is -inf).
        float sv[NQ][CH_KT][2], f[NQ];
        bool same = true;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            float mx = m[j];
#pragma unroll
            for (int t = 0; t < CH_KT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float sc = __fadd_rn(sacc[t][j][2 * e], sacc[t][j][2 * e + 1]);  // both parts
                    sv[j][t][e] = 16 * t + g + 8 * e < n ? __fmul_rn(sc, a.scale) : -INFINITY;
                    mx = fmaxf(mx, sv[j][t][e]);
                }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, x));
            const float ref = mx == -INFINITY ? 0.0f : mx;
            f[j] = m[j] == mx ? 1.0f : expf(__fsub_rn(m[j], ref));
            same = same && f[j] == 1.0f;
            m[j] = mx;
            float s = 0.0f;
#pragma unroll
            for (int t = 0; t < CH_KT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sv[j][t][e] = 16 * t + g + 8 * e < n ? expf(__fsub_rn(sv[j][t][e], ref)) : 0.0f;
                    s = __fadd_rn(s, sv[j][t][e]);
                }
            l[j] = __fmaf_rn(l[j], f[j], s);
        }
        if (__any_sync(FULL_MASK, !same)) {
#pragma unroll
            for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int mt = 0; mt < NU / 2; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][j][i] = __fmul_rn(o[mt][j][i], f[j]);
        }
        cp_wait_but<2 * D - 1>();  // the V part
        if (has_new) put_new(item, 1, slot);
        const int src0 = (2 * c) * 4 + colh, src1 = src0 + 4;
#pragma unroll
        for (int js = 0; js < CH_KT; ++js) {
            if (16 * js < n) {
                constexpr int VB = 4;  // 16-dim tiles fetched at a time
                uint32_t va[VB][4];
                auto load_v = [&](int mt0) {
#pragma unroll
                    for (int u = 0; u < VB; ++u)
                        ldsm_x4_trans(vb + L::off(16 * js + (lane >> 4) * 8 + (lane & 7), 2 * (mt0 + u) + ((lane >> 3) & 1)),
                                      va[u][0], va[u][1], va[u][2], va[u][3]);
                };
                load_v(0);
                uint32_t pb[NQ][2];
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const float v00 = __shfl_sync(FULL_MASK, sv[j][js][0], src0), v01 = __shfl_sync(FULL_MASK, sv[j][js][0], src1);
                    const float v10 = __shfl_sync(FULL_MASK, sv[j][js][1], src0), v11 = __shfl_sync(FULL_MASK, sv[j][js][1], src1);
                    const bool on = 4 * j + colh < GQ;
                    pb[j][0] = !on ? 0u : (col_lo ? f2_lo(v00, v01) : f2_hi(v00, v01));
                    pb[j][1] = !on ? 0u : (col_lo ? f2_lo(v10, v11) : f2_hi(v10, v11));
                }
                static_assert(NU / 2 % VB == 0, "whole groups of tiles");
#pragma unroll
                for (int mt0 = 0; mt0 < NU / 2; mt0 += VB) {
                    if (mt0) load_v(mt0);
#pragma unroll
                    for (int u = 0; u < VB; ++u)
#pragma unroll
                        for (int j = 0; j < NQ; ++j)
                            mma_16816_acc(o[mt0 + u][j], va[u][0], va[u][1], va[u][2], va[u][3], pb[j][0], pb[j][1]);
                }
            }
        }
        __syncwarp();
        issue(fetch, 1, slot);
        if (ends && nx < n_items) {
            store(turn++);
            start();
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    static_assert((R == 2 ? CS * RECORDS : RECORDS + GQ * HD * 4) <= AREA, "records, or a record and a sum, fit a warp's buffers");
    if (first < n_items) store(turn);

    const int chains = min(CHAINS, n_items);
    // The merge.  No cluster size changes a bit of it.
    if constexpr (R > 2) {
        // M = max m_x, out = sum_x e^{m_x - M} o_x / sum_x e^{m_x - M} l_x: each CTA sums groups of
        // its chains, in order, and the groups' sums are added in order.
        if (CS > 1) {
            cluster_sync();
            for (int e = threadIdx.x; e < chains * GQ; e += NW * 32) {
                const int owner = e / (P * NW * GQ);
                if (owner != rank) chain_ml[e] = ld_other2(smem_u32(chain_ml + e), owner);
            }
        }
        __syncthreads();
        __shared__ float weight[GQ][CHAINS], denom[GQ];
        for (int h = warp; h < GQ; h += NW) {  // the chains' weights and the denominator, a warp per head
            constexpr int NL = (CHAINS + 31) / 32;
            float2 v[NL];
            float M = -INFINITY;
#pragma unroll
            for (int q = 0; q < NL; ++q) {
                const int x = lane + 32 * q;
                v[q] = x < chains ? chain_ml[x * GQ + h] : make_float2(-INFINITY, 0.0f);
                M = fmaxf(M, v[q].x);
            }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, x));
            const float ref = M == -INFINITY ? 0.0f : M;
            float den = 0.0f;
#pragma unroll
            for (int q = 0; q < NL; ++q) {
                const int x = lane + 32 * q;
                if (32 * q < chains) {
                    const float e = x < chains ? expf(__fsub_rn(v[q].x, ref)) : 0.0f;
                    if (x < chains) weight[h][x] = e;
                    den = __fmaf_rn(e, v[q].y, den);
                }
            }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) den = __fadd_rn(den, __shfl_xor_sync(FULL_MASK, den, x));
            if (lane == 0) denom[h] = den;
        }
        __syncthreads();
        // Groups of chains: their weighted sums, in the buffers behind the records.
        constexpr int G = CHAINS / 8, GROUPS = 8 / CS, QUADS = GQ * HD / 4;
        static_assert(NW % G == 0, "a group's chains are of one turn");
        auto sums = [&](int p) { return chain_smem + p * AREA + RECORDS; };
        static_assert(GROUPS <= NW, "a sum per warp's buffers");
        for (int u = threadIdx.x; u < GROUPS * QUADS; u += NW * 32) {
            const int p = u / QUADS, q = u - p * QUADS, h = q / (HD / 4), x0 = (rank * GROUPS + p) * G, n = chains - x0;
            int stride;
            const float* rec = records(p * G / NW, stride);
            rec += p * G % NW * stride + h * REC + 4 * (q % (HD / 4));
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float4 v[G];
#pragma unroll
            for (int w = 0; w < G; ++w)
                if (w < n) v[w] = *reinterpret_cast<const float4*>(rec + w * stride);
#pragma unroll
            for (int w = 0; w < G; ++w)
                if (w < n) {
                    const float e = weight[h][x0 + w];
                    acc.x = __fmaf_rn(e, v[w].x, acc.x);
                    acc.y = __fmaf_rn(e, v[w].y, acc.y);
                    acc.z = __fmaf_rn(e, v[w].z, acc.z);
                    acc.w = __fmaf_rn(e, v[w].w, acc.w);
                }
            *reinterpret_cast<float4*>(sums(p) + 16 * q) = acc;
        }
        if (CS > 1)
            cluster_sync();
        else
            __syncthreads();
        // every CTA of the cluster writes its share of the heads' dims
        constexpr int SHARE = GQ * HD / CS;
        const int used = (chains + G - 1) / G;
        for (int t = threadIdx.x; t < SHARE; t += NW * 32) {
            const int i = rank * SHARE + t;
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < used) {
                    const uint8_t* at = sums(r % GROUPS) + 4 * i;
                    v[r] = CS > 1 ? ld_other(smem_u32(at), r / GROUPS) : *reinterpret_cast<const float*>(at);
                }
            float num = v[0];
#pragma unroll
            for (int r = 1; r < 8; ++r)
                if (r < used) num = __fadd_rn(num, v[r]);
            a.out[(size_t)b * a.nh * HD + (size_t)kvh * GQ * HD + i] = __float2half_rn(__fdiv_rn(num, denom[i / HD]));
        }
        if (CS > 1) cluster_sync();  // the others have read this one's sums
    } else {
        // The merge, chains in order.  A single CTA holds all records; of a cluster each CTA
        // merges its share of the dims, after copying the others' records of them to its own:
        // chain x, of warp w of CTA r, is in warp w's buffers at r records' distance.
        constexpr int MD = HD / CS;  // dims merged here
        const int d0 = rank * MD;
        __shared__ float weight[GQ][CHAINS], denom[GQ];
        if (CS > 1) {
            cluster_sync();
            // the other CTAs' records of these dims, and their (m, l)
            const uint32_t buf0 = smem_u32(chain_smem);
            constexpr int QUADS = MD / 4 + 1;
            for (int t = threadIdx.x; t < chains * GQ * QUADS; t += NW * 32) {
                const int q = t % QUADS, xh = t / QUADS, x = xh / GQ, h = xh - x * GQ, r = x / NW;
                const int at = (x - r * NW) * AREA + r * RECORDS + (h * REC + (q < MD / 4 ? d0 + 4 * q : HD)) * 4;
                if (r != rank) *reinterpret_cast<float4*>(chain_smem + at) = ld_other4(buf0 + at, r);
            }
            __syncwarp();
            asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // this CTA has read what it needs
        }
        __syncthreads();
        // Chain x's record.
        auto record = [&](int x) -> const float* {
            const int r = x / NW, w = x - r * NW;
            if (CS > 1) return reinterpret_cast<const float*>(chain_smem + w * AREA + r * RECORDS);
            return reinterpret_cast<const float*>(r == 0 ? chain_smem + NW * AREA + w * RECORDS : chain_smem + w * AREA);
        };
        for (int h = warp; h < GQ; h += NW) {  // the chains' weights and the denominator, a warp per head
            static_assert(CHAINS <= 32, "a lane per chain");
            const float2 ml = lane < chains ? *reinterpret_cast<const float2*>(record(lane) + h * REC + HD)
                                            : make_float2(-INFINITY, 0.0f);
            float M = ml.x;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, x));
            const float e = lane < chains ? expf(__fsub_rn(ml.x, M == -INFINITY ? 0.0f : M)) : 0.0f;
            float den = __fmul_rn(e, ml.y);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) den = __fadd_rn(den, __shfl_xor_sync(FULL_MASK, den, x));
            if (lane < CHAINS) weight[h][lane] = e;
            if (lane == 0) denom[h] = den;
        }
        __syncthreads();
        for (int t = threadIdx.x; t < GQ * MD; t += NW * 32) {
            const int h = t / MD, d = d0 + t - h * MD;
            float num = 0.0f;
#pragma unroll 8
            for (int x = 0; x < chains; ++x) num = __fmaf_rn(weight[h][x], record(x)[h * REC + d], num);
            a.out[(size_t)b * a.nh * HD + ((size_t)kvh * GQ + h) * HD + d] = __float2half_rn(__fdiv_rn(num, denom[h]));
        }
        __syncwarp();
        if (CS > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the others have read this one's records
    }
    tl_exit(a.tl);
}

#define KD_CHAIN_GROUPS(HD_, MACRO)      \
    switch (group) {                     \
        case 1: MACRO(HD_, 1); break;    \
        case 2: MACRO(HD_, 2); break;    \
        case 4: MACRO(HD_, 4); break;    \
        case 8: MACRO(HD_, 8); break;    \
        default: return cudaErrorInvalidValue; \
    }

// The kernel's attributes on device dev (the current one), set before its first launch there: a process
// uses few of the 64 kernels, and setting all of them up took 10 ms.
template <int HD, int GQ, int R, int CS>
static cudaError_t chain_attributes(int dev) {
    static OncePerDevice once;
    return once(dev, [] {
        const cudaError_t e = cudaFuncSetAttribute(attn_chain_kernel<HD, GQ, R, CS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   chain_smem_bytes<HD>(GQ, R, CS));
        if (e != cudaSuccess) return e;
        return cudaFuncSetAttribute(attn_chain_kernel<HD, GQ, R, CS>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                    cudaSharedmemCarveoutMaxShared);
    });
}
template <int HD, int GQ, int R>
static cudaError_t chain_attributes_all(int dev) {
    cudaError_t e = chain_attributes<HD, GQ, R, 1>(dev);
    if (e == cudaSuccess) e = chain_attributes<HD, GQ, R, 2>(dev);
    if (e == cudaSuccess) e = chain_attributes<HD, GQ, R, 4>(dev);
    if (e == cudaSuccess) e = chain_attributes<HD, GQ, R, 8>(dev);
    return e;
}

// Launch on clusters of CS, or, with `most`, ask how many of them the GPU holds at once.
template <int HD, int GQ, int R, int CS>
static cudaError_t launch_chain(const AttnWinArgs& a, int dev, bool pdl, cudaStream_t s, int* most = nullptr) {
    const cudaError_t e = chain_attributes<HD, GQ, R, CS>(dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    if (CS > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = CS;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    if (pdl && !most) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.gridDim = dim3(CS * a.nkv, a.B);
    cfg.blockDim = dim3(chain_cta_warps(GQ, R, CS) * 32);
    cfg.dynamicSmemBytes = chain_smem_bytes<HD>(GQ, R, CS);
    cfg.stream = s;
    if (most) return cudaOccupancyMaxActiveClusters(most, attn_chain_kernel<HD, GQ, R, CS>, &cfg);
    return cudaLaunchKernelEx(&cfg, attn_chain_kernel<HD, GQ, R, CS>, a);
}

// The largest cluster of which all fit the GPU at once and every CTA has a chain to take.
template <int HD, int GQ, int R>
static cudaError_t launch_chain(const AttnWinArgs& a, int max_keys, int dev, int num_sms, bool pdl, cudaStream_t s) {
    static std::atomic<int> fit[2];  // clusters of 8 and 4 at once, asked once
    const int units = a.nkv * a.B, pieces = (max_keys + CH_KEYS - 1) / CH_KEYS;
    if (pieces <= chain_warps(GQ) || 2 * units > num_sms) return launch_chain<HD, GQ, R, 1>(a, dev, pdl, s);
    if (pieces > 2 * chain_warps(GQ))
        for (int k = 0; k < 2; ++k) {
            if (units * (8 >> k) > num_sms) continue;
            int most = fit[k].load(std::memory_order_relaxed);
            if (!most) {
                const cudaError_t e = k == 0 ? launch_chain<HD, GQ, R, 8>(a, dev, pdl, s, &most)
                                             : launch_chain<HD, GQ, R, 4>(a, dev, pdl, s, &most);
                if (e != cudaSuccess) return e;
                if (most < 1) most = -1;
                fit[k].store(most, std::memory_order_relaxed);
            }
            if (units <= most)
                return k == 0 ? launch_chain<HD, GQ, R, 8>(a, dev, pdl, s) : launch_chain<HD, GQ, R, 4>(a, dev, pdl, s);
        }
    return launch_chain<HD, GQ, R, 2>(a, dev, pdl, s);
}

#define KD_CHAIN_SHAPES(M2, M4)                                       \
    const bool wide = max_splits > WIN_CHAIN_ITEMS;                   \
    if (hd == 128 && wide) {                                          \
        KD_CHAIN_GROUPS(128, M4)                                      \
    } else if (hd == 128) {                                           \
        KD_CHAIN_GROUPS(128, M2)                                      \
    } else if (hd == 64 && wide) {                                    \
        KD_CHAIN_GROUPS(64, M4)                                       \
    } else if (hd == 64) {                                            \
        KD_CHAIN_GROUPS(64, M2)                                       \
    }                                                                 \
    return cudaErrorInvalidValue;

cudaError_t attn_chain_prepare(int hd, int group, int max_splits, int dev) {
#define KD_PREPARE_2(HD_, GQ_) return chain_attributes_all<HD_, GQ_, 2>(dev)
#define KD_PREPARE_4(HD_, GQ_) return chain_attributes_all<HD_, GQ_, 4>(dev)
    KD_CHAIN_SHAPES(KD_PREPARE_2, KD_PREPARE_4)
#undef KD_PREPARE_4
#undef KD_PREPARE_2
}

cudaError_t launch_attn_chain(const AttnWinArgs& a, int max_keys, int dev, int num_sms, bool pdl, cudaStream_t s) {
    const int hd = a.hd, group = a.nh / a.nkv, max_splits = a.max_splits;
#define KD_LAUNCH_2(HD_, GQ_) return launch_chain<HD_, GQ_, 2>(a, max_keys, dev, num_sms, pdl, s)
#define KD_LAUNCH_4(HD_, GQ_) return launch_chain<HD_, GQ_, 4>(a, max_keys, dev, num_sms, pdl, s)
    KD_CHAIN_SHAPES(KD_LAUNCH_2, KD_LAUNCH_4)
#undef KD_LAUNCH_4
#undef KD_LAUNCH_2
}

}  // namespace kd
