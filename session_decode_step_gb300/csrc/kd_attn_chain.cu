// kd_attn_chain.cu -- windowed attention over fp16 rows in one launch, for windows
// of up to WIN_CHAIN_ITEMS * 64 keys: no partial results in memory, no merge kernel.
//
// A row's visible keys of one KV head -- the leading ones, then the window, as one
// sequence -- are cut into pieces of 32; piece p belongs to chain p mod 2 NW, a
// running maximum and sum over its pieces in order, and the 2 NW chains are merged
// in order.  Pieces, chains and the merge depend on the row's own position, window
// and sinks, so the result does not depend on the batch.  Where two CTAs per (row,
// KV head) fit the GPU at once, a cluster of two takes them, a chain per warp, and
// merges through distributed shared memory; else one CTA, whose warps take a chain
// of the first half, then one of the second.
//
// Each warp copies its own pieces with 16-byte asynchronous copies into its own
// buffer (a K and a V part, the next piece's copied while this one is computed),
// placed as the 128-byte swizzle does, so the products are the split kernel's.
// Rows that do not exist are filled with zeros and never read.  No barrier is
// waited on, so nothing can run out and the call's fault word is only cleared.
//
// What bounds it: with few rows the latency of a piece (copy, scores, softmax,
// values) times the chain's length, and what one SM can draw (about 130 GB/s);
// with many the copies, of which an SM holds 192 KB in flight.  Against split and merge: one launch instead of two,
// and no 528-byte record per head and 64 keys written and read back.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kd_attn_common.cuh"

namespace kd {

constexpr int CH_KEYS = 32;          // keys per piece
constexpr int CH_KT = CH_KEYS / 16;  // 16-key MMA tiles of a piece

// Chains (warps) per CTA: as many as 192 KB of buffers and the registers of a group of 8 allow.
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
// All but the last committed group have landed, for every lane of the warp.
__device__ __forceinline__ void cp_wait_but_one() {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
}

// The other CTA of a cluster of two: its shared memory at the same offset, and a barrier of both.
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
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Bytes of the first half's records, which a single CTA keeps while its warps' buffers serve the second.
template <int HD>
__host__ __device__ constexpr int chain_record(int gq) { return gq * (HD + 4) * 4; }
template <int HD>
constexpr int chain_smem_bytes(int gq, bool pair) {
    return chain_warps(gq) * (ChainSmem<HD>::WARP + (pair ? 0 : chain_record<HD>(gq)));
}

template <int HD, int GQ, bool PAIR>
__global__ void __launch_bounds__(chain_warps(GQ) * 32, 1) attn_chain_kernel(const __grid_constant__ AttnWinArgs a) {
    using L = ChainSmem<HD>;
    constexpr int NW = chain_warps(GQ);
    constexpr int KS = HD / 16, NU = HD / 8, CH = HD / 8;  // k-steps, 8-dim tiles, 16-byte chunks of a row
    constexpr int NQ = GQ > 4 ? GQ / 4 : 1;                // N-tiles of heads
    extern __shared__ __align__(1024) uint8_t chain_smem[];
    tl_entry(a.tl);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int kvh = PAIR ? blockIdx.x >> 1 : blockIdx.x, b = blockIdx.y, rank = PAIR ? blockIdx.x & 1 : 0;
    uint8_t* mine = chain_smem + warp * L::WARP;
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
    auto issue = [&](int item, int part) {
        if (item < n_items) {
            const uint32_t dst = part ? vbase : kbase;
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
    // The warp's pieces: chain `first`, then (one CTA) the chain NW further.
    const int first = warp + rank * NW;
    auto after = [&](int item) {
        const int nx = item + 2 * NW;
        return PAIR || nx < n_items || item % (2 * NW) >= NW ? nx : first + NW;
    };
    // In the step the kernel before writes the new row and nothing else of the cache: a
    // piece without that row is fetched before the wait.
    const bool early = !append && (first + 1) * CH_KEYS < nvis;
    pdl_launch_dependents();
    if (!early) pdl_wait();
    issue(first, 0);
    issue(first, 1);
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
    // The chain's (o, m, l), heads HD + 4 floats apart.
    constexpr int REC = HD + 4;
    auto finish = [&](float* rec) {
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
                if (g == 0) *reinterpret_cast<float2*>(dst + HD) = make_float2(m[j], l[j]);
            }
        }
    };
    // Records: the CTA's last chains' in the warps' buffers, a single CTA's first ones' behind the buffers.
    float* kept = reinterpret_cast<float*>(chain_smem + NW * L::WARP + warp * chain_record<HD>(GQ));
    // the new row: converted, into the cache and into the warp's piece
    auto put_new = [&](int item, int part) {
        if (lane < CH) {
            const float* src = (part ? a.v_new : a.k_new) + ((size_t)b * a.nkv + kvh) * HD + 8 * lane;
            const uint4 w = make_uint4(f2_hi(src[0], src[1]), f2_hi(src[2], src[3]), f2_hi(src[4], src[5]), f2_hi(src[6], src[7]));
            *reinterpret_cast<uint4*>((__half*)(part ? a.v_dst : a.k_dst) + (row0 + pos) * HD + 8 * lane) = w;
            *reinterpret_cast<uint4*>(mine + part * L::PART + L::off(nvis - 1 - item * CH_KEYS, lane)) = w;
        }
        __syncwarp();
    };

    for (int item = first, nx; item < n_items; item = nx) {
        nx = after(item);
        const int n = min(CH_KEYS, nvis - item * CH_KEYS);
        const bool has_new = append && item == n_items - 1;
        cp_wait_but_one();  // the K part
        if (has_new) put_new(item, 0);
        float sacc[CH_KT][NQ][4];
#pragma unroll
        for (int t = 0; t < CH_KT; ++t)
#pragma unroll
            for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) sacc[t][j][i] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t ka[CH_KT][4];
#pragma unroll
            for (int t = 0; t < CH_KT; ++t)
                ldsm_x4(kbase + L::off(16 * t + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * ks + (lane >> 4)), ka[t][0], ka[t][1],
                        ka[t][2], ka[t][3]);
#pragma unroll
            for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int t = 0; t < CH_KT; ++t)
                    mma_16816_acc(sacc[t][j], ka[t][0], ka[t][1], ka[t][2], ka[t][3], qb[j][ks][0], qb[j][ks][1]);
        }
        __syncwarp();
        issue(nx, 0);  // the next piece's K part
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
        cp_wait_but_one();  // the V part
        if (has_new) put_new(item, 1);
        const int src0 = (2 * c) * 4 + colh, src1 = src0 + 4;
#pragma unroll
        for (int js = 0; js < CH_KT; ++js) {
            if (16 * js < n) {
                uint32_t pb[NQ][2];
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const float v00 = __shfl_sync(FULL_MASK, sv[j][js][0], src0), v01 = __shfl_sync(FULL_MASK, sv[j][js][0], src1);
                    const float v10 = __shfl_sync(FULL_MASK, sv[j][js][1], src0), v11 = __shfl_sync(FULL_MASK, sv[j][js][1], src1);
                    const bool on = 4 * j + colh < GQ;
                    pb[j][0] = !on ? 0u : (col_lo ? f2_lo(v00, v01) : f2_hi(v00, v01));
                    pb[j][1] = !on ? 0u : (col_lo ? f2_lo(v10, v11) : f2_hi(v10, v11));
                }
#pragma unroll
                for (int mt = 0; mt < NU / 2; ++mt) {
                    uint32_t va[4];
                    ldsm_x4_trans(vbase + L::off(16 * js + (lane >> 4) * 8 + (lane & 7), 2 * mt + ((lane >> 3) & 1)), va[0],
                                  va[1], va[2], va[3]);
#pragma unroll
                    for (int j = 0; j < NQ; ++j) mma_16816_acc(o[mt][j], va[0], va[1], va[2], va[3], pb[j][0], pb[j][1]);
                }
            }
        }
        __syncwarp();
        issue(nx, 1);  // the next piece's V part
        if (!PAIR && nx == first + NW && nx < n_items) {  // the first chain ends here
            finish(kept);
            start();
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    // The warp's last chain; one that only had a chain of the first half leaves it with those.
    static_assert(GQ * REC * 4 <= L::WARP, "a chain's record fits its buffer");
    if (!PAIR && first + NW >= n_items)
        finish(kept);
    else
        finish(reinterpret_cast<float*>(mine));

    // The merge, chains in order.  A single CTA holds all records; of a cluster, rank 0
    // those of chains 0 .. NW - 1, and each CTA merges half of the dims, after copying the
    // other's records of them behind its own.
    constexpr int RECORDS = chain_record<HD>(GQ);
    static_assert(2 * RECORDS <= L::WARP, "two records fit a buffer");
    const int chains = min(2 * NW, n_items);
    constexpr int MD = PAIR ? HD / 2 : HD;  // dims merged here
    const int d0 = PAIR ? rank * MD : 0;
    __shared__ float weight[GQ][2 * NW], denom[GQ];
    if (PAIR) {
        cluster_sync();
        // the other CTA's records of these dims, and its (m, l)
        const uint32_t buf0 = smem_u32(chain_smem);
        const int others = rank ? min(NW, n_items) : max(0, chains - NW);
        constexpr int QUADS = MD / 4 + 1;
        for (int t = threadIdx.x; t < others * GQ * QUADS; t += NW * 32) {
            const int q = t % QUADS, wh = t / QUADS, w = wh / GQ, h = wh - w * GQ;
            const int at = h * REC + (q < MD / 4 ? d0 + 4 * q : HD);
            const float4 v = ld_other4(buf0 + w * L::WARP + at * 4, rank ^ 1);
            *reinterpret_cast<float4*>(chain_smem + w * L::WARP + RECORDS + at * 4) = v;
        }
        asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // this CTA has read what it needs
    }
    __syncthreads();
    // Chain x's record.
    auto record = [&](int x) -> const float* {
        const int w = x < NW ? x : x - NW;
        if (PAIR) return reinterpret_cast<const float*>(chain_smem + w * L::WARP + ((x >= NW) != (rank != 0) ? RECORDS : 0));
        return reinterpret_cast<const float*>(x < NW ? chain_smem + NW * L::WARP + w * chain_record<HD>(GQ)
                                                     : chain_smem + w * L::WARP);
    };
    if (warp < GQ) {  // head `warp`: the chains' weights and the denominator
        static_assert(2 * NW <= 32 && GQ <= NW, "a lane per chain, a warp per head");
        const float2 ml = lane < chains ? *reinterpret_cast<const float2*>(record(lane) + warp * REC + HD)
                                        : make_float2(-INFINITY, 0.0f);
        float M = ml.x;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, x));
        const float e = lane < chains ? expf(__fsub_rn(ml.x, M == -INFINITY ? 0.0f : M)) : 0.0f;
        float den = __fmul_rn(e, ml.y);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) den = __fadd_rn(den, __shfl_xor_sync(FULL_MASK, den, x));
        if (lane < 2 * NW) weight[warp][lane] = e;
        if (lane == 0) denom[warp] = den;
    }
    __syncthreads();
    for (int t = threadIdx.x; t < GQ * MD; t += NW * 32) {
        const int h = t / MD, d = d0 + t - h * MD;
        float num = 0.0f;
#pragma unroll 4
        for (int x = 0; x < chains; ++x) num = __fmaf_rn(weight[h][x], record(x)[h * REC + d], num);
        a.out[(size_t)b * a.nh * HD + ((size_t)kvh * GQ + h) * HD + d] = __float2half_rn(__fdiv_rn(num, denom[h]));
    }
    if (PAIR) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the other has read this one's records
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

cudaError_t attn_chain_init_attributes() {
    cudaError_t e = cudaSuccess;
#define KD_SET_ONE(HD_, GQ_, PAIR_)                                                                                     \
    e = cudaFuncSetAttribute(attn_chain_kernel<HD_, GQ_, PAIR_>, cudaFuncAttributeMaxDynamicSharedMemorySize,           \
                             chain_smem_bytes<HD_>(GQ_, PAIR_));                                                        \
    if (e != cudaSuccess) return e;                                                                                     \
    e = cudaFuncSetAttribute(attn_chain_kernel<HD_, GQ_, PAIR_>, cudaFuncAttributePreferredSharedMemoryCarveout,        \
                             cudaSharedmemCarveoutMaxShared);                                                           \
    if (e != cudaSuccess) return e;
#define KD_SET(HD_, GQ_)           \
    KD_SET_ONE(HD_, GQ_, false)    \
    KD_SET_ONE(HD_, GQ_, true)
    for (int group : {1, 2, 4, 8}) {
        KD_CHAIN_GROUPS(64, KD_SET)
        KD_CHAIN_GROUPS(128, KD_SET)
    }
#undef KD_SET
#undef KD_SET_ONE
    return cudaSuccess;
}

cudaError_t launch_attn_chain(const AttnWinArgs& a, int max_keys, int num_sms, bool pdl, cudaStream_t s) {
    const int group = a.nh / a.nkv;
    // a cluster of two where both fit and a row has chains for the second
    const bool pair = 2L * a.nkv * a.B <= num_sms && max_keys > chain_warps(group) * CH_KEYS;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    if (pdl) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (pair) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = 2;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.gridDim = dim3(pair ? 2 * a.nkv : a.nkv, a.B);
    cfg.stream = s;
#define KD_LAUNCH(HD_, GQ_)                                                                                   \
    cfg.blockDim = dim3(chain_warps(GQ_) * 32);                                                               \
    cfg.dynamicSmemBytes = chain_smem_bytes<HD_>(GQ_, pair);                                                  \
    return pair ? cudaLaunchKernelEx(&cfg, attn_chain_kernel<HD_, GQ_, true>, a)                              \
                : cudaLaunchKernelEx(&cfg, attn_chain_kernel<HD_, GQ_, false>, a);
    if (a.hd == 64) { KD_CHAIN_GROUPS(64, KD_LAUNCH) } else if (a.hd == 128) { KD_CHAIN_GROUPS(128, KD_LAUNCH) }
#undef KD_LAUNCH
    return cudaErrorInvalidValue;
}

}  // namespace kd
