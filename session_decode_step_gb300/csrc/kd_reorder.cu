// kd_reorder.cu -- sessions' caches permuted, forked and joined in place.
//
// dst_i := src_i for all i at once, the same slots on both sides (what a beam
// selection asks for: beams trade places, some parents are taken several times,
// some not at all).  Byte x of one slot's (layer, head) slab only ever depends on
// byte x of others, so a thread that owns one piece of the slab in every slot of
// a set of connected moves can make them all without a second buffer: it loads
// before it stores.  Sets of up to four moves (eight where few bytes move) are loaded
// whole; for larger ones, taken so many moves at a time, the host orders the moves so that a slot is read
// before it is overwritten, and as a set has at most one cycle (every destination
// has one source), one overwritten piece held in a register is enough.
//
// No arithmetic: bound by HBM, one read per source row (a row taken several
// times comes from L1 the second time) and one write per destination row.  What
// it takes is bytes in flight: a thread issues 8 loads of 16 bytes before it
// waits for the first -- over 8 pieces of one move, 4 of two, 2 of four or 1 of eight
// moves at a time, whichever fits the set.  32 layers of fp16 K and V, 8 sessions of 1238
// rows, 974 MB read and written: 142 us, 6.85 TB/s, a copy's rate.  A Q8_0 cache's
// windows (430 MB): 68 us, 6.3 TB/s; its scale rows are 8 bytes, so loads are.
#include <cuda_runtime.h>

#include "kd_device.cuh"
#include "kd_host.h"
#include "kd_reorder.h"

namespace kd {

constexpr int RO_THREADS = 256;
constexpr long RO_EIGHT_BYTES = 32 << 20;  // moved, up to which sets are taken by eights
constexpr int RO_FULL = 3 * 152;  // blocks resident at once: 3 per SM keep 80 registers, so the loads of a set stay in flight

struct ReorderMove {
    int dst, src;  // src -1: the piece held from the cycle's first destination
    int lo, len;   // it moves rows t < len that are leading rows (t < sinks) or t >= lo
    int hold;      // hold the destination's old piece first
};
// One range of rows of one connected set: all leading rows, or none.
struct ReorderRange {
    int first, count;   // its set's moves
    int lo, hi;         // rows [lo, hi)
    int all_lo, all_hi; // of these, the rows that every move of the set covers
    int leading, kind;
    int run0[4];        // runs of tiles before it, per plane
};
// CAP: the most moves (a call's parameters are copied at every launch, so small
// calls take the small form).
template <int CAP>
struct ReorderArgs {
    ReorderPlane plane[4];
    int plane0[4];  // first run (blockIdx.x) of each plane
    int n_planes, slots, heads, cap;
    int n_ranges, runs;
    int run;        // consecutive tiles a block makes
    ReorderRange range[2 * CAP];
    ReorderMove move[CAP];
};

// How a set's moves are taken: MB at a time, P pieces of each: (1, 8), (2, 4), (4, 2) and (8, 1),
// with a held piece (4, 1) or (8, 1).  Eights are for calls of few bytes, which wait for each batch
// of moves in turn (16 moves of up to 33 rows, 19 layers of Q8_0: 5.7 us against 7.5 in fours; 16 of
// 837 rows, 1 layer: 3.3, 6.7); many bytes are the slower so (11 moves, 45 MB: 22.3, 19.5).
// Their kernel leaves them the registers.
enum ReorderKind : int { RO_ONE, RO_TWO, RO_FOUR, RO_EIGHT, RO_CYCLE };
__host__ __device__ constexpr int reorder_pieces(int kind) {
    return kind == RO_ONE ? 8 : kind == RO_TWO ? 4 : kind == RO_FOUR ? 2 : 1;
}

// One tile of a range: pieces x0, x0 + stride, ... of the slab.  ALL: every move
// covers all of them (almost every tile), so nothing is compared.
template <typename T, int MB, int P, bool CYC, bool ALL>
__device__ __forceinline__ void reorder_tile(const ReorderMove* moves, const ReorderRange& s, char* slab, size_t slot_bytes,
                                             int row_bytes, int x0) {
    constexpr int STRIDE = RO_THREADS * (int)sizeof(T);
    const int hi = s.hi * row_bytes;
    auto covers = [&](const ReorderMove& m, int o) {
        return ALL || (o >= (s.leading ? 0 : m.lo * row_bytes) && o < min(m.len * row_bytes, hi));
    };
    slab += x0;
    T held[P] = {};
#pragma unroll 1
    for (int m0 = 0; m0 < s.count; m0 += MB) {
        T x[MB][P];
#pragma unroll
        for (int u = 0; u < MB; ++u)
            if (m0 + u < s.count) {
                const ReorderMove& m = moves[s.first + m0 + u];
                const char* src = slab + m.src * slot_bytes;
                if (CYC && m.hold) {
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        if (ALL || x0 + j * STRIDE < hi)
                            held[j] = *reinterpret_cast<const T*>(slab + m.dst * slot_bytes + j * STRIDE);
                }
                if (CYC && m.src < 0) {
#pragma unroll
                    for (int j = 0; j < P; ++j) x[u][j] = held[j];
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        if (covers(m, x0 + j * STRIDE)) x[u][j] = *reinterpret_cast<const T*>(src + j * STRIDE);
                }
            }
#pragma unroll
        for (int u = 0; u < MB; ++u)
            if (m0 + u < s.count) {
                const ReorderMove& m = moves[s.first + m0 + u];
                char* dst = slab + m.dst * slot_bytes;
#pragma unroll
                for (int j = 0; j < P; ++j)
                    if (covers(m, x0 + j * STRIDE)) *reinterpret_cast<T*>(dst + j * STRIDE) = x[u][j];
            }
    }
}

template <typename T, int MB, int P, bool CYC>
__device__ __forceinline__ void reorder_run(const ReorderMove* moves, const ReorderRange& s, char* slab, size_t slot_bytes,
                                            int row_bytes, int tile, int tiles) {
    constexpr int TILE = P * RO_THREADS * (int)sizeof(T);
#pragma unroll 1
    for (int k = 0; k < tiles; ++k) {
        const int t0 = s.lo * row_bytes + (tile + k) * TILE, x0 = t0 + (int)threadIdx.x * (int)sizeof(T);
        if (t0 >= s.hi * row_bytes) return;
        if (t0 >= s.all_lo * row_bytes && t0 + TILE <= s.all_hi * row_bytes)
            reorder_tile<T, MB, P, CYC, true>(moves, s, slab, slot_bytes, row_bytes, x0);
        else
            reorder_tile<T, MB, P, CYC, false>(moves, s, slab, slot_bytes, row_bytes, x0);
    }
}

template <typename T, int BATCH>
__device__ __forceinline__ void reorder_plane(const ReorderMove* moves, const ReorderRange& s, char* slab, size_t slot_bytes,
                                              int row_bytes, int tile, int tiles) {
    if (s.kind == RO_ONE)
        reorder_run<T, 1, 8, false>(moves, s, slab, slot_bytes, row_bytes, tile, tiles);
    else if (s.kind == RO_TWO)
        reorder_run<T, 2, 4, false>(moves, s, slab, slot_bytes, row_bytes, tile, tiles);
    else if (s.kind == RO_FOUR)
        reorder_run<T, 4, 2, false>(moves, s, slab, slot_bytes, row_bytes, tile, tiles);
    else if (BATCH == 8 && s.kind == RO_EIGHT)
        reorder_run<T, 8, 1, false>(moves, s, slab, slot_bytes, row_bytes, tile, tiles);
    else
        reorder_run<T, BATCH, 1, true>(moves, s, slab, slot_bytes, row_bytes, tile, tiles);
}

// Block (x, y): run x of the planes' ranges' tiles, (layer, head) y.
template <int CAP, int BATCH>
__global__ void __launch_bounds__(RO_THREADS, BATCH == 8 ? 2 : 3)
    kv_reorder_kernel(const __grid_constant__ ReorderArgs<CAP> a) {
    pdl_launch_dependents();
    int p = 0;
    while (p + 1 < a.n_planes && (int)blockIdx.x >= a.plane0[p + 1]) ++p;
    const int t = (int)blockIdx.x - a.plane0[p];
    int c = 0;
    while (c + 1 < a.n_ranges && t >= a.range[c + 1].run0[p]) ++c;
    const ReorderRange& s = a.range[c];
    const int row_bytes = a.plane[p].row_bytes;
    const int layer = blockIdx.y / a.heads, head = blockIdx.y - layer * a.heads;
    const size_t slab_bytes = (size_t)a.cap * row_bytes, slot_bytes = slab_bytes * a.heads;
    char* slab = (char*)a.plane[p].base + (size_t)layer * a.slots * slot_bytes + head * slab_bytes;
    const int tile = (t - s.run0[p]) * a.run;
    pdl_wait();
    if (row_bytes % 16 == 0)
        reorder_plane<uint4, BATCH>(a.move, s, slab, slot_bytes, row_bytes, tile, a.run);
    else
        reorder_plane<uint2, BATCH>(a.move, s, slab, slot_bytes, row_bytes, tile, a.run);
}

// Order the moves into connected sets (see the file comment), to be taken at most `batch` (4 or 8) at a time.
template <int CAP>
static void plan_moves(const ReorderPlan& p, const int32_t* dst, const int32_t* src, const int32_t* len, int n, int batch,
                       ReorderArgs<CAP>& a) {
    constexpr int N = CAP;
    int id[N], m = 0;  // the moves that move something
    for (int i = 0; i < n; ++i)
        if (dst[i] != src[i] && len[i] > 0) id[m++] = i;
    int next[N], before[N] = {}, set[N];
    for (int i = 0; i < m; ++i) {
        next[i] = -1;
        set[i] = i;
    }
    auto find = [&](int x) {
        while (set[x] != x) x = set[x] = set[set[x]];
        return x;
    };
    for (int i = 0; i < m; ++i)
        for (int j = 0; j < m; ++j) {
            if (dst[id[j]] == src[id[i]]) {  // j overwrites what i reads: i goes first
                next[i] = j;
                ++before[j];
                set[find(i)] = find(j);
            }
            if (src[id[j]] == src[id[i]]) set[find(i)] = find(j);  // one source: together, so it is read once
        }
    int order[N], no = 0;  // moves nothing waits for, then those they release
    for (int i = 0; i < m; ++i)
        if (!before[i]) order[no++] = i;
    for (int k = 0; k < no; ++k) {
        const int j = next[order[k]];
        if (j >= 0 && --before[j] == 0) order[no++] = j;
    }
    bool hold[N] = {}, from_held[N] = {}, done[N] = {};
    for (int k = 0; k < no; ++k) done[order[k]] = true;
    for (int i = 0; i < m; ++i)
        if (!done[i]) {  // a cycle
            hold[i] = true;
            int j = i, last = i;
            do {
                order[no++] = j;
                done[j] = true;
                last = j;
                j = next[j];
            } while (j != i);
            from_held[last] = true;
        }
    int at = 0;
    for (int root = 0; root < m; ++root) {
        if (find(root) != root) continue;
        const int first = at;
        int count = 0;
        bool cycle = false;
        for (int k = 0; k < no; ++k)
            if (find(order[k]) == root) {
                ++count;
                cycle = cycle || hold[order[k]];
            }
        cycle = cycle && count > batch;  // a batch is loaded before the first of it is stored
        const int kind = cycle ? RO_CYCLE : count == 1 ? RO_ONE : count == 2 ? RO_TWO : count <= 4 || batch == 4 ? RO_FOUR : RO_EIGHT;
        int hi = 0, lo = 0x7fffffff, all_hi = 0x7fffffff, all_lo = 0;
        for (int k = 0; k < no; ++k) {
            const int i = order[k];
            if (find(i) != root) continue;
            const int l = len[id[i]], b = p.window && l + 1 > p.window ? l + 1 - p.window : 0;
            a.move[at++] = {dst[id[i]], cycle && from_held[i] ? -1 : src[id[i]], b, l, cycle && hold[i]};
            hi = l > hi ? l : hi;
            lo = b < lo ? b : lo;
            all_hi = l < all_hi ? l : all_hi;
            all_lo = b > all_lo ? b : all_lo;
        }
        // the leading rows, which every move keeps, then the windows from the first of them
        const int lead = !p.window ? 0 : p.sinks < hi ? p.sinks : hi;
        const int from = lead > lo ? lead : lo;
        if (lead > 0) a.range[a.n_ranges++] = {first, count, 0, lead, 0, lead < all_hi ? lead : all_hi, 1, kind, {}};
        if (from < hi) a.range[a.n_ranges++] = {first, count, from, hi, all_lo, all_hi, 0, kind, {}};
    }
}

template <int CAP>
static cudaError_t launch_reorder(const ReorderPlan& p, const int32_t* dst, const int32_t* src, const int32_t* len, int n,
                                  cudaStream_t s) {
    ReorderArgs<CAP> a{};
    a.n_planes = p.n_planes;
    a.slots = p.slots;
    a.heads = p.heads;
    a.cap = p.cap;
    plan_moves(p, dst, src, len, n, 4, a);
    if (a.n_ranges == 0) return cudaSuccess;
    // Tiles of a range on a plane, and how many a block makes in a row: several once
    // the blocks fill the GPU a few times over (they share the block's set-up).
    auto tiles_of = [&](const ReorderRange& r, int row_bytes) -> long {
        const int tile = reorder_pieces(r.kind) * RO_THREADS * (row_bytes % 16 ? 8 : 16);
        return ((r.hi - r.lo) * row_bytes + tile - 1) / tile;
    };
    long total = 0, bytes = 0;
    auto add_up = [&]() {
        total = bytes = 0;
        for (int i = 0; i < p.n_planes; ++i)
            for (int c = 0; c < a.n_ranges; ++c) {
                const ReorderRange& r = a.range[c];
                total += tiles_of(r, p.plane[i].row_bytes);
                bytes += (long)(r.hi - r.lo) * p.plane[i].row_bytes * r.count;
            }
        total *= p.layers * p.heads;
        bytes *= p.layers * p.heads;
    };
    add_up();
    const bool eights = n > 4 && bytes <= RO_EIGHT_BYTES;
    if (eights) {
        a.n_ranges = 0;
        plan_moves(p, dst, src, len, n, 8, a);
        add_up();
    }
    a.run = total >= 16L * RO_FULL ? 4 : total >= 8L * RO_FULL ? 2 : 1;
    for (int i = 0; i < p.n_planes; ++i) {
        a.plane[i] = p.plane[i];
        a.plane0[i] = a.runs;
        int runs = 0;
        for (int c = 0; c < a.n_ranges; ++c) {
            a.range[c].run0[i] = runs;
            runs += (int)((tiles_of(a.range[c], p.plane[i].row_bytes) + a.run - 1) / a.run);
        }
        a.runs += runs;
    }
    cudaLaunchConfig_t cfg = {};  // may start while the kernel before it ends; waits for it first
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(a.runs, p.layers * p.heads);
    cfg.blockDim = dim3(RO_THREADS);
    cfg.stream = s;
    return eights ? cudaLaunchKernelEx(&cfg, kv_reorder_kernel<CAP, 8>, a) : cudaLaunchKernelEx(&cfg, kv_reorder_kernel<CAP, 4>, a);
}

cudaError_t launch_kv_reorder(const ReorderPlan& p, const int32_t* dst, const int32_t* src, const int32_t* len, int n,
                              cudaStream_t s) {
    return n <= 16 ? launch_reorder<16>(p, dst, src, len, n, s) : launch_reorder<KD_REORDER_MAX>(p, dst, src, len, n, s);
}

}  // namespace kd

extern "C" kd_status kd_kv_reorder(void* const* planes, const int32_t* row_bytes, int32_t n_planes, int32_t n_layers,
                                   int32_t n_slots, int32_t n_kv_heads, int32_t cap, const int32_t* dst,
                                   const int32_t* src, const int32_t* lens, int32_t n, int32_t window, int32_t sinks,
                                   kd_stream stream) {
    using namespace kd;
    if (!planes || !row_bytes || !dst || !src || !lens) return failf(KD_ERR_INVALID_ARG, "kd_kv_reorder: null argument");
    if (n < 1 || n > KD_REORDER_MAX) return failf(KD_ERR_BATCH, "kd_kv_reorder: n=%d outside [1, %d]", n, KD_REORDER_MAX);
    if (n_planes < 1 || n_planes > 4) return failf(KD_ERR_INVALID_ARG, "kd_kv_reorder: n_planes=%d", n_planes);
    if (n_layers < 1 || n_slots < 1 || n_kv_heads < 1 || cap < 1 || window < 0 || sinks < 0)
        return failf(KD_ERR_INVALID_ARG, "kd_kv_reorder: sizes must be positive, window and sinks not negative");
    if ((int64_t)n_layers * n_kv_heads > 65535 || cap > KD_REORDER_MAX_CAP)
        return failf(KD_ERR_UNSUPPORTED, "kd_kv_reorder: n_layers * n_kv_heads exceeds 65535 or cap exceeds %d",
                     KD_REORDER_MAX_CAP);
    ReorderPlan p{};
    for (int i = 0; i < n_planes; ++i) {
        if (!planes[i]) return failf(KD_ERR_INVALID_ARG, "kd_kv_reorder: null plane");
        if (row_bytes[i] < 8 || row_bytes[i] % 8 || row_bytes[i] > 1024)
            return failf(KD_ERR_UNSUPPORTED, "kd_kv_reorder: rows of %d bytes (a multiple of 8, at most 1024)", row_bytes[i]);
        if (reinterpret_cast<uintptr_t>(planes[i]) & 15)
            return failf(KD_ERR_INVALID_ARG, "kd_kv_reorder: planes must be 16-byte aligned");
        p.plane[i] = {planes[i], row_bytes[i]};
    }
    for (int i = 0; i < n; ++i) {
        if (dst[i] < 0 || dst[i] >= n_slots || src[i] < 0 || src[i] >= n_slots)
            return failf(KD_ERR_BAD_SESSION, "kd_kv_reorder: slot %d <- %d outside [0, %d)", dst[i], src[i], n_slots);
        for (int j = 0; j < i; ++j)
            if (dst[j] == dst[i]) return failf(KD_ERR_BAD_SESSION, "kd_kv_reorder: slot %d written twice", dst[i]);
        if (lens[i] < 0 || lens[i] > cap)
            return failf(KD_ERR_POSITION, "kd_kv_reorder: length %d outside [0, %d]", lens[i], cap);
    }
    p.n_planes = n_planes;
    p.layers = n_layers;
    p.slots = n_slots;
    p.heads = n_kv_heads;
    p.cap = cap;
    p.window = window;
    p.sinks = sinks;
    KD_TRY(launch_kv_reorder(p, dst, src, lens, n, (cudaStream_t)stream));
    return KD_OK;
}
