// kd_reorder.cu -- sessions' caches permuted, forked and joined in place.
//
// dst_i := src_i for all i at once, the same slots on both sides (what a beam
// selection asks for: beams trade places, some parents are taken several times,
// some not at all).  Row t of one slot only ever depends on row t of others, so
// a thread that owns one 16-byte piece of row t in every slot of a set of
// connected moves can make them all without a second buffer: it loads before it
// stores.  The host orders each connected set so that a slot is read before it
// is overwritten; a set has at most one cycle (every destination has one
// source), whose first overwritten piece is held in a register.
// No arithmetic: bound by HBM, one read per source row (a row taken several
// times is read once per thread) and one write per destination row.
#include <cuda_runtime.h>

#include "kd_device.cuh"
#include "kd_host.h"
#include "kd_reorder.h"

namespace kd {

constexpr int RO_THREADS = 256;
constexpr int RO_BATCH = 8;  // moves whose pieces a thread holds at once

struct ReorderMove {
    int dst, src, len;  // src -1: the piece held from the cycle's first destination
    int hold;           // hold the destination's old piece first
};
struct ReorderSet {
    int first, count;    // its moves
    int row0;            // rows of the sets before it
    int hi_a, lo_b;      // its rows: [0, hi_a), then lo_b, lo_b + 1, ...
};
struct ReorderArgs {
    ReorderPlane plane[4];
    int chunk0[4];  // first chunk (blockIdx.x) of each plane
    int n_planes, slots, heads, cap, window, sinks;
    int n_sets, rows;
    ReorderSet set[KD_REORDER_MAX];
    ReorderMove move[KD_REORDER_MAX];
};
static_assert(sizeof(ReorderArgs) <= 4096, "kernel parameters");

template <typename T>
__device__ __forceinline__ void reorder_piece(const ReorderArgs& a, char* base, int row_bytes, int chunk, int lh) {
    const int per_row = row_bytes / (int)sizeof(T);
    const int v = chunk * RO_THREADS + threadIdx.x;
    const int row = v / per_row;
    if (row >= a.rows) return;
    int c = 0;
    while (c + 1 < a.n_sets && row >= a.set[c + 1].row0) ++c;
    const ReorderSet s = a.set[c];
    const int k = row - s.row0, t = k < s.hi_a ? k : s.lo_b + (k - s.hi_a);
    const int layer = lh / a.heads, head = lh - layer * a.heads;
    // the thread's piece of row t in slot 0
    const size_t slot_bytes = (size_t)a.heads * a.cap * row_bytes;
    char* p0 = base + (size_t)layer * a.slots * slot_bytes + ((size_t)head * a.cap + t) * row_bytes +
               (size_t)(v - row * per_row) * sizeof(T);
    T held{};
    for (int m0 = 0; m0 < s.count; m0 += RO_BATCH) {
        T x[RO_BATCH];
        bool on[RO_BATCH];
#pragma unroll
        for (int u = 0; u < RO_BATCH; ++u) {
            on[u] = false;
            if (m0 + u < s.count) {
                const ReorderMove m = a.move[s.first + m0 + u];
                if (m.hold) held = *reinterpret_cast<const T*>(p0 + m.dst * slot_bytes);
                on[u] = t < m.len && (!a.window || t < a.sinks || t > m.len - a.window);
                if (on[u]) x[u] = m.src < 0 ? held : *reinterpret_cast<const T*>(p0 + m.src * slot_bytes);
            }
        }
#pragma unroll
        for (int u = 0; u < RO_BATCH; ++u)
            if (on[u]) *reinterpret_cast<T*>(p0 + a.move[s.first + m0 + u].dst * slot_bytes) = x[u];
    }
}

// Block (x, y): chunk x of the planes' row pieces, (layer, head) y.
__global__ void __launch_bounds__(RO_THREADS) kv_reorder_kernel(const __grid_constant__ ReorderArgs a) {
    int p = 0;
    while (p + 1 < a.n_planes && (int)blockIdx.x >= a.chunk0[p + 1]) ++p;
    const int chunk = (int)blockIdx.x - a.chunk0[p];
    const ReorderPlane pl = a.plane[p];
    if (pl.row_bytes % 16 == 0)
        reorder_piece<uint4>(a, (char*)pl.base, pl.row_bytes, chunk, blockIdx.y);
    else
        reorder_piece<uint2>(a, (char*)pl.base, pl.row_bytes, chunk, blockIdx.y);
}

// Order the moves into connected sets (see the file comment).
static void plan_moves(const int32_t* dst, const int32_t* src, const int32_t* len, int n, ReorderArgs& a) {
    constexpr int N = KD_REORDER_MAX;
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
    a.n_sets = 0;
    a.rows = 0;
    int at = 0;
    for (int root = 0; root < m; ++root) {
        if (find(root) != root) continue;
        ReorderSet& s = a.set[a.n_sets++];
        s.first = at;
        int hi = 0, lo = 0x7fffffff;
        for (int k = 0; k < no; ++k) {
            const int i = order[k];
            if (find(i) != root) continue;
            const int l = len[id[i]];
            a.move[at++] = {dst[id[i]], from_held[i] ? -1 : src[id[i]], l, hold[i]};
            hi = l > hi ? l : hi;
            const int b = a.window && l + 1 > a.window ? l + 1 - a.window : 0;
            lo = b < lo ? b : lo;
        }
        s.count = at - s.first;
        s.hi_a = a.sinks < lo ? a.sinks : lo;
        s.lo_b = lo;
        s.row0 = a.rows;
        a.rows += s.hi_a + hi - lo;
    }
}

cudaError_t launch_kv_reorder(const ReorderPlan& p, const int32_t* dst, const int32_t* src, const int32_t* len, int n,
                              cudaStream_t s) {
    ReorderArgs a{};
    a.n_planes = p.n_planes;
    a.slots = p.slots;
    a.heads = p.heads;
    a.cap = p.cap;
    a.window = p.window;
    a.sinks = p.sinks;
    plan_moves(dst, src, len, n, a);
    if (a.rows == 0) return cudaSuccess;
    int chunks = 0;
    for (int i = 0; i < p.n_planes; ++i) {
        a.plane[i] = p.plane[i];
        a.chunk0[i] = chunks;
        const long pieces = (long)a.rows * (p.plane[i].row_bytes / (p.plane[i].row_bytes % 16 ? 8 : 16));
        chunks += (int)((pieces + RO_THREADS - 1) / RO_THREADS);
    }
    kv_reorder_kernel<<<dim3(chunks, p.layers * p.heads), RO_THREADS, 0, s>>>(a);
    return cudaGetLastError();
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
