// kd_paged.h -- attention over a paged cache: the plan of a call, made on the host, and the
// launch interface (library internal).
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kd.h"

namespace kd {

// `total` pieces of work in a row for `parts` takers, each a run of them: the first `more` take
// `least` + 1.  (No division to find a taker's run; one to find a piece's taker.)
struct Shares {
    int least, more;
    Shares() = default;
    Shares(int total, int parts) : least(total / parts), more(total % parts) {}
    __host__ __device__ int begin(int i) const { return i * least + (i < more ? i : more); }
    __host__ __device__ int taker(int x) const {
        const int big = more * (least + 1);
        return x < big ? x / (least + 1) : more + (x - big) / least;
    }
};

// The keys of the sessions that each reads for itself are cut into blocks of PAGED_BLOCK.
// Blocks are numbered session by session, head by head, and every CTA takes an equal share of
// them in a row, which may end one (session, head) and begin the next.  What CTA i finds of (session, head) x is record i + x, so a
// (session, head)'s records are consecutive and no record is used twice.
constexpr int PAGED_WARPS = 4;
constexpr int PAGED_KEYS = 32;  // keys of a warp's piece
constexpr int PAGED_BLOCK = PAGED_WARPS * PAGED_KEYS;
constexpr int PAGED_MAX_CTAS = 1024, PAGED_HINTS = 64;
__host__ __device__ constexpr int PAGED_REC(int hd) { return hd + 4; }  // floats of one head's record: o, m, l

struct PagedArgs {
    const float* q;
    const void *k, *v;          // pages: fp16 rows, or quants
    const __half *ks, *vs;      // scales (Q8_0)
    const int* table;
    __half* out;
    float* part;                // records
    int* fault;                 // nullable
    int* err;
    int table_ld, n_pages, ps, B, nh, nkv, ctas;
    // Started beside the prefix kernel, which writes `call` here once all before it has ended; NULL: not, waits for the kernel before.
    const unsigned long long* started;
    unsigned long long call;
    float scale;
    Shares share;               // of all blocks, among the CTAs
    // Session b reads keys [from, to); those before lead_keys through session lead's table.  A session's
    // words lie together: each cache line of a launch's arguments that is touched first costs a
    // microsecond or so.
    struct Session {
        int first;      // first block of its first head, in blocks / nkv; session B has the end
        int from, to, lead_keys;
        short lead;
        short group;    // in SharedArgs, or SHARED_NONE
    } s[KD_PAGED_MAX_SEQS + 1];
    int empty;                  // some session has no keys
    short hint[PAGED_HINTS];    // a session at or before the first one of CTAs [i ctas / PAGED_HINTS, ..)
};
constexpr int SHARED_NONE = -1;

__host__ __device__ inline int paged_blocks(int keys) { return (keys + PAGED_BLOCK - 1) / PAGED_BLOCK; }

// Groups whose shared keys are read once for all their queries (kd_attn_shared.cu).  A pass of a
// (group, KV head) is its keys, in tiles of SHARED_TILE, for up to `side` tiles of
// shared_queries() queries, one for each of the CTAs side by side; the tiles of all passes are one
// sequence, of which every one of the `sets` of CTAs takes an equal share.
// A set's CTAs leave a record of each query that has tiles there.
constexpr int SHARED_TILE = 128, SHARED_MAX_QUERIES = 128, SHARED_MAX_SIDE = 8;
__host__ __device__ constexpr int shared_queries(bool q8) { return q8 ? 64 : SHARED_MAX_QUERIES; }
constexpr int SHARED_MAX_GROUPS = KD_PAGED_MAX_SEQS / 2;  // of two sessions at least
constexpr int SHARED_MAX_CTAS = 256;
struct SharedArgs {
    const float* q;
    const int* table;
    float* part;
    int* fault;
    const uint8_t *kq, *vq;  // Q8_0: quants and scales
    const __half *ks, *vs;
    int* status;  // [CTA]: 1 where a bounded wait ran out
    unsigned long long* started;  // as PagedArgs'; the merge clears it
    unsigned long long call;
    int table_ld, n_pages, ps, rows, box_runs, nh, nkv, gq, n_groups, side, sets;
    int tile_queries;  // shared_queries()
    int inject;        // debug fault hook (0 in normal use): 1 for K of the first CTA's first tile, 2 for V
    float scale;
    Shares share;  // of all tiles, among the sets
    struct Group {
        int first;          // first tile of its first head's first pass, in tiles / nkv; group n_groups has the end
        int keys, queries;  // shared keys (whole pages), sessions times gq
        int before;         // queries of the groups before it
        int lead;           // first session
    } g[SHARED_MAX_GROUPS + 1];
    __host__ __device__ int tiles(int i) const { return (g[i].keys + SHARED_TILE - 1) / SHARED_TILE; }
    __host__ __device__ int passes(int i) const { return (g[i].queries + tile_queries * side - 1) / (tile_queries * side); }
};
// The record of query `query` of a pass that set `set` leaves: those of different (pass, set)s do not
// overlap, as each step along the sequence moves on by a pass's queries, or by a set's most.
__host__ __device__ inline int64_t shared_row(const SharedArgs& a, int g, int h, int pass, int set, int query) {
    const int pass_queries = a.tile_queries * a.side;
    return (int64_t)a.g[g].before * a.nkv + (int64_t)h * a.g[g].queries + (int64_t)pass * pass_queries + (int64_t)set * pass_queries + query;
}
cudaError_t launch_shared(const SharedArgs& a, int hd, bool q8, const void* k, const void* v, int dev, cudaStream_t s);

// CTAs of the kernel that device dev, the current one, holds at once (0 on a CUDA error, left in *e).
int paged_slots(int hd, int group, bool q8, int dev, int num_sms, cudaError_t* e);
cudaError_t launch_paged(const PagedArgs& a, int hd, bool q8, cudaStream_t s);
cudaError_t launch_paged_merge(const PagedArgs& a, const SharedArgs& sh, int hd, cudaStream_t s);

}  // namespace kd
