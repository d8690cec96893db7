// kd_paged_api.cu -- the paged attention's entry points: checks, the plan, the launches.
// The plan travels with the launches, so a call copies nothing to the device and can be
// captured into a graph (its lengths and groups are then part of it; the table is not).
#include <atomic>
#include <cmath>

#include "kd_host.h"
#include "kd_paged.h"

namespace kd {

static std::atomic<int> paged_inject{0};  // kd_debug_attn_paged_inject_wait_timeout

static bool paged_shape(int32_t nh, int32_t nkv, int32_t hd, bool q8) {
    if (nkv < 1 || nh < 1 || nh % nkv) return false;
    const int g = nh / nkv;
    return (g == 1 || g == 2 || g == 4 || g == 8) && (hd == 128 || (hd == 64 && !q8));
}
constexpr int PAGED_MAX_KV_HEADS = 1024;
constexpr int PAGED_HEAD_BYTES = 256 + SHARED_MAX_CTAS * 4;  // the workspace's words before its records: the call's, a CTA's status
constexpr int PAGED_STARTED = 192;                          // byte of PagedArgs::started among them
static_assert((2 * KD_MAX_BATCH + 1) * 4 <= PAGED_STARTED, "behind the fault word");

// A word for PagedArgs::call that no other call has, and that memory nobody has written yet will not hold by chance.
static unsigned long long paged_call_word() {
    static std::atomic<unsigned long long> calls{0};
    unsigned long long x = (calls.fetch_add(1, std::memory_order_relaxed) + 1) * 0x9e3779b97f4a7c15ull;
    x ^= x >> 32;
    return x ? x : 1;
}
// Records of the sessions' own keys: one per CTA and (session, head) at most.
static size_t paged_records(int B, int nkv) { return (size_t)PAGED_MAX_CTAS + (size_t)B * nkv; }

// A group's shared keys go to the kernel that reads them once where that saves its other sessions enough bytes of
// reading: the kernel costs some 3 us (5 on Q8_0 caches) of its own before it gains, and a tile of it takes as long as two
// or three sessions' reading of the tile.  Each session with 128 keys of its own, 8 KV heads, caches not in L2, read once / by each (us):
//   fp16, heads of 128, 24 MB: one query a KV head, 3 sessions 13.3 / 14.7, 4 11.0 / 14.2; four, 2 15.3 / 14.0, 4 of 16 MB 11 / 9.6
//     (of 24 11.0 / 11.4), 2 of 32768 keys 36.7 / 48.0; eight, 3 of 16 MB 11.7 / 13.0;
//   heads of 64: 2 sessions lose at any length (24 MB 16.4 / 14.0, 65536 keys 47 / 42); 4 of 16 MB 10.3 / 8.2, of 24 10.5 / 11.4, of 48 14.1 / 16.0
//     (between them, where shares of the tiles end within a head, 14.8 / 12.3); 16 of 24 MB 9.6 / 9.6, of 32 10.0 / 10.9;
//   Q8_0, up to four queries a KV head: 2 and 3 sessions lose (24 MB 28.5 / 20.5 and 20.2 / 16.2; 3 gain from 128 MB on, 47.8 / 51.6);
//     4 of 16 MB 15.0 / 12.6, of 24 15.4 / 15.3, of 128 37.9 / 45.5; 8 of 48 15.5 / 19.8;
//   Q8_0, eight: 3 of 16 MB 15.7 / 19.3, 2 of 24 MB 28.7 / 27.0, of 48 40.4 / 45.8.
static bool shared_once(int rows, int keys, int nkv, int gq, int hd, bool q8) {
    if (rows < 2 || keys < 1) return false;
    const int64_t saves = (int64_t)(rows - 1) * keys * nkv * (q8 ? 272 : hd * 4) >> 20;
    if (q8) return gq == 8 ? saves >= (rows > 2 ? 16 : 40) : rows > 3 && saves >= 24;
    return saves >= 24 && (hd == 128 || rows > 2);
}

// Choose the sets of CTAs: `side` of them take a (group, head)'s tiles of queries side by side.
// The time goes as the tiles of all passes over the sets; of equal ones the widest, which read each key
// most often at the same time.
static void shared_plan(SharedArgs& t, int sms) {
    if (sms > SHARED_MAX_CTAS) sms = SHARED_MAX_CTAS;
    double best = 0;
    int most = 1;
    for (int g = 0; g < t.n_groups; ++g) {
        const int tiles = (t.g[g].queries + t.tile_queries - 1) / t.tile_queries;
        if (tiles > most) most = tiles;
    }
    for (int side = 1; side <= most && side <= SHARED_MAX_SIDE && side <= sms; ++side) {
        double work = 0;
        for (int g = 0; g < t.n_groups; ++g) {
            const int per = t.tile_queries * side;
            work += (double)t.tiles(g) * ((t.g[g].queries + per - 1) / per);
        }
        const double time = work / (sms / side);
        if (side == 1 || time <= best * 1.02) {
            best = time < best || side == 1 ? time : best;
            t.side = side;
        }
    }
    int64_t first = 0;
    int before = 0;
    for (int g = 0; g < t.n_groups; ++g) {
        t.g[g].first = (int)first;
        t.g[g].before = before;
        first += (int64_t)t.tiles(g) * t.passes(g);
        before += t.g[g].queries;
    }
    t.g[t.n_groups].first = (int)first;
    const int64_t total = first * t.nkv;
    t.sets = sms / t.side;
    // No more sets than the longest share needs: the SMs left over take the sessions' own keys meanwhile (16 beams behind 8111
    // keys, 4 tiles a CTA: 17.3 us with 128 CTAs, 19.9 with 152).
    const int64_t most_tiles = (total + t.sets - 1) / t.sets;
    t.sets = (int)((total + most_tiles - 1) / most_tiles);
    t.share = Shares((int)total, t.sets);
}

static kd_status paged_call(const char* fn, bool q8, const float* q, const void* kp, const void* vp, const uint16_t* ks,
                            const uint16_t* vs, const int32_t* table, int32_t table_ld, const int32_t* lens, int32_t B,
                            const int32_t* group_rows, const int32_t* group_prefix, int32_t n_groups, int32_t nh,
                            int32_t nkv, int32_t hd, int32_t n_pages, int32_t ps, uint16_t* out, void* ws, size_t ws_bytes,
                            int32_t* fault, kd_stream stream) {
    if (!q || !kp || !vp || (q8 && (!ks || !vs)) || !table || !lens || !out || !ws ||
        (n_groups > 0 && (!group_rows || !group_prefix)))
        return failf(KD_ERR_INVALID_ARG, "%s: null argument", fn);
    if (B < 1 || B > KD_PAGED_MAX_SEQS) return failf(KD_ERR_BATCH, "%s: B=%d outside [1, %d]", fn, B, KD_PAGED_MAX_SEQS);
    if (!paged_shape(nh, nkv, hd, q8) || nkv > PAGED_MAX_KV_HEADS)
        return failf(KD_ERR_UNSUPPORTED, "%s: head_dim %d, %d query heads, %d KV heads", fn, hd, nh, nkv);
    if (ps < 16 || ps % 16 || ps > 65536) return failf(KD_ERR_UNSUPPORTED, "%s: page_size %d", fn, ps);
    if (n_pages < 1 || table_ld < 1 || n_groups < 0)
        return failf(KD_ERR_INVALID_ARG, "%s: n_pages %d, table_ld %d, n_groups %d", fn, n_pages, table_ld, n_groups);
    if ((int64_t)n_pages * nkv > 0x7fffffff / ps) return failf(KD_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 cache rows", fn);
    if (ws_bytes < kd_attn_paged_workspace_bytes(B, nh, nkv, hd)) return failf(KD_ERR_INVALID_ARG, "%s: workspace too small", fn);
    if (((uintptr_t)q | (uintptr_t)kp | (uintptr_t)vp | (uintptr_t)ks | (uintptr_t)vs | (uintptr_t)ws) & 15)
        return failf(KD_ERR_INVALID_ARG, "%s: q, pages and workspace must be 16-byte aligned", fn);
    if ((((uintptr_t)table | (uintptr_t)fault) & 3) || ((uintptr_t)out & 1))
        return failf(KD_ERR_INVALID_ARG, "%s: table and fault must be 4-byte aligned, out 2-byte", fn);
    PagedArgs a = {};
    SharedArgs sh = {};
    int64_t total = 0, shared_tiles = 0;
    for (int b = 0; b < B; ++b) {
        if (lens[b] < 0 || lens[b] > (int64_t)table_ld * ps || lens[b] > KD_PAGED_MAX_LEN)
            return failf(KD_ERR_POSITION, "%s: length %d in tables of %d pages of %d", fn, lens[b], table_ld, ps);
        a.s[b].to = lens[b];
        a.s[b].lead = (short)b;
        a.s[b].group = SHARED_NONE;
        a.empty |= lens[b] == 0;
    }
    if (n_groups) {
        int b = 0;
        for (int g = 0; g < n_groups; ++g) {
            if (group_rows[g] < 1 || group_rows[g] > B - b)
                return failf(KD_ERR_INVALID_ARG, "%s: group %d of %d sessions", fn, g, group_rows[g]);
            const int shared = group_prefix[g] / ps * ps;  // the page that the prefix ends in is each session's own
            const bool once = shared_once(group_rows[g], shared, nkv, nh / nkv, hd, q8);
            for (int i = b; i < b + group_rows[g]; ++i) {
                if (group_prefix[g] < 0 || group_prefix[g] > lens[i])
                    return failf(KD_ERR_POSITION, "%s: prefix %d of a session of length %d", fn, group_prefix[g], lens[i]);
                a.s[i].lead = (short)b;
                a.s[i].lead_keys = shared;
                if (once) {
                    a.s[i].from = shared;
                    a.s[i].group = (short)sh.n_groups;
                }
            }
            if (once) {
                shared_tiles += (int64_t)(shared / SHARED_TILE + 1) * (group_rows[g] * (nh / nkv) / shared_queries(q8) + 1);
                if (shared_tiles > 0x7fffffff / nkv) return failf(KD_ERR_UNSUPPORTED, "%s: 2^31 or more blocks of keys", fn);
                sh.g[sh.n_groups].lead = (short)b;
                sh.g[sh.n_groups].keys = shared;
                sh.g[sh.n_groups++].queries = group_rows[g] * (nh / nkv);
            }
            b += group_rows[g];
        }
        if (b != B) return failf(KD_ERR_INVALID_ARG, "%s: groups of %d sessions in all, B=%d", fn, b, B);
    }
    for (int b = 0; b < B; ++b) {
        a.s[b].first = (int)total;
        total += paged_blocks(a.s[b].to - a.s[b].from);
        if (total > 0x7fffffff / nkv) return failf(KD_ERR_UNSUPPORTED, "%s: 2^31 or more blocks of keys", fn);
    }
    a.s[B].first = (int)total;
    int dev = 0, sms = 0;
    KD_TRY(cudaGetDevice(&dev));
    KD_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    cudaError_t e;
    const int slots = paged_slots(hd, nh / nkv, q8, dev, sms, &e);
    KD_TRY(e);
    a.q = q;
    a.k = kp;
    a.v = vp;
    a.ks = (const __half*)ks;
    a.vs = (const __half*)vs;
    a.table = table;
    a.table_ld = table_ld;
    a.out = (__half*)out;
    a.part = (float*)((char*)ws + PAGED_HEAD_BYTES);
    a.err = (int*)ws + 2 * KD_MAX_BATCH;  // where kd_attn_device_status looks
    a.fault = fault;
    a.n_pages = n_pages;
    a.ps = ps;
    a.B = B;
    a.nh = nh;
    a.nkv = nkv;
    a.scale = 1.0f / std::sqrt((float)hd);
    const int blocks = (int)(total * nkv);
    a.ctas = blocks < 1 ? 1 : blocks < slots ? blocks : slots;
    a.share = Shares(blocks, a.ctas);
    for (int i = 0, b = 0; i < PAGED_HINTS && blocks; ++i) {
        const int x = a.share.begin((int)((int64_t)i * a.ctas / PAGED_HINTS));
        while (x >= a.s[b + 1].first * nkv) ++b;
        a.hint[i] = (short)b;
    }
    bool merge = sh.n_groups > 0;
    for (int b = 0; b < B && !merge; ++b) {
        const int nb = a.s[b + 1].first - a.s[b].first;
        for (int h = 0; h < nkv && nb && !merge; ++h) {
            const int s0 = a.s[b].first * nkv + h * nb;
            merge = a.share.taker(s0) != a.share.taker(s0 + nb - 1);
        }
    }
    cudaStream_t s = (cudaStream_t)stream;
    if (sh.n_groups) {
        sh.q = q;
        sh.table = table;
        sh.part = a.part + paged_records(B, nkv) * (nh / nkv) * PAGED_REC(hd);
        sh.fault = fault;
        sh.status = (int*)ws + 64;
        sh.table_ld = table_ld;
        sh.n_pages = n_pages;
        sh.ps = ps;
        sh.rows = n_pages * nkv * ps;
        sh.box_runs = (ps & -ps) >= SHARED_TILE ? SHARED_TILE / 16 : (ps & -ps) / 16;
        sh.nh = nh;
        sh.nkv = nkv;
        sh.gq = nh / nkv;
        sh.scale = a.scale;
        sh.tile_queries = shared_queries(q8);
        shared_plan(sh, sms);
        a.started = sh.started = (unsigned long long*)((char*)ws + PAGED_STARTED);
        a.call = sh.call = paged_call_word();
        sh.kq = (const uint8_t*)kp;
        sh.vq = (const uint8_t*)vp;
        sh.ks = a.ks;
        sh.vs = a.vs;
        sh.inject = paged_inject.exchange(0, std::memory_order_relaxed);
        KD_TRY(launch_shared(sh, hd, q8, kp, vp, dev, s));
    }
    KD_TRY(launch_paged(a, hd, q8, s));
    if (merge) KD_TRY(launch_paged_merge(a, sh, hd, s));
    return KD_OK;
}

}  // namespace kd

extern "C" {

kd_status kd_debug_attn_paged_inject_wait_timeout(int32_t part) {
    if (part < 0 || part > 1) return kd::failf(KD_ERR_INVALID_ARG, "kd_debug_attn_paged_inject_wait_timeout: part %d", part);
    kd::paged_inject.store(part + 1, std::memory_order_relaxed);
    return KD_OK;
}

int32_t kd_attn_paged_reads_once(int32_t rows, int32_t prefix, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t page_size,
                                 int32_t q8) {
    using namespace kd;
    if (rows < 1 || rows > KD_PAGED_MAX_SEQS || prefix < 0 || prefix > KD_PAGED_MAX_LEN || !paged_shape(n_heads, n_kv_heads, head_dim, q8 != 0) ||
        n_kv_heads > PAGED_MAX_KV_HEADS || page_size < 16 || page_size % 16 || page_size > 65536)
        return 0;
    return shared_once(rows, prefix / page_size * page_size, n_kv_heads, n_heads / n_kv_heads, head_dim, q8 != 0);
}

size_t kd_attn_paged_workspace_bytes(int32_t B, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
    using namespace kd;
    if (B < 1 || B > KD_PAGED_MAX_SEQS || !paged_shape(n_heads, n_kv_heads, head_dim, false) || n_kv_heads > PAGED_MAX_KV_HEADS) return 0;
    // of shared keys: a record for every query, and for as many as a CTA takes per CTA
    const size_t shared = B < 2 ? 0 : (size_t)B * n_heads + (size_t)SHARED_MAX_CTAS * SHARED_MAX_QUERIES;
    return PAGED_HEAD_BYTES + (paged_records(B, n_kv_heads) * (n_heads / n_kv_heads) + shared) * PAGED_REC(head_dim) * sizeof(float);
}

kd_status kd_attn_paged_decode(const float* q, const uint16_t* k_pages, const uint16_t* v_pages, const int32_t* table,
                               int32_t table_ld, const int32_t* lens, int32_t B, const int32_t* group_rows,
                               const int32_t* group_prefix, int32_t n_groups, int32_t n_heads, int32_t n_kv_heads,
                               int32_t head_dim, int32_t n_pages, int32_t page_size, uint16_t* out, void* workspace,
                               size_t workspace_bytes, int32_t* fault, kd_stream stream) {
    return kd::paged_call("kd_attn_paged_decode", false, q, k_pages, v_pages, nullptr, nullptr, table, table_ld, lens, B,
                          group_rows, group_prefix, n_groups, n_heads, n_kv_heads, head_dim, n_pages, page_size, out,
                          workspace, workspace_bytes, fault, stream);
}

kd_status kd_attn_paged_decode_q8(const float* q, const uint8_t* k_quants, const uint16_t* k_scales,
                                  const uint8_t* v_quants, const uint16_t* v_scales, const int32_t* table,
                                  int32_t table_ld, const int32_t* lens, int32_t B, const int32_t* group_rows,
                                  const int32_t* group_prefix, int32_t n_groups, int32_t n_heads, int32_t n_kv_heads,
                                  int32_t n_pages, int32_t page_size, uint16_t* out, void* workspace,
                                  size_t workspace_bytes, int32_t* fault, kd_stream stream) {
    return kd::paged_call("kd_attn_paged_decode_q8", true, q, k_quants, v_quants, k_scales, v_scales, table, table_ld, lens,
                          B, group_rows, group_prefix, n_groups, n_heads, n_kv_heads, 128, n_pages, page_size, out,
                          workspace, workspace_bytes, fault, stream);
}

}  // extern "C"
