// kd_api.cu -- the C ABI (include/kd.h): model load and repack, the session
// slot arena, and the batched decode step's launch train.
//
// Structure of one step (memra-engine decode_batch.rs, `decode_step_batch_lean_masked`
// and `decode_batch_layers`): stage the [B] session slots, tokens and positions
// (one host-to-device copy), gather the B embedding rows, then per layer
//   RMSNorm -> QKV mmvq (+RoPE at each row's position, +KV append) ->
//   split-K flash-decode -> combine -> O mmvq (+residual) -> RMSNorm ->
//   gate|up mmvq (+SwiGLU) -> down mmvq (+residual),
// then the final RMSNorm, the lm_head mmvq and the device argmax.  The launch
// train is captured once per (B, output buffers) as a CUDA graph and replayed;
// consecutive kernels overlap through programmatic dependent launch (each
// kernel's weight prefetch runs before it waits for its predecessor).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <tuple>
#include <vector>

#include "kd.h"
#include "kd_host.h"
#include "kd_kernels.h"
#include "kd_reorder.h"
#include "kd_window.h"

using kd::PackedQ8;
static_assert(KD_TIMELINE_CTAS == kd::TL_CTAS, "timeline record layout");

namespace {

thread_local std::string g_err;

kd_status fail(kd_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return st;
}

#define KD_CK(call)                                                                               \
    do {                                                                                          \
        cudaError_t e_ = (call);                                                                  \
        if (e_ != cudaSuccess)                                                                    \
            return fail(e_ == cudaErrorMemoryAllocation ? KD_ERR_OOM : KD_ERR_CUDA, "%s: %s (%s:%d)", \
                        #call, cudaGetErrorString(e_), __FILE__, __LINE__);                      \
    } while (0)

// The kernels of the step and of the plain op-level calls; windowed attention and beam selection
// set up their own when they are first used.
cudaError_t init_device_attributes(int dev) {
    static kd::OncePerDevice once;
    return once(dev, [] {
        cudaError_t e = kd::mmvq_init_attributes();
        if (e == cudaSuccess) e = kd::attn_init_attributes();
        if (e == cudaSuccess) e = kd::attn_q8_init_attributes();
        if (e == cudaSuccess) e = kd::rowops_init_attributes();
        return e;
    });
}

constexpr int RING = 4;        // pinned staging slots for the per-step descriptor
// slot[16], token[16], pos[16], then the rows' sampling parameters (kd::SAMP_INTS words)
constexpr int DESC_INTS = 3 * KD_MAX_BATCH + kd::SAMP_INTS;

// Source-row maps of the packed tiles (see the layout note in kd_kernels.h).
std::vector<int> tiles_natural(int rows) {
    std::vector<int> t(rows / kd::TILE_ROWS);
    for (size_t i = 0; i < t.size(); ++i) t[i] = (int)i * kd::TILE_ROWS;
    return t;
}
std::vector<int> tiles_swiglu(int ffn) {  // group g = (gate tile g, up tile g)
    std::vector<int> t;
    for (int g = 0; g < ffn / kd::TILE_ROWS; ++g) {
        t.push_back(g * kd::TILE_ROWS);
        t.push_back(ffn + g * kd::TILE_ROWS);
    }
    return t;
}
std::vector<int> tiles_qkv(int heads, int hd) {  // group = (dims 16j.., dims hd/2 + 16j..) of one head
    std::vector<int> t;
    for (int h = 0; h < heads; ++h)
        for (int j = 0; j < hd / kd::GROUP_ROWS; ++j) {
            t.push_back(h * hd + j * kd::TILE_ROWS);
            t.push_back(h * hd + hd / 2 + j * kd::TILE_ROWS);
        }
    return t;
}

size_t q8_row_bytes(int K) { return (size_t)(K / 32) * 34; }

// ---- the allocation-failure switch (kd_debug_fail_alloc) ------------------------
// Every device or pinned-host allocation a model load makes goes through
// load_malloc, which counts them; an armed count fails as out of memory.
int g_fail_at = 0;          // armed for the next load: its allocation number that fails (1-based)
int g_load_fail_at = 0;     // the current load's copy
int g_load_count = -1;      // allocations counted in the current load (-1: no load running)
int g_last_load_allocs = 0; // allocations the last completed load made

cudaError_t load_malloc(void** p, size_t bytes, bool host = false) {
    if (g_load_count >= 0 && ++g_load_count == g_load_fail_at) {
        *p = nullptr;
        return cudaErrorMemoryAllocation;
    }
    return host ? cudaMallocHost(p, bytes) : cudaMalloc(p, bytes);
}

// Upload canonical Q8_0 parts (stacked by rows) through `staging`, then repack.
kd_status upload_packed(const std::vector<std::pair<const void*, int>>& parts, int K,
                        const std::vector<int>& tile_src, uint8_t* staging, int* d_tiles, int num_sms,
                        PackedQ8& out, int force_mode = -1) {
    size_t off = 0;
    int rows = 0;
    for (auto& p : parts) {
        if (!p.first) return fail(KD_ERR_INVALID_ARG, "null weight matrix");
        const size_t bytes = (size_t)p.second * q8_row_bytes(K);
        KD_CK(cudaMemcpy(staging + off, p.first, bytes, cudaMemcpyHostToDevice));
        off += bytes;
        rows += p.second;
    }
    out.K = K;
    out.rows = rows;
    out.G = (int)tile_src.size() / kd::MT;
    out.KG = K / kd::KGROUP;
    kd::plan_split(out, num_sms, force_mode);
    KD_CK(load_malloc((void**)&out.w, out.bytes()));
    KD_CK(cudaMemcpy(d_tiles, tile_src.data(), tile_src.size() * sizeof(int), cudaMemcpyHostToDevice));
    KD_CK(kd::launch_repack(staging, K, d_tiles, out.G, out.w, 0));
    KD_CK(cudaDeviceSynchronize());
    return KD_OK;
}

}  // namespace

void kd::set_last_error(const char* msg) { g_err = msg ? msg : ""; }
kd_status kd::failf(kd_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return st;
}
cudaError_t kd::ensure_device_attributes(int dev) { return init_device_attributes(dev); }

struct kd_model {
    kd_config cfg{};
    int dev = 0, num_sms = 0, attn_grid = 0;
    bool pdl = true;
    uint8_t* tok_embd = nullptr;
    std::vector<PackedQ8> qkv, wo, gu, down;
    PackedQ8 head;
    float* norms = nullptr;   // [2L+1][H]: attn_norm l, ffn_norm l, then output_norm
    float2* rope = nullptr;   // [max_ctx][hd/2]
    __half* kc = nullptr;     // [L][slots][nkv][cap][hd] (fp16 KV)
    __half* vc = nullptr;
    bool kvq8 = false;        // Q8_0 KV cache (KD_FLAG_KV_Q8_0)
    uint8_t* kq = nullptr;    // [L][slots][nkv][cap][128] quants u = q + 128
    uint8_t* vq = nullptr;
    __half* ks = nullptr;     // [L][slots][nkv][cap][4] block scales
    __half* vs = nullptr;
    float* knew = nullptr;    // [16][nkv][hd] the step's rotated k rows before quantisation
    float* vnew = nullptr;
    size_t layer_kv = 0;      // elements per layer of one arena
    kd::AttnMaps kmaps{};     // tensor maps over the K and V arenas
    CUtensorMap map_xn{}, map_attn{}, map_act{};  // activation maps the projections read through
    float* x = nullptr;       // [16][H] residual stream
    __half* xn = nullptr;     // [16][H] normed activations (written by the fused RMSNorm)
    float* ssq = nullptr;     // [H/32][16] per-group sums of squares of the residual rows
    float* q = nullptr;       // [16][nh][hd]
    __half* attn = nullptr;   // [16][nh*hd]
    __half* act = nullptr;    // [16][F]
    float* part = nullptr;    // mmvq split-K partials
    int* cnt = nullptr;       // mmvq arrival counters
    int cnt_n = 0;            // entries of cnt
    float* apart = nullptr;   // attention split partials
    int max_splits = 0;
    float* logits_ws = nullptr;
    float* yraw = nullptr;    // the unfused train's plain projection results [16][max rows]
    int yraw_ld = 0;
    int* err = nullptr;
    unsigned long long* amax_keys = nullptr;  // argmax scratch: [KD_MAX_BATCH] keys, then a counter (zero between launches)
    int* desc = nullptr;      // device [slot16 | token16 | pos16]
    int32_t* pinned = nullptr;
    cudaEvent_t ring_ev[RING] = {};
    int ring_i = 0;
    cudaEvent_t last_step = nullptr;
    cudaStream_t cap_stream = nullptr;
    std::vector<uint8_t> bound;
    std::vector<int32_t> len;
    // Rows [lo, hi) of a session's cache that were not copied when it became a
    // copy under a window (kd_session_reorder): no step may attend them.
    struct Gap { int32_t lo = 0, hi = 0; };
    std::vector<Gap> gap;
    int window = 0, sinks = 0;  // kd_model_set_window (window 0: every key)
    std::map<std::tuple<int, float*, int*, unsigned long long*, bool>, cudaGraphExec_t> graphs;
    float* hidden_dbg = nullptr;
    int inject_cls = -1;      // debug fault hook: kernel class whose next launch's bounded wait runs out
    unsigned long long* tl = nullptr;  // timeline records (kd_profile_timeline), or nullptr
    int tl_launches = 0;      // launches the timeline buffer holds
    std::vector<void*> allocs;
    // measurement: (kernel class, start, end) of every bracketed launch since the last read
    bool prof = false;
    std::vector<std::tuple<int, cudaEvent_t, cudaEvent_t>> prof_marks;
    std::vector<cudaEvent_t> ev_pool;

    template <class T>
    cudaError_t alloc(T** p, size_t bytes) {
        cudaError_t e = load_malloc((void**)p, std::max<size_t>(bytes, 16));
        if (e == cudaSuccess) allocs.push_back((void*)*p);
        return e;
    }
    void release() {
        for (auto& g : graphs) cudaGraphExecDestroy(g.second);
        graphs.clear();
        for (void* p : allocs) cudaFree(p);
        allocs.clear();
        for (auto* v : {&qkv, &wo, &gu, &down})
            for (auto& p : *v) cudaFree(p.w);
        cudaFree(head.w);
        if (pinned) cudaFreeHost(pinned);
        for (auto& e : ring_ev)
            if (e) cudaEventDestroy(e);
        for (auto& t : prof_marks) {
            cudaEventDestroy(std::get<1>(t));
            cudaEventDestroy(std::get<2>(t));
        }
        for (auto e : ev_pool) cudaEventDestroy(e);
        if (last_step) cudaEventDestroy(last_step);
        if (cap_stream) cudaStreamDestroy(cap_stream);
    }
};

static kd_status check_config(const kd_config* c) {
    if (c->n_layers < 1 || c->hidden < 128 || c->n_heads < 1 || c->n_kv_heads < 1 ||
        c->head_dim < 1 || c->ffn < 128 || c->vocab < 32 || c->max_sessions < 1 || c->max_ctx < 1)
        return fail(KD_ERR_INVALID_ARG, "kd_config: sizes must be positive (got L=%d H=%d nh=%d nkv=%d "
                    "hd=%d F=%d V=%d S=%d ctx=%d)", c->n_layers, c->hidden, c->n_heads, c->n_kv_heads,
                    c->head_dim, c->ffn, c->vocab, c->max_sessions, c->max_ctx);
    if (!(c->rms_eps >= 0.0f) || !(c->rope_theta > 0.0f))
        return fail(KD_ERR_INVALID_ARG, "kd_config: rms_eps must be >= 0 and rope_theta > 0");
    if (c->hidden % 128 || c->hidden > 131072 || c->ffn % 128 || c->vocab % 32 ||
        (c->n_heads * c->head_dim) % 128 || c->n_heads % c->n_kv_heads ||
        !kd::attn_supported(c->head_dim, c->n_heads / c->n_kv_heads))
        return fail(KD_ERR_UNSUPPORTED,
                    "kd_config: need hidden, ffn, n_heads*head_dim multiples of 128, hidden <= 131072, vocab "
                    "a multiple of 32, head_dim in {64,128}, n_heads/n_kv_heads in {1,2,4,8}");
    if ((c->flags & KD_FLAG_KV_Q8_0) && (!kd::attn_q8_supported(c->head_dim, c->n_heads / c->n_kv_heads) ||
                                         c->max_ctx % 2))
        return fail(KD_ERR_UNSUPPORTED, "kd_config: the Q8_0 KV cache needs head_dim 128 and an even max_ctx");
    return KD_OK;
}

static kd_status load_impl(kd_model* m, const kd_weights* w) {
    const kd_config& c = m->cfg;
    const int L = c.n_layers, H = c.hidden, nh = c.n_heads, nkv = c.n_kv_heads, hd = c.head_dim;
    const int F = c.ffn, V = c.vocab, S = c.max_sessions, cap = c.max_ctx;
    KD_CK(cudaGetDevice(&m->dev));
    KD_CK(cudaDeviceGetAttribute(&m->num_sms, cudaDevAttrMultiProcessorCount, m->dev));
    KD_CK(init_device_attributes(m->dev));
    m->attn_grid = kd::attn_split_grid(m->num_sms, hd, nh / nkv);
    m->pdl = true;

    // ---- weights: canonical bytes in through a staging buffer, repacked on the device
    const size_t stage_bytes = std::max({(size_t)V * q8_row_bytes(H), (size_t)2 * F * q8_row_bytes(H),
                                         (size_t)(nh + 2 * nkv) * hd * q8_row_bytes(H),
                                         (size_t)H * q8_row_bytes(F), (size_t)H * q8_row_bytes(nh * hd)});
    uint8_t* staging = nullptr;
    int* d_tiles = nullptr;
    KD_CK(load_malloc((void**)&staging, stage_bytes));
    const size_t max_tiles = std::max({(size_t)V, (size_t)2 * F, (size_t)(nh + 2 * nkv) * hd}) / kd::TILE_ROWS;
    if (load_malloc((void**)&d_tiles, max_tiles * sizeof(int)) != cudaSuccess) {
        cudaFree(staging);
        return fail(KD_ERR_OOM, "tile map allocation failed");
    }
    kd_status st = KD_OK;
    const int fm = (c.flags & KD_FLAG_SCHEDULE_STREAM) ? kd::MMVQ_STREAM
                 : (c.flags & KD_FLAG_SCHEDULE_GROUP) ? kd::MMVQ_GROUP : -1;
    m->qkv.resize(L);
    m->wo.resize(L);
    m->gu.resize(L);
    m->down.resize(L);
    for (int l = 0; l < L && st == KD_OK; ++l) {
        st = upload_packed({{w->wq[l], nh * hd}, {w->wk[l], nkv * hd}, {w->wv[l], nkv * hd}}, H,
                           tiles_qkv(nh + 2 * nkv, hd), staging, d_tiles, m->num_sms, m->qkv[l], fm);
        if (st == KD_OK)
            st = upload_packed({{w->wo[l], H}}, nh * hd, tiles_natural(H), staging, d_tiles, m->num_sms, m->wo[l], fm);
        if (st == KD_OK)
            st = upload_packed({{w->w_gate[l], F}, {w->w_up[l], F}}, H, tiles_swiglu(F), staging, d_tiles,
                               m->num_sms, m->gu[l], fm);
        if (st == KD_OK)
            st = upload_packed({{w->w_down[l], H}}, F, tiles_natural(H), staging, d_tiles, m->num_sms, m->down[l], fm);
    }
    if (st == KD_OK) st = upload_packed({{w->output, V}}, H, tiles_natural(V), staging, d_tiles, m->num_sms, m->head, fm);
    cudaFree(staging);
    cudaFree(d_tiles);
    if (st != KD_OK) return st;

    KD_CK(m->alloc(&m->tok_embd, (size_t)V * q8_row_bytes(H)));
    KD_CK(cudaMemcpy(m->tok_embd, w->tok_embd, (size_t)V * q8_row_bytes(H), cudaMemcpyHostToDevice));
    KD_CK(m->alloc(&m->norms, (size_t)(2 * L + 1) * H * sizeof(float)));
    for (int l = 0; l < L; ++l) {
        if (!w->attn_norm[l] || !w->ffn_norm[l]) return fail(KD_ERR_INVALID_ARG, "null norm weight");
        KD_CK(cudaMemcpy(m->norms + (size_t)(2 * l) * H, w->attn_norm[l], H * sizeof(float), cudaMemcpyHostToDevice));
        KD_CK(cudaMemcpy(m->norms + (size_t)(2 * l + 1) * H, w->ffn_norm[l], H * sizeof(float), cudaMemcpyHostToDevice));
    }
    KD_CK(cudaMemcpy(m->norms + (size_t)(2 * L) * H, w->output_norm, H * sizeof(float), cudaMemcpyHostToDevice));

    // ---- RoPE table in fp64 on the host, stored fp32: angle = p * theta^(-2i/hd)
    {
        const int half = hd / 2;
        std::vector<float2> tab((size_t)cap * half);
        std::vector<double> inv(half);
        for (int i = 0; i < half; ++i) inv[i] = std::pow((double)c.rope_theta, -2.0 * i / hd);
        for (int p = 0; p < cap; ++p)
            for (int i = 0; i < half; ++i) {
                const double a = (double)p * inv[i];
                tab[(size_t)p * half + i] = make_float2((float)std::cos(a), (float)std::sin(a));
            }
        KD_CK(m->alloc(&m->rope, tab.size() * sizeof(float2)));
        KD_CK(cudaMemcpy(m->rope, tab.data(), tab.size() * sizeof(float2), cudaMemcpyHostToDevice));
    }

    // ---- KV arena and workspaces
    const int MB = KD_MAX_BATCH;
    m->layer_kv = (size_t)S * nkv * cap * hd;
    if (!m->kvq8) {
        KD_CK(m->alloc(&m->kc, (size_t)L * m->layer_kv * sizeof(__half)));
        KD_CK(m->alloc(&m->vc, (size_t)L * m->layer_kv * sizeof(__half)));
        KD_CK(cudaMemset(m->kc, 0, (size_t)L * m->layer_kv * sizeof(__half)));
        KD_CK(cudaMemset(m->vc, 0, (size_t)L * m->layer_kv * sizeof(__half)));
        KD_CK(kd::make_attn_maps(m->kc, m->vc, (long)L * S * nkv * cap, hd, &m->kmaps));
    } else {
        const size_t rows = (size_t)L * S * nkv * cap;
        KD_CK(m->alloc(&m->kq, rows * 128));
        KD_CK(m->alloc(&m->vq, rows * 128));
        KD_CK(m->alloc(&m->ks, rows * 4 * sizeof(__half) + 16));  // + a 16-byte tail for rounded scale copies
        KD_CK(m->alloc(&m->vs, rows * 4 * sizeof(__half) + 16));
        for (void* p : {(void*)m->kq, (void*)m->vq}) KD_CK(cudaMemset(p, 0x80, rows * 128));  // q = 0
        for (void* p : {(void*)m->ks, (void*)m->vs}) KD_CK(cudaMemset(p, 0, rows * 4 * sizeof(__half) + 16));
        KD_CK(kd::make_attn_q8_maps(m->kq, m->vq, (long)rows, &m->kmaps));
        KD_CK(m->alloc(&m->knew, (size_t)MB * nkv * hd * sizeof(float)));
        KD_CK(m->alloc(&m->vnew, (size_t)MB * nkv * hd * sizeof(float)));
    }
    KD_CK(m->alloc(&m->x, (size_t)MB * H * sizeof(float)));
    KD_CK(m->alloc(&m->xn, (size_t)MB * H * sizeof(__half)));
    KD_CK(m->alloc(&m->ssq, (size_t)(H / kd::GROUP_ROWS) * kd::MAX_NORM_SLOTS * sizeof(float)));

    KD_CK(m->alloc(&m->q, (size_t)MB * nh * hd * sizeof(float)));
    KD_CK(m->alloc(&m->attn, (size_t)MB * nh * hd * sizeof(__half)));
    KD_CK(m->alloc(&m->act, (size_t)MB * F * sizeof(__half)));
    KD_CK(kd::make_x_map(m->xn, H, MB, &m->map_xn));
    KD_CK(kd::make_x_map(m->attn, nh * hd, MB, &m->map_attn));
    KD_CK(kd::make_x_map(m->act, F, MB, &m->map_act));
    size_t part = m->head.part_floats();
    int max_g = m->head.G;
    for (auto* v : {&m->qkv, &m->wo, &m->gu, &m->down})
        for (auto& p : *v) {
            part = std::max(part, p.part_floats());
            max_g = std::max(max_g, p.G);
        }
    KD_CK(m->alloc(&m->part, part * sizeof(float)));
    KD_CK(m->alloc(&m->cnt, (size_t)max_g * sizeof(int)));
    KD_CK(cudaMemset(m->cnt, 0, (size_t)max_g * sizeof(int)));
    m->cnt_n = max_g;
    m->max_splits = (cap + kd::ATT_CHUNK - 1) / kd::ATT_CHUNK;
    if (m->max_splits > kd::ATT_MAX_SPLITS)
        return fail(KD_ERR_UNSUPPORTED, "max_ctx %d exceeds %d positions", cap, kd::ATT_MAX_SPLITS * kd::ATT_CHUNK);
    KD_CK(m->alloc(&m->apart, (size_t)MB * nh * m->max_splits * kd::ATT_REC(hd) * sizeof(float)));
    KD_CK(m->alloc(&m->logits_ws, (size_t)MB * V * sizeof(float)));
    if (c.flags & KD_FLAG_UNFUSED) {
        m->yraw_ld = std::max({(nh + 2 * nkv) * hd, 2 * F, H});
        KD_CK(m->alloc(&m->yraw, (size_t)MB * m->yraw_ld * sizeof(float)));
    }
    KD_CK(m->alloc(&m->err, sizeof(int)));
    KD_CK(m->alloc(&m->amax_keys, (KD_MAX_BATCH + 1) * sizeof(unsigned long long)));
    KD_CK(cudaMemset(m->amax_keys, 0, (KD_MAX_BATCH + 1) * sizeof(unsigned long long)));
    KD_CK(cudaMemset(m->err, 0, sizeof(int)));
    KD_CK(m->alloc(&m->desc, DESC_INTS * sizeof(int)));
    KD_CK(cudaMemset(m->desc, 0, DESC_INTS * sizeof(int)));
    KD_CK(load_malloc((void**)&m->pinned, (size_t)RING * DESC_INTS * sizeof(int32_t), true));
    for (auto& e : m->ring_ev) KD_CK(cudaEventCreateWithFlags(&e, cudaEventDisableTiming));
    KD_CK(cudaEventCreateWithFlags(&m->last_step, cudaEventDisableTiming));
    KD_CK(cudaStreamCreateWithFlags(&m->cap_stream, cudaStreamNonBlocking));
    m->bound.assign(S, 0);
    m->len.assign(S, 0);
    m->gap.assign(S, {});
    KD_CK(cudaDeviceSynchronize());
    return KD_OK;
}

// Whether a projection fed by an RMSNorm takes the norm inside its activation
// load (group schedule, K <= 4096) rather than after a norm kernel of its own.
static bool fused_norm(const kd_model* m, const PackedQ8& p) {
    return (m->cfg.flags & KD_FLAG_FUSED_NORM) && !(m->cfg.flags & KD_FLAG_UNFUSED) && p.mode == kd::MMVQ_GROUP &&
           p.KG <= kd::MMVQ_WARPS * kd::NORM_IN_MAX_KG;
}

// The embedding kernel forms layer 0's attention-norm input itself (unless the
// unfused train runs, or q|k|v forms its normed input in its own load).
static bool embed_norm(const kd_model* m) {
    return !(m->cfg.flags & KD_FLAG_UNFUSED) && !fused_norm(m, m->qkv[0]);
}
// A windowed step's attention over fp16 rows is one launch.
static bool window_chain(const kd_model* m) { return m->window > 0 && !m->kvq8; }
// The lm_head launch makes each row's pick itself (stream schedule, fused train).
static bool head_pick(const kd_model* m) {
    return !(m->cfg.flags & KD_FLAG_UNFUSED) && m->head.mode == kd::MMVQ_STREAM;
}

// The launch train of one step; `lg` receives the logits, `am` (nullable) the argmax.
// With only_layer >= 0: that layer alone, on residual rows already in m->x and
// their per-group sums of squares in m->ssq; no embedding, no head.
// Hidden-state capture (kd_debug_capture_hidden) of a chunk of a larger step:
// its rows start at hrow0 of the step's hB rows.
// sampled: the pick applies each row's sampling parameters (staged with the descriptor).
static cudaError_t enqueue_step(kd_model* m, int B, float* lg, int* am, cudaStream_t s, int only_layer = -1,
                                int hrow0 = 0, int hB = 0, bool sampled = false) {
    if (hB == 0) hB = B;
    const kd_config& c = m->cfg;
    const int L = c.n_layers, H = c.hidden, nh = c.n_heads, nkv = c.n_kv_heads, hd = c.head_dim;
    const int F = c.ffn, V = c.vocab;
    const int* slot = m->desc;
    const int* tok = m->desc + KD_MAX_BATCH;
    const int* pos = m->desc + 2 * KD_MAX_BATCH;
    const bool pdl = m->pdl && !m->prof;
    cudaError_t e;
    // Timeline records of the step's i-th launch (kd_profile_timeline), or nullptr.
    int launch_i = 0;
    auto tl_next = [&]() -> unsigned long long* {
        const int i = launch_i++;
        return m->tl && i < m->tl_launches ? m->tl + (size_t)i * kd::TL_CTAS * kd::TL_WORDS : nullptr;
    };
    // With measurement on, every launch is bracketed by two events (no host wait).
    cudaEvent_t ev0 = nullptr;
    auto mark0 = [&]() -> cudaError_t {
        if (!m->prof) return cudaSuccess;
        if (m->ev_pool.empty()) {
            cudaEvent_t x;
            cudaError_t r = cudaEventCreate(&x);
            if (r != cudaSuccess) return r;
            m->ev_pool.push_back(x);
        }
        ev0 = m->ev_pool.back();
        m->ev_pool.pop_back();
        return cudaEventRecord(ev0, s);
    };
    auto mark1 = [&](int cls) -> cudaError_t {
        if (!m->prof) return cudaSuccess;
        cudaEvent_t x;
        if (m->ev_pool.empty()) {
            cudaError_t r = cudaEventCreate(&x);
            if (r != cudaSuccess) return r;
        } else {
            x = m->ev_pool.back();
            m->ev_pool.pop_back();
        }
        m->prof_marks.emplace_back(cls, ev0, x);
        return cudaEventRecord(x, s);
    };
#define KD_RUN(cls, launch)                                 \
    do {                                                    \
        if ((e = mark0()) != cudaSuccess) return e;         \
        if ((e = (launch)) != cudaSuccess) return e;        \
        if ((e = mark1(cls)) != cudaSuccess) return e;      \
    } while (0)

    auto mm = [&](const PackedQ8& p, const __half* x) {
        kd::MmvqArgs a{};
        a.w = p.w; a.G = p.G; a.KG = p.KG; a.W = p.W; a.maxc = p.maxc; a.K = p.K;
        a.x = x; a.B = B; a.part = m->part; a.cnt = m->cnt; a.err = m->err;
        return a;
    };
    // The debug fault hook: the first launch of the chosen class expects a few
    // bytes its copies never deliver, so one of its bounded waits runs out.
    auto inject = [&](int cls) {
        if (m->inject_cls != cls) return 0;
        m->inject_cls = -1;
        return 16;
    };
    // RMSNorm: the residual writers (embedding, o-proj, down) leave per-group sums
    // of squares; q|k|v and gate|up form their normed fp16 input from them inside
    // their activation load (fused_norm), else an elementwise kernel forms m->xn.
    auto resid = [&](kd::MmvqArgs& a) {
        a.y = m->x; a.ld = H; a.ssq_out = m->ssq;
    };
    auto norm = [&](const float* w) {
        return kd::launch_norm_from_ssq(m->x, m->ssq, B, H, w, c.rms_eps, m->xn, pdl, s, tl_next());
    };
    auto norm_in = [&](kd::MmvqArgs& a, const float* w) {
        a.nx = m->x; a.nssq = m->ssq; a.nw = w; a.neps = c.rms_eps;
    };
    // A projection with its epilogue; in the unfused train, the plain result to
    // m->yraw and the epilogue as a kernel of its own.
    const bool unfused = (c.flags & KD_FLAG_UNFUSED) != 0;
    auto proj = [&](const kd::MmvqArgs& a, const CUtensorMap& xm, int mode, int epi) -> cudaError_t {
        if (!unfused) return kd::launch_mmvq(a, xm, mode, epi, m->num_sms, pdl, s);
        kd::MmvqArgs st = a;
        st.y = m->yraw;
        st.ld = m->yraw_ld;
        cudaError_t r = kd::launch_mmvq(st, xm, mode, kd::EPI_STORE, m->num_sms, pdl, s);
        if (r != cudaSuccess) return r;
        return kd::launch_unfused_epilogue(a, m->yraw, m->yraw_ld, epi, s);
    };
    const int l0 = only_layer >= 0 ? only_layer : 0, l1 = only_layer >= 0 ? only_layer + 1 : L;
    const bool whole = only_layer < 0;
    const bool en = whole && embed_norm(m);
    if (whole)
        KD_RUN(KD_K_EMBED, kd::launch_embed(m->tok_embd, tok, B, H, m->x, m->ssq, en ? m->norms : nullptr,
                                            c.rms_eps, m->xn, pdl, s, tl_next()));
    if (whole && m->hidden_dbg &&
        (e = cudaMemcpyAsync(m->hidden_dbg + (size_t)hrow0 * H, m->x, (size_t)B * H * 4, cudaMemcpyDeviceToDevice,
                             s)) != cudaSuccess)
        return e;
    for (int l = l0; l < l1; ++l) {
        __half* kc = m->kc + (size_t)l * m->layer_kv;
        __half* vc = m->vc + (size_t)l * m->layer_kv;
        const float* attn_w = m->norms + (size_t)(2 * l) * H;
        const bool fq = fused_norm(m, m->qkv[l]);
        if (!fq && !(en && l == 0)) KD_RUN(KD_K_RMSNORM, norm(attn_w));
        kd::MmvqArgs a = mm(m->qkv[l], m->xn);
        if (fq) norm_in(a, attn_w);
        a.q_out = m->q; a.kc = kc; a.vc = vc; a.slot = slot; a.pos = pos; a.rope = m->rope;
        if (m->kvq8) { a.k_out = m->knew; a.v_out = m->vnew; }
        a.nh = nh; a.nkv = nkv; a.hd = hd; a.cap = c.max_ctx;
        a.inject_tx = inject(KD_K_QKV);
        a.tl = tl_next();
        KD_RUN(KD_K_QKV, proj(a, m->map_xn, m->qkv[l].mode, kd::EPI_QKV));
        kd::AttnArgs t{};
        t.q = m->q; t.kc = kc; t.vc = vc; t.row0 = (long)l * c.max_sessions * nkv * c.max_ctx;
        t.slot = slot; t.pos = pos; t.B = B; t.nh = nh; t.nkv = nkv;
        t.hd = hd; t.cap = c.max_ctx; t.scale = 1.0f / std::sqrt((float)hd); t.part = m->apart;
        t.max_splits = m->max_splits; t.out = m->attn; t.err = m->err;
        t.inject_tx = inject(KD_K_ATTN_SPLIT);
        t.tl = tl_next();
        if (m->kvq8) {
            t.ks = m->ks;
            t.vs = m->vs;
        }
        const bool win = m->window > 0;
        kd::AttnWinArgs tw{};  // the same for windowed rows, whose records are packed by their own item count
        if (win) {
            static_cast<kd::AttnArgs&>(tw) = t;
            tw.window = m->window;
            tw.sinks = m->sinks;
            tw.max_splits = kd::win_max_items(c.max_ctx, m->window, m->sinks);
            kd::win_fill(tw, false);
        }
        const bool chain = window_chain(m);
        if (chain) {
            KD_RUN(KD_K_ATTN_SPLIT, kd::launch_attn_chain(
                                        tw, (int)std::min<int64_t>((int64_t)m->window + m->sinks, c.max_ctx), m->dev, m->num_sms,
                                        pdl, s));
        } else if (!m->kvq8) {
            KD_RUN(KD_K_ATTN_SPLIT, kd::launch_attn_split(t, m->kmaps, m->attn_grid, pdl, s));
        } else {  // quantised append of the new rows, then the attention over the Q8_0 cache
            KD_RUN(KD_K_ATTN_SPLIT, kd::launch_kvq8_append(m->knew, m->vnew, m->kq, m->ks, m->vq, m->vs, slot, pos, B,
                                                           nkv, c.max_ctx, t.row0, pdl, s));
            KD_RUN(KD_K_ATTN_SPLIT, win ? kd::launch_attn_split_q8(tw, m->kmaps, m->num_sms, pdl, s)
                                        : kd::launch_attn_split_q8(t, m->kmaps, m->num_sms, pdl, s));
        }
        if (!chain) {
            t.tl = tw.tl = tl_next();
            KD_RUN(KD_K_ATTN_COMBINE, win ? kd::launch_attn_combine(tw, pdl, s) : kd::launch_attn_combine(t, pdl, s));
        }
        a = mm(m->wo[l], m->attn);
        resid(a);
        a.inject_tx = inject(KD_K_WO);
        a.tl = tl_next();
        KD_RUN(KD_K_WO, proj(a, m->map_attn, m->wo[l].mode, kd::EPI_RESID));
        const float* ffn_w = m->norms + (size_t)(2 * l + 1) * H;
        const bool fg = fused_norm(m, m->gu[l]);
        if (!fg) KD_RUN(KD_K_RMSNORM, norm(ffn_w));
        a = mm(m->gu[l], m->xn);
        if (fg) norm_in(a, ffn_w);
        a.act = m->act; a.ld = F;
        a.inject_tx = inject(KD_K_GATE_UP);
        a.tl = tl_next();
        KD_RUN(KD_K_GATE_UP, proj(a, m->map_xn, m->gu[l].mode, kd::EPI_SWIGLU));
        a = mm(m->down[l], m->act);
        resid(a);
        a.inject_tx = inject(KD_K_DOWN);
        a.tl = tl_next();
        KD_RUN(KD_K_DOWN, proj(a, m->map_act, m->down[l].mode, kd::EPI_RESID));
        if (whole && m->hidden_dbg &&
            (e = cudaMemcpyAsync(m->hidden_dbg + ((size_t)(l + 1) * hB + hrow0) * H, m->x, (size_t)B * H * 4,
                                 cudaMemcpyDeviceToDevice, s)) != cudaSuccess)
            return e;
    }
    if (!whole) return cudaSuccess;
    KD_RUN(KD_K_RMSNORM, norm(m->norms + (size_t)(2 * L) * H));  // the output norm
    kd::MmvqArgs a = mm(m->head, m->xn);
    a.y = lg; a.ld = V;
    a.inject_tx = inject(KD_K_LM_HEAD);
    a.tl = tl_next();
    const int* samp = sampled ? m->desc + 3 * KD_MAX_BATCH : nullptr;
    const bool pick = am && head_pick(m);
    if (pick) {
        a.pick_keys = m->amax_keys;
        a.pick_done = reinterpret_cast<unsigned*>(m->amax_keys + KD_MAX_BATCH);
        a.pick_out = am;
        a.samp = samp;
    }
    KD_RUN(KD_K_LM_HEAD, kd::launch_mmvq(a, m->map_xn, m->head.mode, pick ? kd::EPI_PICK : kd::EPI_STORE,
                                         m->num_sms, pdl, s));
    if (am && !pick)
        KD_RUN(KD_K_ARGMAX, kd::launch_argmax(lg, B, V, am, m->amax_keys,
                                              reinterpret_cast<unsigned*>(m->amax_keys + KD_MAX_BATCH), pdl, s,
                                              tl_next(), samp));
#undef KD_RUN
    return cudaSuccess;
}

static kd_status get_graph(kd_model* m, int B, float* lg, int* am, bool sampled, cudaGraphExec_t* out) {
    auto key = std::make_tuple(B, lg, am, m->tl, sampled);
    auto it = m->graphs.find(key);
    if (it != m->graphs.end()) {
        *out = it->second;
        return KD_OK;
    }
    if (m->graphs.size() >= 64) {  // bound the cache: drop everything, recapture on demand
        KD_CK(cudaStreamSynchronize(m->cap_stream));
        KD_CK(cudaEventSynchronize(m->last_step));
        for (auto& g : m->graphs) cudaGraphExecDestroy(g.second);
        m->graphs.clear();
    }
    cudaGraph_t graph = nullptr;
    KD_CK(cudaStreamBeginCapture(m->cap_stream, cudaStreamCaptureModeThreadLocal));
    cudaError_t e = enqueue_step(m, B, lg, am, m->cap_stream, -1, 0, 0, sampled);
    cudaError_t e2 = cudaStreamEndCapture(m->cap_stream, &graph);
    if (e != cudaSuccess || e2 != cudaSuccess) {
        if (graph) cudaGraphDestroy(graph);
        return fail(KD_ERR_CUDA, "capturing the step graph failed: %s",
                    cudaGetErrorString(e != cudaSuccess ? e : e2));
    }
    cudaGraphExec_t exec = nullptr;
    e = cudaGraphInstantiate(&exec, graph, 0);
    cudaGraphDestroy(graph);
    KD_CK(e);
    m->graphs[key] = exec;
    *out = exec;
    return KD_OK;
}

extern "C" {

const char* kd_last_error(void) { return g_err.c_str(); }

kd_status kd_model_load(const kd_config* cfg, const kd_weights* w, kd_model** out) {
    if (!cfg || !w || !out) return fail(KD_ERR_INVALID_ARG, "kd_model_load: null argument");
    *out = nullptr;
    kd_status st = check_config(cfg);
    if (st != KD_OK) return st;
    if (!w->tok_embd || !w->output || !w->output_norm || !w->wq || !w->wk || !w->wv || !w->wo ||
        !w->w_gate || !w->w_up || !w->w_down || !w->attn_norm || !w->ffn_norm)
        return fail(KD_ERR_INVALID_ARG, "kd_model_load: null weight pointer");
    kd_model* m = new (std::nothrow) kd_model();
    if (!m) return fail(KD_ERR_OOM, "kd_model_load: host allocation failed");
    m->cfg = *cfg;
    m->kvq8 = (cfg->flags & KD_FLAG_KV_Q8_0) != 0;
    g_load_fail_at = g_fail_at;  // an armed failure applies to this load only
    g_fail_at = 0;
    g_load_count = 0;
    st = load_impl(m, w);
    g_last_load_allocs = g_load_count;
    g_load_count = -1;
    if (st != KD_OK) {
        m->release();
        delete m;
        return st;
    }
    g_err.clear();
    *out = m;
    return KD_OK;
}

kd_status kd_model_free(kd_model* m) {
    if (!m) return fail(KD_ERR_INVALID_ARG, "kd_model_free: null model");
    cudaSetDevice(m->dev);
    cudaEventSynchronize(m->last_step);
    cudaStreamSynchronize(m->cap_stream);
    m->release();
    delete m;
    return KD_OK;
}

kd_status kd_session_bind(kd_model* m, int32_t* id_out) {
    if (!m || !id_out) return fail(KD_ERR_INVALID_ARG, "kd_session_bind: null argument");
    for (size_t i = 0; i < m->bound.size(); ++i)
        if (!m->bound[i]) {
            m->bound[i] = 1;
            m->len[i] = 0;
            m->gap[i] = {};
            *id_out = (int32_t)i;
            return KD_OK;
        }
    return fail(KD_ERR_NO_FREE_SLOT, "kd_session_bind: all %zu slots are bound", m->bound.size());
}

static kd_status check_session(const kd_model* m, int32_t id) {
    if (id < 0 || id >= (int32_t)m->bound.size() || !m->bound[id])
        return fail(KD_ERR_BAD_SESSION, "session %d is not bound", id);
    return KD_OK;
}

kd_status kd_session_free(kd_model* m, int32_t id) {
    if (!m) return fail(KD_ERR_INVALID_ARG, "kd_session_free: null model");
    kd_status st = check_session(m, id);
    if (st != KD_OK) return st;
    KD_CK(cudaSetDevice(m->dev));
    KD_CK(cudaEventSynchronize(m->last_step));
    m->bound[id] = 0;
    m->len[id] = 0;
    return KD_OK;
}

kd_status kd_session_length(const kd_model* m, int32_t id, int32_t* len_out) {
    if (!m || !len_out) return fail(KD_ERR_INVALID_ARG, "kd_session_length: null argument");
    kd_status st = check_session(m, id);
    if (st != KD_OK) return st;
    *len_out = m->len[id];
    return KD_OK;
}

kd_status kd_session_load_kv(kd_model* m, int32_t id, const void* k, const void* v, int32_t len,
                             kd_stream stream) {
    if (!m) return fail(KD_ERR_INVALID_ARG, "kd_session_load_kv: null model");
    kd_status st = check_session(m, id);
    if (st != KD_OK) return st;
    if (len < 0 || len > m->cfg.max_ctx)
        return fail(KD_ERR_POSITION, "kd_session_load_kv: len %d outside [0, %d]", len, m->cfg.max_ctx);
    if (len > 0 && (!k || !v)) return fail(KD_ERR_INVALID_ARG, "kd_session_load_kv: null cache");
    KD_CK(cudaSetDevice(m->dev));
    cudaStream_t s = (cudaStream_t)stream;
    KD_CK(cudaStreamWaitEvent(s, m->last_step, 0));
    const kd_config& c = m->cfg;
    if (m->kvq8 && len > 0) {
        // Q8_0 cache: the fp16 rows to a stream-ordered temporary, quantised into the slot's rows.
        const size_t n_rows = (size_t)c.n_layers * c.n_kv_heads * len, bytes = n_rows * c.head_dim * sizeof(__half);
        void* tmp = nullptr;
        KD_CK(cudaMallocAsync(&tmp, bytes, s));
        const long layer_rows = (long)c.max_sessions * c.n_kv_heads * c.max_ctx, base = (long)id * c.n_kv_heads * c.max_ctx;
        cudaError_t e = cudaSuccess;
        for (int part = 0; part < 2 && e == cudaSuccess; ++part) {
            e = cudaMemcpyAsync(tmp, part ? v : k, bytes, cudaMemcpyDefault, s);
            if (e == cudaSuccess)
                e = kd::launch_kvq8_rows(tmp, true, (long)n_rows, c.n_kv_heads, len, c.max_ctx, layer_rows, base,
                                         part ? m->vq : m->kq, part ? m->vs : m->ks, s);
        }
        const cudaError_t e2 = cudaFreeAsync(tmp, s);
        KD_CK(e);
        KD_CK(e2);
        KD_CK(cudaEventRecord(m->last_step, s));
        m->len[id] = len;
        m->gap[id] = {};
        return KD_OK;
    }
    const size_t row = (size_t)c.head_dim * sizeof(__half);
    for (int l = 0; l < c.n_layers && len > 0; ++l) {
        const size_t dst = (size_t)l * m->layer_kv + (size_t)id * c.n_kv_heads * c.max_ctx * c.head_dim;
        const size_t src = (size_t)l * c.n_kv_heads * len * c.head_dim;
        KD_CK(cudaMemcpy2DAsync(m->kc + dst, c.max_ctx * row, (const __half*)k + src, len * row, len * row,
                                c.n_kv_heads, cudaMemcpyDefault, s));
        KD_CK(cudaMemcpy2DAsync(m->vc + dst, c.max_ctx * row, (const __half*)v + src, len * row, len * row,
                                c.n_kv_heads, cudaMemcpyDefault, s));
    }
    KD_CK(cudaEventRecord(m->last_step, s));
    m->len[id] = len;
    m->gap[id] = {};
    return KD_OK;
}

static kd_status check_rows(kd_model* m, const char* fn, const int32_t* ids, const int32_t* tokens,
                            const int32_t* positions, int32_t B, int32_t max_b) {
    if (B < 1 || B > max_b) return fail(KD_ERR_BATCH, "%s: B=%d outside [1, %d]", fn, B, max_b);
    if (!ids || !positions) return fail(KD_ERR_INVALID_ARG, "%s: null host array", fn);
    const kd_config& c = m->cfg;
    for (int b = 0; b < B; ++b) {
        kd_status st = check_session(m, ids[b]);
        if (st != KD_OK) return st;
        for (int j = 0; j < b; ++j)
            if (ids[j] == ids[b]) return fail(KD_ERR_BAD_SESSION, "session %d appears twice in one step", ids[b]);
        if (tokens && (tokens[b] < 0 || tokens[b] >= c.vocab))
            return fail(KD_ERR_INVALID_ARG, "token %d of row %d outside [0, %d)", tokens[b], b, c.vocab);
        if (positions[b] < 0 || positions[b] > m->len[ids[b]] || positions[b] >= c.max_ctx)
            return fail(KD_ERR_POSITION, "position %d of session %d: length is %d, capacity %d", positions[b],
                        ids[b], m->len[ids[b]], c.max_ctx);
        const kd_model::Gap g = m->gap[ids[b]];
        if (g.lo < g.hi) {  // the rows before p that a step at p attends: [0, a) and [w, p)
            const int32_t p = positions[b], w = m->window > 0 ? std::max(0, p + 1 - m->window) : 0;
            const int32_t a = std::min(m->window > 0 ? m->sinks : 0, w);
            if (g.lo < a || std::max(g.lo, w) < std::min(g.hi, p))
                return fail(KD_ERR_POSITION, "position %d of session %d attends rows [%d, %d), which its copy left out",
                            p, ids[b], g.lo, g.hi);
        }
    }
    return KD_OK;
}

// Stage the [slot | token | pos] descriptor through a pinned ring slot no earlier
// copy still reads, ordered after the model's previous step.
static kd_status stage_descriptor(kd_model* m, const int32_t* ids, const int32_t* tokens, const int32_t* positions,
                                  int32_t B, cudaStream_t s, const kd_sample_params* sp = nullptr) {
    const int ri = m->ring_i;
    KD_CK(cudaEventSynchronize(m->ring_ev[ri]));
    int32_t* d = m->pinned + (size_t)ri * DESC_INTS;
    std::memset(d, 0, DESC_INTS * sizeof(int32_t));
    for (int b = 0; b < B; ++b) {
        d[b] = ids[b];
        d[KD_MAX_BATCH + b] = tokens ? tokens[b] : 0;
        d[2 * KD_MAX_BATCH + b] = positions[b];
        if (sp) {  // the layout launch_argmax documents
            int32_t* q = d + 3 * KD_MAX_BATCH;
            std::memcpy(&q[b], &sp[b].temperature, sizeof(float));
            q[16 + 2 * b] = (int32_t)(uint32_t)sp[b].seed;
            q[17 + 2 * b] = (int32_t)(uint32_t)(sp[b].seed >> 32);
            q[48 + 2 * b] = (int32_t)(uint32_t)sp[b].counter;
            q[49 + 2 * b] = (int32_t)(uint32_t)(sp[b].counter >> 32);
        }
    }
    KD_CK(cudaStreamWaitEvent(s, m->last_step, 0));
    KD_CK(cudaMemcpyAsync(m->desc, d, DESC_INTS * sizeof(int32_t), cudaMemcpyHostToDevice, s));
    KD_CK(cudaEventRecord(m->ring_ev[ri], s));
    m->ring_i = (ri + 1) % RING;
    return KD_OK;
}

// One step, greedy (sp == nullptr) or with each row's sampling parameters.
static kd_status decode_impl(kd_model* m, const char* fn, const int32_t* ids, const int32_t* tokens,
                             const int32_t* positions, int32_t B, const kd_sample_params* sp, float* logits_out,
                             int32_t* argmax_out, kd_stream stream) {
    if (!m) return fail(KD_ERR_INVALID_ARG, "%s: null model", fn);
    if (!tokens && B >= 1) return fail(KD_ERR_INVALID_ARG, "%s: null host array", fn);
    // Any number of distinct bound sessions; above KD_MAX_BATCH the step runs as
    // consecutive groups of at most KD_MAX_BATCH rows on the same kernels.
    kd_status st0 = check_rows(m, fn, ids, tokens, positions, B, (int32_t)m->bound.size());
    if (st0 != KD_OK) return st0;
    if (reinterpret_cast<uintptr_t>(logits_out) & 15)
        return fail(KD_ERR_INVALID_ARG, "%s: logits_out must be 16-byte aligned", fn);
    const kd_config& c = m->cfg;
    KD_CK(cudaSetDevice(m->dev));
    cudaStream_t s = (cudaStream_t)stream;
    const bool direct = m->hidden_dbg || m->prof || (c.flags & KD_FLAG_NO_GRAPH) || m->inject_cls >= 0;
    for (int r0 = 0; r0 < B; r0 += KD_MAX_BATCH) {
        const int n = std::min(B - r0, KD_MAX_BATCH);
        st0 = stage_descriptor(m, ids + r0, tokens + r0, positions + r0, n, s, sp ? sp + r0 : nullptr);
        if (st0 != KD_OK) return st0;
        float* lg = logits_out ? logits_out + (size_t)r0 * c.vocab : m->logits_ws;
        int* am = argmax_out ? argmax_out + r0 : nullptr;
        if (direct) {
            KD_CK(enqueue_step(m, n, lg, am, s, -1, r0, B, sp != nullptr));
        } else {
            cudaGraphExec_t g = nullptr;
            kd_status st = get_graph(m, n, lg, am, sp != nullptr, &g);
            if (st != KD_OK) return st;
            KD_CK(cudaGraphLaunch(g, s));
        }
        KD_CK(cudaEventRecord(m->last_step, s));
    }
    for (int b = 0; b < B; ++b) {
        m->len[ids[b]] = positions[b] + 1;
        m->gap[ids[b]].hi = std::min(m->gap[ids[b]].hi, positions[b]);  // a rewind forgets rows, gap and all
    }
    return KD_OK;
}

kd_status kd_model_set_window(kd_model* m, int32_t window, int32_t sinks) {
    if (!m || window < 0 || sinks < 0)
        return fail(KD_ERR_INVALID_ARG, "kd_model_set_window: null model, or window %d, sinks %d", window, sinks);
    if (window > 0 && m->cfg.n_kv_heads > kd::WIN_MAX_KV_HEADS)
        return fail(KD_ERR_UNSUPPORTED, "kd_model_set_window: more than %d KV heads", kd::WIN_MAX_KV_HEADS);
    KD_CK(cudaSetDevice(m->dev));
    KD_CK(cudaStreamSynchronize(m->cap_stream));
    KD_CK(cudaEventSynchronize(m->last_step));
    if (window > 0) {  // the kernels' set-up, before steps are captured
        const kd_config& c = m->cfg;
        KD_CK(m->kvq8 ? kd::attn_q8_win_prepare(m->dev) : kd::attn_chain_prepare(c.head_dim, c.n_heads / c.n_kv_heads, kd::win_max_items(c.max_ctx, window, sinks), m->dev));
    }
    for (auto& g : m->graphs) cudaGraphExecDestroy(g.second);
    m->graphs.clear();
    m->window = window;
    m->sinks = window > 0 ? sinks : 0;
    return KD_OK;
}

kd_status kd_session_reorder(kd_model* m, const int32_t* ids, const int32_t* parents, int32_t n, kd_stream stream) {
    if (!m || !ids || !parents) return fail(KD_ERR_INVALID_ARG, "kd_session_reorder: null argument");
    if (n < 1 || n > KD_REORDER_MAX) return fail(KD_ERR_BATCH, "kd_session_reorder: n=%d outside [1, %d]", n, KD_REORDER_MAX);
    int32_t src[KD_REORDER_MAX], len[KD_REORDER_MAX];
    kd_model::Gap gap[KD_REORDER_MAX];
    for (int i = 0; i < n; ++i) {
        kd_status st = check_session(m, ids[i]);
        if (st != KD_OK) return st;
        src[i] = parents[i] == -1 ? ids[i] : parents[i];
        if ((st = check_session(m, src[i])) != KD_OK) return st;
        for (int j = 0; j < i; ++j)
            if (ids[j] == ids[i]) return fail(KD_ERR_BAD_SESSION, "session %d appears twice in one reorder", ids[i]);
        len[i] = m->len[src[i]];
        gap[i] = m->gap[src[i]];
        if (m->window > 0 && src[i] != ids[i]) {  // the rows no later step attends stay behind
            const int32_t hi = std::max(0, len[i] + 1 - m->window), lo = std::min(m->sinks, hi);
            if (lo < hi) gap[i] = gap[i].lo < gap[i].hi ? kd_model::Gap{std::min(lo, gap[i].lo), std::max(hi, gap[i].hi)}
                                                       : kd_model::Gap{lo, hi};
        }
    }
    const kd_config& c = m->cfg;
    if ((int64_t)c.n_layers * c.n_kv_heads > 65535)
        return fail(KD_ERR_UNSUPPORTED, "kd_session_reorder: n_layers * n_kv_heads exceeds 65535");
    kd::ReorderPlan p{};
    if (!m->kvq8) {
        p.n_planes = 2;
        p.plane[0] = {m->kc, c.head_dim * (int)sizeof(__half)};
        p.plane[1] = {m->vc, c.head_dim * (int)sizeof(__half)};
    } else {
        p.n_planes = 4;
        p.plane[0] = {m->kq, 128};
        p.plane[1] = {m->ks, 8};
        p.plane[2] = {m->vq, 128};
        p.plane[3] = {m->vs, 8};
    }
    p.layers = c.n_layers;
    p.slots = c.max_sessions;
    p.heads = c.n_kv_heads;
    p.cap = c.max_ctx;
    p.window = m->window;
    p.sinks = m->sinks;
    KD_CK(cudaSetDevice(m->dev));
    cudaStream_t s = (cudaStream_t)stream;
    KD_CK(cudaStreamWaitEvent(s, m->last_step, 0));
    KD_CK(kd::launch_kv_reorder(p, ids, src, len, n, s));
    KD_CK(cudaEventRecord(m->last_step, s));
    for (int i = 0; i < n; ++i) {
        m->len[ids[i]] = len[i];
        m->gap[ids[i]] = gap[i];
    }
    return KD_OK;
}

kd_status kd_session_fork(kd_model* m, int32_t id, int32_t* new_id_out, kd_stream stream) {
    if (!m || !new_id_out) return fail(KD_ERR_INVALID_ARG, "kd_session_fork: null argument");
    kd_status st = check_session(m, id);
    if (st != KD_OK) return st;
    int32_t to = -1;
    if ((st = kd_session_bind(m, &to)) != KD_OK) return st;
    if ((st = kd_session_reorder(m, &to, &id, 1, stream)) != KD_OK) {
        m->bound[to] = 0;
        return st;
    }
    *new_id_out = to;
    return KD_OK;
}

kd_status kd_decode_step(kd_model* m, const int32_t* ids, const int32_t* tokens, const int32_t* positions,
                         int32_t B, float* logits_out, int32_t* argmax_out, kd_stream stream) {
    return decode_impl(m, "kd_decode_step", ids, tokens, positions, B, nullptr, logits_out, argmax_out, stream);
}

kd_status kd_decode_step_sampled(kd_model* m, const int32_t* ids, const int32_t* tokens, const int32_t* positions,
                                 int32_t B, const kd_sample_params* params, float* logits_out, int32_t* token_out,
                                 kd_stream stream) {
    if (!params || !token_out) return fail(KD_ERR_INVALID_ARG, "kd_decode_step_sampled: null params or token_out");
    return decode_impl(m, "kd_decode_step_sampled", ids, tokens, positions, B, params, logits_out, token_out, stream);
}

kd_status kd_debug_layer(kd_model* m, int32_t layer, const int32_t* ids, const int32_t* positions, int32_t B,
                         const float* x_in, float* x_out, kd_stream stream) {
    if (!m || !x_in || !x_out) return fail(KD_ERR_INVALID_ARG, "kd_debug_layer: null argument");
    if (layer < 0 || layer >= m->cfg.n_layers)
        return fail(KD_ERR_INVALID_ARG, "kd_debug_layer: layer %d outside [0, %d)", layer, m->cfg.n_layers);
    kd_status st = check_rows(m, "kd_debug_layer", ids, nullptr, positions, B, KD_MAX_BATCH);
    if (st != KD_OK) return st;
    KD_CK(cudaSetDevice(m->dev));
    cudaStream_t s = (cudaStream_t)stream;
    st = stage_descriptor(m, ids, nullptr, positions, B, s);
    if (st != KD_OK) return st;
    const size_t bytes = (size_t)B * m->cfg.hidden * sizeof(float);
    KD_CK(cudaMemcpyAsync(m->x, x_in, bytes, cudaMemcpyDefault, s));
    // The per-group sums of squares of the rows (as a residual writer leaves them);
    // the layer then forms its attention norm from them as in a step.
    KD_CK(kd::launch_ssq_rows(m->x, B, m->cfg.hidden, m->ssq, s));
    const bool prof = m->prof;
    m->prof = false;
    cudaError_t e = enqueue_step(m, B, nullptr, nullptr, s, layer);
    m->prof = prof;
    KD_CK(e);
    KD_CK(cudaMemcpyAsync(x_out, m->x, bytes, cudaMemcpyDefault, s));
    KD_CK(cudaEventRecord(m->last_step, s));
    return KD_OK;
}

kd_status kd_debug_fail_alloc(int32_t nth, int32_t* allocs_out) {
    if (nth < 0) return fail(KD_ERR_INVALID_ARG, "kd_debug_fail_alloc: nth=%d", nth);
    g_fail_at = nth;
    if (allocs_out) *allocs_out = g_last_load_allocs;
    return KD_OK;
}

kd_status kd_debug_capture_hidden(kd_model* m, float* dev_buf) {
    if (!m) return fail(KD_ERR_INVALID_ARG, "kd_debug_capture_hidden: null model");
    m->hidden_dbg = dev_buf;
    return KD_OK;
}

kd_status kd_profile_enable(kd_model* m, int32_t on) {
    if (!m) return fail(KD_ERR_INVALID_ARG, "kd_profile_enable: null model");
    m->prof = on != 0;
    return KD_OK;
}

kd_status kd_profile_timeline(kd_model* m, uint64_t* dev_buf, int32_t max_launches, int32_t* classes_out) {
    if (!m) return fail(KD_ERR_INVALID_ARG, "kd_profile_timeline: null model");
    if (dev_buf && max_launches < 1) return fail(KD_ERR_INVALID_ARG, "kd_profile_timeline: max_launches < 1");
    m->tl = reinterpret_cast<unsigned long long*>(dev_buf);
    m->tl_launches = dev_buf ? max_launches : 0;
    if (classes_out) {  // the launch train of a whole step, in order
        const int L = m->cfg.n_layers;
        std::vector<int32_t> cls;
        cls.push_back(KD_K_EMBED);
        for (int l = 0; l < L; ++l) {
            if (!fused_norm(m, m->qkv[l]) && !(l == 0 && embed_norm(m))) cls.push_back(KD_K_RMSNORM);
            for (int k : {KD_K_QKV, KD_K_ATTN_SPLIT, KD_K_ATTN_COMBINE, KD_K_WO})
                if (k != KD_K_ATTN_COMBINE || !window_chain(m)) cls.push_back(k);
            if (!fused_norm(m, m->gu[l])) cls.push_back(KD_K_RMSNORM);
            for (int k : {KD_K_GATE_UP, KD_K_DOWN}) cls.push_back(k);
        }
        cls.push_back(KD_K_RMSNORM);
        cls.push_back(KD_K_LM_HEAD);
        if (!head_pick(m)) cls.push_back(KD_K_ARGMAX);
        for (int i = 0; i < max_launches; ++i) classes_out[i] = i < (int)cls.size() ? cls[i] : -1;
    }
    return KD_OK;
}

kd_status kd_profile_read(kd_model* m, int32_t* launches, double* ms) {
    if (!m || !launches || !ms) return fail(KD_ERR_INVALID_ARG, "kd_profile_read: null argument");
    KD_CK(cudaSetDevice(m->dev));
    KD_CK(cudaEventSynchronize(m->last_step));
    for (int i = 0; i < KD_K_COUNT; ++i) {
        launches[i] = 0;
        ms[i] = 0.0;
    }
    cudaError_t first = cudaSuccess;
    for (auto& t : m->prof_marks) {
        float x = 0.0f;
        cudaError_t e = cudaEventElapsedTime(&x, std::get<1>(t), std::get<2>(t));
        if (e != cudaSuccess && first == cudaSuccess) first = e;
        launches[std::get<0>(t)] += 1;
        ms[std::get<0>(t)] += x;
        m->ev_pool.push_back(std::get<1>(t));
        m->ev_pool.push_back(std::get<2>(t));
    }
    m->prof_marks.clear();
    KD_CK(first);
    return KD_OK;
}

kd_status kd_device_status(kd_model* m, int32_t* flags_out) {
    if (!m || !flags_out) return fail(KD_ERR_INVALID_ARG, "kd_device_status: null argument");
    KD_CK(cudaSetDevice(m->dev));
    KD_CK(cudaEventSynchronize(m->last_step));
    int v = 0;
    KD_CK(cudaMemcpy(&v, m->err, sizeof(int), cudaMemcpyDeviceToHost));
    KD_CK(cudaMemset(m->err, 0, sizeof(int)));
    *flags_out = v;
    if (v) {
        // The kernels keep their arrival counters consistent when they give up;
        // clear them anyway, so nothing a faulted step left can reach the next one.
        KD_CK(cudaMemset(m->cnt, 0, (size_t)m->cnt_n * sizeof(int)));
        KD_CK(cudaDeviceSynchronize());
        return fail(KD_ERR_DEVICE, "a kernel gave up a bounded wait (flags 0x%x)", v);
    }
    return KD_OK;
}

kd_status kd_debug_inject_wait_timeout(kd_model* m, int32_t kernel_class) {
    if (!m) return fail(KD_ERR_INVALID_ARG, "kd_debug_inject_wait_timeout: null model");
    if (kernel_class == KD_K_ATTN_SPLIT && window_chain(m))
        return fail(KD_ERR_INVALID_ARG, "kd_debug_inject_wait_timeout: windowed attention over fp16 rows has no bounded wait");
    switch (kernel_class) {
        case KD_K_QKV: case KD_K_ATTN_SPLIT: case KD_K_WO: case KD_K_GATE_UP: case KD_K_DOWN: case KD_K_LM_HEAD:
            m->inject_cls = kernel_class;
            return KD_OK;
        default:
            return fail(KD_ERR_INVALID_ARG, "kd_debug_inject_wait_timeout: kernel class %d has no bounded wait",
                        kernel_class);
    }
}

// ------------------------------------------------------------- op level ----
struct kd_q8_matrix {
    PackedQ8 p;
    float* part = nullptr;
    int* cnt = nullptr;
    int* err = nullptr;
    int dev = 0, num_sms = 0;
};

kd_status kd_q8_matrix_create(const void* host, int32_t rows, int32_t cols, kd_q8_matrix** out) {
    if (!host || !out) return fail(KD_ERR_INVALID_ARG, "kd_q8_matrix_create: null argument");
    *out = nullptr;
    if (rows < kd::GROUP_ROWS || rows % kd::GROUP_ROWS || cols < kd::KGROUP || cols % kd::KGROUP)
        return fail(KD_ERR_UNSUPPORTED, "kd_q8_matrix_create: need rows %% 32 == 0 and cols %% 128 == 0 (got %d x %d)",
                    rows, cols);
    kd_q8_matrix* w = new (std::nothrow) kd_q8_matrix();
    if (!w) return fail(KD_ERR_OOM, "host allocation failed");
    auto cleanup = [&](kd_status st) {
        cudaFree(w->p.w);
        cudaFree(w->part);
        cudaFree(w->cnt);
        cudaFree(w->err);
        delete w;
        return st;
    };
    uint8_t* staging = nullptr;
    int* d_tiles = nullptr;
    if (cudaGetDevice(&w->dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&w->num_sms, cudaDevAttrMultiProcessorCount, w->dev) != cudaSuccess ||
        init_device_attributes(w->dev) != cudaSuccess)
        return cleanup(fail(KD_ERR_CUDA, "kd_q8_matrix_create: no usable CUDA device"));
    if (cudaMalloc(&staging, (size_t)rows * q8_row_bytes(cols)) != cudaSuccess ||
        cudaMalloc(&d_tiles, (size_t)rows / kd::TILE_ROWS * sizeof(int)) != cudaSuccess) {
        cudaFree(staging);
        return cleanup(fail(KD_ERR_OOM, "kd_q8_matrix_create: device allocation failed"));
    }
    kd_status st = upload_packed({{host, rows}}, cols, tiles_natural(rows), staging, d_tiles, w->num_sms, w->p);
    cudaFree(staging);
    cudaFree(d_tiles);
    if (st != KD_OK) return cleanup(st);
    if (cudaMalloc(&w->part, std::max<size_t>(w->p.part_floats(), 4) * sizeof(float)) != cudaSuccess ||
        cudaMalloc(&w->cnt, (size_t)w->p.G * sizeof(int)) != cudaSuccess ||
        cudaMalloc(&w->err, sizeof(int)) != cudaSuccess)
        return cleanup(fail(KD_ERR_OOM, "kd_q8_matrix_create: workspace allocation failed"));
    if (cudaMemset(w->cnt, 0, (size_t)w->p.G * sizeof(int)) != cudaSuccess ||
        cudaMemset(w->err, 0, sizeof(int)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)
        return cleanup(fail(KD_ERR_CUDA, "kd_q8_matrix_create: workspace init failed"));
    *out = w;
    return KD_OK;
}

kd_status kd_q8_matrix_free(kd_q8_matrix* w) {
    if (!w) return fail(KD_ERR_INVALID_ARG, "kd_q8_matrix_free: null matrix");
    cudaDeviceSynchronize();
    cudaFree(w->p.w);
    cudaFree(w->part);
    cudaFree(w->cnt);
    cudaFree(w->err);
    delete w;
    return KD_OK;
}

kd_status kd_mmvq(const kd_q8_matrix* w, const uint16_t* x, int32_t m, float* y, kd_stream stream) {
    if (!w || !x || !y) return fail(KD_ERR_INVALID_ARG, "kd_mmvq: null argument");
    if (m < 1 || m > KD_MAX_BATCH) return fail(KD_ERR_BATCH, "kd_mmvq: m=%d outside [1, %d]", m, KD_MAX_BATCH);
    if (reinterpret_cast<uintptr_t>(x) & 15) return fail(KD_ERR_INVALID_ARG, "kd_mmvq: x must be 16-byte aligned");
    kd::MmvqArgs a{};
    a.w = w->p.w; a.G = w->p.G; a.KG = w->p.KG; a.W = w->p.W; a.maxc = w->p.maxc; a.K = w->p.K;
    a.x = reinterpret_cast<const __half*>(x); a.B = m; a.part = w->part; a.cnt = w->cnt; a.err = w->err;
    a.y = y; a.ld = w->p.rows;
    CUtensorMap xmap;
    KD_CK(kd::make_x_map(a.x, a.K, m, &xmap));
    KD_CK(kd::launch_mmvq(a, xmap, w->p.mode, kd::EPI_STORE, w->num_sms, false, (cudaStream_t)stream));
    return KD_OK;
}

kd_status kd_q8_matrix_status(kd_q8_matrix* w, int32_t* flags_out) {
    if (!w || !flags_out) return fail(KD_ERR_INVALID_ARG, "kd_q8_matrix_status: null argument");
    KD_CK(cudaSetDevice(w->dev));
    KD_CK(cudaDeviceSynchronize());
    int v = 0;
    KD_CK(cudaMemcpy(&v, w->err, sizeof(int), cudaMemcpyDeviceToHost));
    *flags_out = v;
    if (v) {
        KD_CK(cudaMemset(w->err, 0, sizeof(int)));
        KD_CK(cudaMemset(w->cnt, 0, (size_t)w->p.G * sizeof(int)));
        KD_CK(cudaDeviceSynchronize());
        return fail(KD_ERR_DEVICE, "kd_mmvq: a kernel gave up a bounded wait (flags 0x%x)", v);
    }
    return KD_OK;
}

kd_status kd_mmvq_schedule(int32_t rows, int32_t cols, int32_t num_sms, int32_t* mode_out, int32_t* warps_out,
                           int32_t* share_out) {
    if (!mode_out || !warps_out || !share_out) return fail(KD_ERR_INVALID_ARG, "kd_mmvq_schedule: null argument");
    if (num_sms < 1) return fail(KD_ERR_INVALID_ARG, "kd_mmvq_schedule: num_sms=%d", num_sms);
    if (rows < kd::GROUP_ROWS || rows % kd::GROUP_ROWS || cols < kd::KGROUP || cols % kd::KGROUP)
        return fail(KD_ERR_UNSUPPORTED, "kd_mmvq_schedule: need rows %% 32 == 0 and cols %% 128 == 0 (got %d x %d)",
                    rows, cols);
    PackedQ8 p;
    p.rows = rows;
    p.K = cols;
    p.G = rows / kd::GROUP_ROWS;
    p.KG = cols / kd::KGROUP;
    kd::plan_split(p, num_sms);
    *mode_out = p.mode;
    *warps_out = p.W;
    *share_out = p.mode == kd::MMVQ_STREAM ? p.maxc : 1;
    return KD_OK;
}

kd_status kd_argmax(const float* logits, int32_t B, int32_t V, int32_t* out, void* workspace, kd_stream stream) {
    if (!logits || !out || !workspace) return fail(KD_ERR_INVALID_ARG, "kd_argmax: null argument");
    if (B < 1 || B > KD_MAX_BATCH) return fail(KD_ERR_BATCH, "kd_argmax: B=%d outside [1, %d]", B, KD_MAX_BATCH);
    if (V < 1 || V % 4) return fail(KD_ERR_INVALID_ARG, "kd_argmax: V=%d must be a positive multiple of 4", V);
    if ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(workspace)) & 15)
        return fail(KD_ERR_INVALID_ARG, "kd_argmax: logits and workspace must be 16-byte aligned");
    cudaStream_t s = (cudaStream_t)stream;
    int dev = 0;
    KD_CK(cudaGetDevice(&dev));
    KD_CK(init_device_attributes(dev));
    static_assert((KD_MAX_BATCH + 1) * sizeof(unsigned long long) <= KD_ARGMAX_WORKSPACE_BYTES, "argmax workspace");
    auto* keys = reinterpret_cast<unsigned long long*>(workspace);
    KD_CK(cudaMemsetAsync(keys, 0, (KD_MAX_BATCH + 1) * sizeof(unsigned long long), s));
    KD_CK(kd::launch_argmax(logits, B, V, out, keys, reinterpret_cast<unsigned*>(keys + KD_MAX_BATCH), false, s));
    return KD_OK;
}

kd_status kd_sample(const float* logits, int32_t B, int32_t V, const kd_sample_params* params, int32_t* out,
                    void* workspace, kd_stream stream) {
    if (!logits || !params || !out || !workspace) return fail(KD_ERR_INVALID_ARG, "kd_sample: null argument");
    if (B < 1 || B > KD_MAX_BATCH) return fail(KD_ERR_BATCH, "kd_sample: B=%d outside [1, %d]", B, KD_MAX_BATCH);
    if (V < 1 || V % 4) return fail(KD_ERR_INVALID_ARG, "kd_sample: V=%d must be a positive multiple of 4", V);
    if ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(workspace)) & 15)
        return fail(KD_ERR_INVALID_ARG, "kd_sample: logits and workspace must be 16-byte aligned");
    static_assert(256 + kd::SAMP_INTS * sizeof(int32_t) <= KD_SAMPLE_WORKSPACE_BYTES, "sample workspace");
    int32_t q[kd::SAMP_INTS] = {};
    for (int b = 0; b < B; ++b) {
        std::memcpy(&q[b], &params[b].temperature, sizeof(float));
        q[16 + 2 * b] = (int32_t)(uint32_t)params[b].seed;
        q[17 + 2 * b] = (int32_t)(uint32_t)(params[b].seed >> 32);
        q[48 + 2 * b] = (int32_t)(uint32_t)params[b].counter;
        q[49 + 2 * b] = (int32_t)(uint32_t)(params[b].counter >> 32);
    }
    cudaStream_t s = (cudaStream_t)stream;
    int dev = 0;
    KD_CK(cudaGetDevice(&dev));
    KD_CK(init_device_attributes(dev));
    auto* keys = reinterpret_cast<unsigned long long*>(workspace);
    int* dq = reinterpret_cast<int*>(reinterpret_cast<char*>(workspace) + 256);
    KD_CK(cudaMemsetAsync(keys, 0, (KD_MAX_BATCH + 1) * sizeof(unsigned long long), s));
    KD_CK(cudaMemcpyAsync(dq, q, sizeof q, cudaMemcpyHostToDevice, s));
    KD_CK(kd::launch_argmax(logits, B, V, out, keys, reinterpret_cast<unsigned*>(keys + KD_MAX_BATCH), false, s,
                            nullptr, dq));
    return KD_OK;
}

size_t kd_attn_workspace_bytes(int32_t B, int32_t n_heads, int32_t head_dim, int32_t cap) {
    if (B < 1 || n_heads < 1 || head_dim < 1 || cap < 1) return 0;
    const size_t splits = (size_t)(cap + kd::ATT_CHUNK - 1) / kd::ATT_CHUNK;
    return 256 + (size_t)B * n_heads * splits * kd::ATT_REC(head_dim) * sizeof(float);
}

kd_status kd_attn_device_status(const void* workspace, int32_t* flags_out, kd_stream stream) {
    if (!flags_out) return fail(KD_ERR_INVALID_ARG, "kd_attn_device_status: null argument");
    cudaStream_t s = (cudaStream_t)stream;
    KD_CK(cudaStreamSynchronize(s));
    int* word = nullptr;
    if (workspace) {
        word = (int*)workspace + 2 * KD_MAX_BATCH;
    } else {
        int dev = 0;
        KD_CK(cudaGetDevice(&dev));
        KD_CK(kd::noalloc_fault_word(dev, &word));
        if (!word) {  // the allocation-free call never ran on this device: nothing to report
            *flags_out = 0;
            return KD_OK;
        }
    }
    int v = 0;
    KD_CK(cudaMemcpy(&v, word, sizeof(int), cudaMemcpyDeviceToHost));
    *flags_out = v;
    if (v) return fail(KD_ERR_DEVICE, "attention: a kernel gave up a bounded wait (flags 0x%x)", v);
    return KD_OK;
}

kd_status kd_kv_q8_quantize(const float* src, int64_t rows, uint8_t* quants, uint16_t* scales, kd_stream stream) {
    if (!src || !quants || !scales) return fail(KD_ERR_INVALID_ARG, "kd_kv_q8_quantize: null argument");
    if (rows < 1 || rows > 0x7fffffff) return fail(KD_ERR_INVALID_ARG, "kd_kv_q8_quantize: rows=%lld", (long long)rows);
    int dev = 0;
    KD_CK(cudaGetDevice(&dev));
    KD_CK(init_device_attributes(dev));
    KD_CK(kd::launch_kvq8_rows(src, false, (long)rows, 1, (int)rows, (int)rows, 0, 0, quants,
                               reinterpret_cast<__half*>(scales), (cudaStream_t)stream));
    return KD_OK;
}

kd_status kd_attn_append_decode_q8(const float* q, const float* k_new, const float* v_new, uint8_t* k_quants,
                                   uint16_t* k_scales, uint8_t* v_quants, uint16_t* v_scales, const int32_t* slots,
                                   const int32_t* positions, int32_t B, int32_t n_heads, int32_t n_kv_heads,
                                   int32_t n_slots, int32_t cap, uint16_t* out, void* workspace,
                                   size_t workspace_bytes, kd_stream stream) {
    if (!q || !k_new || !v_new || !k_quants || !k_scales || !v_quants || !v_scales || !slots || !positions || !out ||
        !workspace)
        return fail(KD_ERR_INVALID_ARG, "kd_attn_append_decode_q8: null argument");
    if (B < 1 || B > KD_MAX_BATCH) return fail(KD_ERR_BATCH, "kd_attn_append_decode_q8: B=%d", B);
    if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || !kd::attn_q8_supported(128, n_heads / n_kv_heads))
        return fail(KD_ERR_UNSUPPORTED, "kd_attn_append_decode_q8: group %d", n_kv_heads > 0 ? n_heads / n_kv_heads : 0);
    if (n_slots < 1 || cap < 2 || cap % 2) return fail(KD_ERR_INVALID_ARG, "kd_attn_append_decode_q8: n_slots/cap");
    if ((cap + kd::ATT_CHUNK - 1) / kd::ATT_CHUNK > kd::ATT_MAX_SPLITS)
        return fail(KD_ERR_UNSUPPORTED, "kd_attn_append_decode_q8: cap %d exceeds %d", cap,
                    kd::ATT_MAX_SPLITS * kd::ATT_CHUNK);
    if (workspace_bytes < kd_attn_workspace_bytes(B, n_heads, 128, cap))
        return fail(KD_ERR_INVALID_ARG, "kd_attn_append_decode_q8: workspace too small");
    if ((((uintptr_t)workspace | (uintptr_t)k_quants | (uintptr_t)v_quants | (uintptr_t)k_scales |
          (uintptr_t)v_scales | (uintptr_t)q) & 15))
        return fail(KD_ERR_INVALID_ARG, "kd_attn_append_decode_q8: buffers must be 16-byte aligned");
    int32_t desc[2 * KD_MAX_BATCH] = {};
    for (int b = 0; b < B; ++b) {
        if (slots[b] < 0 || slots[b] >= n_slots) return fail(KD_ERR_BAD_SESSION, "slot %d", slots[b]);
        for (int j = 0; j < b; ++j)
            if (slots[j] == slots[b]) return fail(KD_ERR_BAD_SESSION, "slot %d repeated", slots[b]);
        if (positions[b] < 0 || positions[b] >= cap)
            return fail(KD_ERR_POSITION, "position %d outside [0, %d)", positions[b], cap);
        desc[b] = slots[b];
        desc[KD_MAX_BATCH + b] = positions[b];
    }
    cudaStream_t s = (cudaStream_t)stream;
    int dev = 0, sms = 0;
    KD_CK(cudaGetDevice(&dev));
    KD_CK(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    KD_CK(init_device_attributes(dev));
    int* d_desc = (int*)workspace;
    int* d_err = d_desc + 2 * KD_MAX_BATCH;
    KD_CK(cudaMemcpyAsync(d_desc, desc, sizeof desc, cudaMemcpyHostToDevice, s));
    KD_CK(cudaMemsetAsync(d_err, 0, sizeof(int), s));
    __half* ksc = reinterpret_cast<__half*>(k_scales);
    __half* vsc = reinterpret_cast<__half*>(v_scales);
    KD_CK(kd::launch_kvq8_append(k_new, v_new, k_quants, ksc, v_quants, vsc, d_desc, d_desc + KD_MAX_BATCH, B,
                                 n_kv_heads, cap, 0, false, s));
    kd::AttnMaps maps;
    KD_CK(kd::make_attn_q8_maps(k_quants, v_quants, (long)n_slots * n_kv_heads * cap, &maps));
    kd::AttnArgs t{};
    t.q = q; t.row0 = 0; t.slot = d_desc; t.pos = d_desc + KD_MAX_BATCH; t.B = B; t.nh = n_heads; t.nkv = n_kv_heads;
    t.hd = 128; t.cap = cap; t.scale = 1.0f / std::sqrt(128.0f);
    t.part = (float*)((char*)workspace + 256);
    t.max_splits = (cap + kd::ATT_CHUNK - 1) / kd::ATT_CHUNK;
    t.out = (__half*)out;
    t.err = d_err;
    t.ks = ksc;
    t.vs = vsc;
    KD_CK(kd::launch_attn_split_q8(t, maps, sms, false, s));
    KD_CK(kd::launch_attn_combine(t, false, s));
    return KD_OK;
}

kd_status kd_attn_append_decode(const float* q, const float* k_new, const float* v_new, uint16_t* k_cache,
                                uint16_t* v_cache, const int32_t* slots, const int32_t* positions, int32_t B,
                                int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t n_slots,
                                int32_t cap, uint16_t* out, void* workspace, size_t workspace_bytes,
                                kd_stream stream) {
    if (!q || !k_new || !v_new || !k_cache || !v_cache || !slots || !positions || !out || !workspace)
        return fail(KD_ERR_INVALID_ARG, "kd_attn_append_decode: null argument");
    if (B < 1 || B > KD_MAX_BATCH) return fail(KD_ERR_BATCH, "kd_attn_append_decode: B=%d", B);
    if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || !kd::attn_supported(head_dim, n_heads / n_kv_heads))
        return fail(KD_ERR_UNSUPPORTED, "kd_attn_append_decode: head_dim %d, group %d", head_dim,
                    n_kv_heads > 0 ? n_heads / n_kv_heads : 0);
    if (n_slots < 1 || cap < 1) return fail(KD_ERR_INVALID_ARG, "kd_attn_append_decode: n_slots/cap");
    if ((cap + kd::ATT_CHUNK - 1) / kd::ATT_CHUNK > kd::ATT_MAX_SPLITS)
        return fail(KD_ERR_UNSUPPORTED, "kd_attn_append_decode: cap %d exceeds %d", cap,
                    kd::ATT_MAX_SPLITS * kd::ATT_CHUNK);
    if (workspace_bytes < kd_attn_workspace_bytes(B, n_heads, head_dim, cap))
        return fail(KD_ERR_INVALID_ARG, "kd_attn_append_decode: workspace too small");
    if ((((uintptr_t)workspace | (uintptr_t)k_cache | (uintptr_t)v_cache) & 15) || ((uintptr_t)q & 7))
        return fail(KD_ERR_INVALID_ARG, "kd_attn_append_decode: caches and workspace must be 16-byte aligned, q 8-byte");
    int32_t desc[2 * KD_MAX_BATCH] = {};
    for (int b = 0; b < B; ++b) {
        if (slots[b] < 0 || slots[b] >= n_slots) return fail(KD_ERR_BAD_SESSION, "slot %d", slots[b]);
        for (int j = 0; j < b; ++j)
            if (slots[j] == slots[b]) return fail(KD_ERR_BAD_SESSION, "slot %d repeated", slots[b]);
        if (positions[b] < 0 || positions[b] >= cap)
            return fail(KD_ERR_POSITION, "position %d outside [0, %d)", positions[b], cap);
        desc[b] = slots[b];
        desc[KD_MAX_BATCH + b] = positions[b];
    }
    cudaStream_t s = (cudaStream_t)stream;
    int dev = 0, sms = 0;
    KD_CK(cudaGetDevice(&dev));
    KD_CK(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    KD_CK(init_device_attributes(dev));
    int* d_desc = (int*)workspace;
    int* d_err = d_desc + 2 * KD_MAX_BATCH;
    KD_CK(cudaMemcpyAsync(d_desc, desc, sizeof desc, cudaMemcpyHostToDevice, s));
    KD_CK(cudaMemsetAsync(d_err, 0, sizeof(int), s));
    KD_CK(kd::launch_kv_append(k_new, v_new, (__half*)k_cache, (__half*)v_cache, d_desc, d_desc + KD_MAX_BATCH, B,
                               n_kv_heads, head_dim, cap, s));
    kd::AttnMaps maps;
    KD_CK(kd::make_attn_maps((const __half*)k_cache, (const __half*)v_cache, (long)n_slots * n_kv_heads * cap, head_dim,
                              &maps));
    kd::AttnArgs t{};
    t.q = q; t.kc = (const __half*)k_cache; t.vc = (const __half*)v_cache; t.row0 = 0; t.slot = d_desc;
    t.pos = d_desc + KD_MAX_BATCH; t.B = B; t.nh = n_heads; t.nkv = n_kv_heads; t.hd = head_dim; t.cap = cap;
    t.scale = 1.0f / std::sqrt((float)head_dim);
    t.part = (float*)((char*)workspace + 256);
    t.max_splits = (cap + kd::ATT_CHUNK - 1) / kd::ATT_CHUNK;
    t.out = (__half*)out;
    t.err = d_err;
    KD_CK(kd::launch_attn_split(t, maps, kd::attn_split_grid(sms, head_dim, n_heads / n_kv_heads), false, s));
    KD_CK(kd::launch_attn_combine(t, false, s));
    return KD_OK;
}

}  // extern "C"
