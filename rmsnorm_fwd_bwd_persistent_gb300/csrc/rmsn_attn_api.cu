// rmsn_attn_api.cu -- entry points of the norms inside attention and of the 4-bit cache:
// argument checks (before anything is enqueued) and dispatch.
#include <cfloat>
#include <cmath>

#include "rmsn.h"
#include "rmsn_internal.h"
#include "rmsn_kv4.cuh"

namespace {

using rmsn::Heads;

constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxStride = (int64_t)1 << 40;  // elements; keeps every product in 64 bits

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool valid_dtype(int dt) { return dt == RMSN_F32 || dt == RMSN_BF16; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? RMSN_OK : RMSN_ERR_CUDA; }

// Runs a launcher; nothing it may throw (its caches allocate) leaves a C entry point.
template <typename F>
int launched(F f) {
    try {
        return from_cuda(f());
    } catch (...) {
        return RMSN_ERR_CUDA;
    }
}
bool head_size_ok(int64_t D) { return D >= 16 && D <= 256 && D % 16 == 0; }
bool cache_head_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }

// The strides of one tensor: an axis of length 1 (or less) has none.
int check_heads(const rmsn_heads_t* h, int64_t B, int64_t T, int64_t D, int dt, bool output,
                Heads* out) {
    if (!h || h->heads < 1 || h->heads > kMaxHeads) return RMSN_ERR_INVALID_ARG;
    if (B * T == 0) return RMSN_OK;
    if (!h->data) return RMSN_ERR_INVALID_ARG;
    struct Axis {
        int64_t n, s;
    } ax[3] = {{B, h->batch_stride}, {T, h->token_stride}, {h->heads, h->head_stride}};
    const int64_t vec = dt == RMSN_BF16 ? 8 : 4;
    if (!aligned(h->data, 16)) return RMSN_ERR_MISALIGNED;
    for (Axis& a : ax) {
        if (a.n <= 1) a.s = 0;
        if (a.s < 0 || a.s > kMaxStride) return RMSN_ERR_INVALID_ARG;
        if (a.s % vec != 0) return RMSN_ERR_MISALIGNED;
    }
    // what the strides span stays far from 64 bits (an axis has below 2^31 steps of 2^40 at most)
    __int128 extent = D;
    for (const Axis& a : ax) extent += (__int128)(a.n > 1 ? a.n - 1 : 0) * a.s;
    if (extent > ((__int128)1 << 47)) return RMSN_ERR_INVALID_ARG;
    out->p = h->data;
    out->sb = ax[0].s;
    out->st = ax[1].s;
    out->sh = ax[2].s;
    if (output) {  // in order of stride, each axis must step over all that the smaller ones span
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2 - i; ++j)
                if (ax[j].s > ax[j + 1].s) {
                    const Axis t = ax[j];
                    ax[j] = ax[j + 1];
                    ax[j + 1] = t;
                }
        int64_t span = D;
        for (const Axis& a : ax)
            if (a.n > 1) {
                if (a.s < span) return RMSN_ERR_INVALID_ARG;
                span += (a.n - 1) * a.s;
            }
    }
    return RMSN_OK;
}

int check_rope(const rmsn_rope_t* r, int64_t B, int64_t T, int64_t D, rmsn::Rope* out) {
    if (!r) return RMSN_ERR_INVALID_ARG;
    if (r->rot_dim < 16 || r->rot_dim > D || r->rot_dim % 16 != 0) return RMSN_ERR_UNSUPPORTED_SHAPE;
    if (r->rows < 1 || r->rows > ((int64_t)1 << 40)) return RMSN_ERR_INVALID_ARG;
    const int64_t sb = B > 1 ? r->pos_batch_stride : 0, st = T > 1 ? r->pos_token_stride : 0;
    if (sb < 0 || st < 0 || sb > kMaxStride || st > kMaxStride) return RMSN_ERR_INVALID_ARG;
    if (B * T == 0) return RMSN_OK;
    if (!r->cos || !r->sin || !r->positions) return RMSN_ERR_INVALID_ARG;
    if (!aligned(r->cos, 16) || !aligned(r->sin, 16) || !aligned(r->positions, 8))
        return RMSN_ERR_MISALIGNED;
    *out = {r->cos, r->sin, r->positions, sb, st, r->rows, (int)r->rot_dim};
    return RMSN_OK;
}

int check_sizes(int64_t B, int64_t T, int64_t D, float eps) {
    if (B < 0 || T < 0 || !(eps >= 0.f) || eps > FLT_MAX) return RMSN_ERR_INVALID_ARG;
    if (!head_size_ok(D)) return RMSN_ERR_UNSUPPORTED_SHAPE;
    const int64_t most = ((int64_t)1 << 31) - 1;
    if (B > most || T > most || B * T > most) return RMSN_ERR_UNSUPPORTED_SHAPE;
    return RMSN_OK;
}

int check_cache(const rmsn_kv4_t* c, int64_t D, bool used) {
    if (!c) return RMSN_ERR_INVALID_ARG;
    if (!cache_head_ok(D)) return RMSN_ERR_UNSUPPORTED_SHAPE;
    if (c->pages < 1 || c->kv_heads < 1 || c->kv_heads > kMaxHeads) return RMSN_ERR_INVALID_ARG;
    if (c->page_size < rmsn::kKv4Block || c->page_size % rmsn::kKv4Block != 0)
        return RMSN_ERR_UNSUPPORTED_SHAPE;
    const int64_t most = ((int64_t)1 << 31) - 1, nb = c->page_size / rmsn::kKv4Block;
    if (c->pages > most || nb > most / c->kv_heads || c->pages > most / (c->kv_heads * nb))
        return RMSN_ERR_UNSUPPORTED_SHAPE;
    if (!used) return RMSN_OK;
    if (!c->data) return RMSN_ERR_INVALID_ARG;
    return aligned(c->data, 16) ? RMSN_OK : RMSN_ERR_MISALIGNED;
}

int check_weights(const void* wq, const void* wk, int w_dtype) {
    if (!valid_dtype(w_dtype)) return RMSN_ERR_INVALID_ARG;
    if (!wq || !wk) return RMSN_ERR_INVALID_ARG;
    return aligned(wq, 16) && aligned(wk, 16) ? RMSN_OK : RMSN_ERR_MISALIGNED;
}

#define RMSN_CHECK(call)                     \
    do {                                     \
        const int st_ = (call);              \
        if (st_ != RMSN_OK) return st_;      \
    } while (0)

// What both directions of the training op share.
int check_qk(const rmsn_heads_t* q, const rmsn_heads_t* k, int x_dtype, const void* wq,
             const void* wk, int w_dtype, const rmsn_rope_t* rope, const rmsn_heads_t* yq,
             const rmsn_heads_t* yk, int64_t B, int64_t T, int64_t D, float eps,
             rmsn::QkCall* c) {
    if (!valid_dtype(x_dtype)) return RMSN_ERR_INVALID_ARG;
    RMSN_CHECK(check_sizes(B, T, D, eps));
    if (!q || !k || !yq || !yk || yq->heads != q->heads || yk->heads != k->heads)
        return RMSN_ERR_INVALID_ARG;
    RMSN_CHECK(check_heads(q, B, T, D, x_dtype, false, &c->x[0]));
    RMSN_CHECK(check_heads(k, B, T, D, x_dtype, false, &c->x[1]));
    RMSN_CHECK(check_heads(yq, B, T, D, x_dtype, true, &c->y[0]));
    RMSN_CHECK(check_heads(yk, B, T, D, x_dtype, true, &c->y[1]));
    RMSN_CHECK(check_rope(rope, B, T, D, &c->rope));
    RMSN_CHECK(check_weights(wq, wk, w_dtype));
    c->w[0] = wq;
    c->w[1] = wk;
    c->heads[0] = (int)q->heads;
    c->heads[1] = (int)k->heads;
    c->tokens = B * T;
    c->T = T;
    c->D = (int)D;
    c->x_dt = x_dtype;
    c->w_dt = w_dtype;
    c->neighbours = rope->neighbours != 0;
    c->eps = eps;
    return RMSN_OK;
}

}  // namespace

extern "C" {

int qk_norm_rope_fwd(const rmsn_heads_t* q, const rmsn_heads_t* k, int x_dtype, const void* wq,
                     const void* wk, int w_dtype, const rmsn_rope_t* rope,
                     const rmsn_heads_t* q_out, const rmsn_heads_t* k_out, int64_t B, int64_t T,
                     int64_t D, float eps, rmsn_stream_t stream) {
    rmsn::QkCall c{};
    RMSN_CHECK(check_qk(q, k, x_dtype, wq, wk, w_dtype, rope, q_out, k_out, B, T, D, eps, &c));
    if (c.tokens == 0) return RMSN_OK;
    uint64_t limit;
    RMSN_CHECK(rmsn::device_facts(&c.sms, &c.err, &limit));
    return launched([&] { return rmsn::launch_qk(c, reinterpret_cast<cudaStream_t>(stream)); });
}

size_t qk_norm_rope_bwd_workspace_bytes(int64_t D, int device) {
    int sms = 0;
    if (!head_size_ok(D) || device < 0 ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return (size_t)sms * rmsn::kQkBwdCtasPerSm * 2 * D * sizeof(float);
}

int qk_norm_rope_bwd(const rmsn_heads_t* gq, const rmsn_heads_t* gk, const rmsn_heads_t* q,
                     const rmsn_heads_t* k, int x_dtype, const void* wq, const void* wk,
                     int w_dtype, const rmsn_rope_t* rope, const rmsn_heads_t* dq,
                     const rmsn_heads_t* dk, float* dwq, float* dwk, int64_t B, int64_t T,
                     int64_t D, float eps, void* workspace, size_t workspace_bytes,
                     rmsn_stream_t stream) {
    rmsn::QkCall c{};
    RMSN_CHECK(check_qk(q, k, x_dtype, wq, wk, w_dtype, rope, dq, dk, B, T, D, eps, &c));
    if (!gq || !gk || gq->heads != q->heads || gk->heads != k->heads || !dwq || !dwk)
        return RMSN_ERR_INVALID_ARG;
    RMSN_CHECK(check_heads(gq, B, T, D, x_dtype, false, &c.g[0]));
    RMSN_CHECK(check_heads(gk, B, T, D, x_dtype, false, &c.g[1]));
    if (!aligned(dwq, 4) || !aligned(dwk, 4)) return RMSN_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (c.tokens == 0) {
        cudaError_t e = cudaMemsetAsync(dwq, 0, (size_t)D * sizeof(float), s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dwk, 0, (size_t)D * sizeof(float), s);
        return from_cuda(e);
    }
    if (!workspace) return workspace_bytes ? RMSN_ERR_INVALID_ARG : RMSN_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 16)) return RMSN_ERR_MISALIGNED;
    uint64_t limit;
    RMSN_CHECK(rmsn::device_facts(&c.sms, &c.err, &limit));
    if (workspace_bytes < (size_t)c.sms * rmsn::kQkBwdCtasPerSm * 2 * D * sizeof(float))
        return RMSN_ERR_WORKSPACE_TOO_SMALL;
    c.ws = static_cast<float*>(workspace);
    c.dw[0] = dwq;
    c.dw[1] = dwk;
    return launched([&] { return rmsn::launch_qk(c, s); });
}

int qk_norm_rope_kv4_append(const rmsn_heads_t* q, const rmsn_heads_t* k, const rmsn_heads_t* v,
                            const void* wq, const void* wk, int w_dtype, const rmsn_rope_t* rope,
                            const rmsn_heads_t* q_out, const rmsn_kv4_t* cache,
                            const int64_t* slots, int64_t T, int64_t D, float eps,
                            rmsn_stream_t stream) {
    rmsn::Kv4Append c{};
    RMSN_CHECK(check_sizes(1, T, D, eps));
    RMSN_CHECK(check_cache(cache, D, T > 0));
    if (!q || !k || !v || !q_out || q_out->heads != q->heads || k->heads != cache->kv_heads ||
        v->heads != cache->kv_heads)
        return RMSN_ERR_INVALID_ARG;
    RMSN_CHECK(check_heads(q, 1, T, D, RMSN_BF16, false, &c.x[0]));
    RMSN_CHECK(check_heads(k, 1, T, D, RMSN_BF16, false, &c.x[1]));
    RMSN_CHECK(check_heads(v, 1, T, D, RMSN_BF16, false, &c.x[2]));
    RMSN_CHECK(check_heads(q_out, 1, T, D, RMSN_BF16, true, &c.y));
    RMSN_CHECK(check_rope(rope, 1, T, D, &c.rope));
    RMSN_CHECK(check_weights(wq, wk, w_dtype));
    if (T == 0) return RMSN_OK;
    if (!slots) return RMSN_ERR_INVALID_ARG;
    if (!aligned(slots, 8)) return RMSN_ERR_MISALIGNED;
    uint64_t limit;
    RMSN_CHECK(rmsn::device_facts(&c.sms, &c.err, &limit));
    c.w[0] = wq;
    c.w[1] = wk;
    c.cache = static_cast<uint8_t*>(cache->data);
    c.slots = slots;
    c.tokens = T;
    c.pages = cache->pages;
    c.heads = (int)q->heads;
    c.kv_heads = (int)cache->kv_heads;
    c.blocks_per_page = (int)(cache->page_size / rmsn::kKv4Block);
    c.D = (int)D;
    c.w_dt = w_dtype;
    c.neighbours = rope->neighbours != 0;
    c.eps = eps;
    return launched([&] { return rmsn::launch_kv4_append(c, reinterpret_cast<cudaStream_t>(stream)); });
}

int kv4_read(const rmsn_kv4_t* cache, const int64_t* slots, const rmsn_heads_t* k,
             const rmsn_heads_t* v, int64_t T, int64_t D, rmsn_stream_t stream) {
    rmsn::Kv4Read c{};
    RMSN_CHECK(check_sizes(1, T, D, 0.f));
    RMSN_CHECK(check_cache(cache, D, T > 0));
    if (!k || !v || k->heads != cache->kv_heads || v->heads != cache->kv_heads)
        return RMSN_ERR_INVALID_ARG;
    RMSN_CHECK(check_heads(k, 1, T, D, RMSN_BF16, true, &c.k));
    RMSN_CHECK(check_heads(v, 1, T, D, RMSN_BF16, true, &c.v));
    if (T == 0) return RMSN_OK;
    if (!slots) return RMSN_ERR_INVALID_ARG;
    if (!aligned(slots, 8)) return RMSN_ERR_MISALIGNED;
    uint64_t limit;
    RMSN_CHECK(rmsn::device_facts(&c.sms, &c.err, &limit));
    c.cache = static_cast<const uint8_t*>(cache->data);
    c.slots = slots;
    c.tokens = T;
    c.pages = cache->pages;
    c.kv_heads = (int)cache->kv_heads;
    c.blocks_per_page = (int)(cache->page_size / rmsn::kKv4Block);
    c.D = (int)D;
    return launched([&] { return rmsn::launch_kv4_read(c, reinterpret_cast<cudaStream_t>(stream)); });
}

size_t kv4_attention_workspace_bytes(int64_t seqs, int64_t D, int device) {
    int sms = 0;
    if (seqs < 0 || seqs > ((int64_t)1 << 31) - 1 || !cache_head_ok(D) || device < 0 ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return (size_t)rmsn::kv4_attention_workspace((int)seqs, (int)D, sms);
}

int kv4_attention(const rmsn_heads_t* q, const rmsn_kv4_t* cache, const int32_t* page_table,
                  int64_t table_width, int64_t table_stride, const int32_t* kv_lens,
                  const int32_t* cu_q, int64_t max_q, int64_t seqs, int64_t T, int64_t D,
                  float scale, const rmsn_heads_t* out, float* lse, void* workspace,
                  size_t workspace_bytes, rmsn_stream_t stream) {
    rmsn::Kv4Attention c{};
    Heads hq{}, ho{};
    RMSN_CHECK(check_sizes(1, T, D, 0.f));
    RMSN_CHECK(check_cache(cache, D, T > 0));
    const int64_t most = ((int64_t)1 << 31) - 1;
    if (seqs < 0 || seqs >= most || max_q < 1 || !std::isfinite(scale)) return RMSN_ERR_INVALID_ARG;
    if (!q || !out || out->heads != q->heads || q->heads % cache->kv_heads != 0)
        return RMSN_ERR_INVALID_ARG;
    RMSN_CHECK(check_heads(q, 1, T, D, RMSN_BF16, false, &hq));
    RMSN_CHECK(check_heads(out, 1, T, D, RMSN_BF16, true, &ho));
    if (table_width < 0 || table_stride < table_width) return RMSN_ERR_INVALID_ARG;
    // token indexes past a sequence's end (partial units, columns) stay in 32 bits
    if (table_width > ((int64_t)1 << 30) / cache->page_size || table_stride > kMaxStride)
        return RMSN_ERR_UNSUPPORTED_SHAPE;
    if (!cu_q && T != seqs) return RMSN_ERR_INVALID_ARG;
    // (query token, head) columns and all units of the work split stay in range
    if (T > (most - 1024) / q->heads) return RMSN_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || seqs == 0) return RMSN_OK;
    if (!kv_lens || (!page_table && table_width > 0)) return RMSN_ERR_INVALID_ARG;
    if (!aligned(kv_lens, 4) || !aligned(page_table, 4) || !aligned(cu_q, 4) || !aligned(lse, 4))
        return RMSN_ERR_MISALIGNED;
    if (!workspace) return workspace_bytes ? RMSN_ERR_INVALID_ARG : RMSN_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 16)) return RMSN_ERR_MISALIGNED;
    RMSN_CHECK(rmsn::device_facts(&c.sms, &c.err, &c.limit_ns));
    if ((int64_t)workspace_bytes < rmsn::kv4_attention_workspace((int)seqs, (int)D, c.sms))
        return RMSN_ERR_WORKSPACE_TOO_SMALL;
    c.q = hq.p;
    c.q_st = hq.st;
    c.q_sh = hq.sh;
    c.out = ho.p;
    c.out_st = ho.st;
    c.out_sh = ho.sh;
    c.lse = lse;
    c.cache = static_cast<const uint8_t*>(cache->data);
    c.page_table = page_table;
    c.table_stride = table_stride;
    c.kv_lens = kv_lens;
    c.cu_q = cu_q;
    c.ws = workspace;
    c.pages = cache->pages;
    c.tokens = (int)T;
    c.seqs = (int)seqs;
    c.heads = (int)q->heads;
    c.kv_heads = (int)cache->kv_heads;
    c.table_width = (int)table_width;
    c.blocks_per_page = (int)(cache->page_size / rmsn::kKv4Block);
    c.max_q = (int)(max_q < T ? max_q : T);
    c.D = (int)D;
    c.scale = scale;
    return launched([&] { return rmsn::launch_kv4_attention(c, reinterpret_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
