// C ABI of the paged Q4_0 cache operators: argument checks, then one launcher
// each.
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv.cuh"

namespace gg {

static gguf_status refuse(gguf_status st, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return report(st, buf);
}
static gguf_status launched(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return GGUF_OK;
    return refuse(GGUF_ERR_CUDA, "%s: CUDA error %d (%s)", what, (int)e, cudaGetErrorString(e));
}
static bool float_type(int t) { return t == GGUF_F32 || t == GGUF_F16 || t == GGUF_BF16; }
static int64_t float_size(int t) { return t == GGUF_F32 ? 4 : 2; }
static bool at(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// every row of an array of rows starts on 16 bytes (or there is none)
static bool rows16(const void *p, int64_t ld, int64_t es) { return p == nullptr || (at(p, 16) && (ld * es) % 16 == 0); }

// sizes that the cache operators share
static gguf_status check_cache(const char *what, int64_t d, int64_t hk, int64_t page, int64_t n_pages) {
    if (d != 64 && d != 128 && d != 256)
        return refuse(GGUF_ERR_SHAPE, "%s: head_dim=%lld is not 64, 128 or 256", what, (long long)d);
    if (hk < 1 || hk > 65535) return refuse(GGUF_ERR_SHAPE, "%s: n_kv_heads=%lld (1..65535)", what, (long long)hk);
    if (page < KV_TILE || page % KV_TILE || page > (1 << 20))
        return refuse(GGUF_ERR_SHAPE, "%s: page_size=%lld is not a multiple of 16 up to 2^20", what, (long long)page);
    if (n_pages < 0 || n_pages > 0x7fffffff) return refuse(GGUF_ERR_INVALID_ARG, "%s: n_pages=%lld", what, (long long)n_pages);
    return GGUF_OK;
}

}  // namespace gg

using namespace gg;

extern "C" {

int64_t gguf_kv_page_bytes(int64_t head_dim, int64_t n_kv_heads, int64_t page_size) {
    if (check_cache("kv_page_bytes", head_dim, n_kv_heads, page_size, 0) != GGUF_OK) return -1;
    return kv_page_bytes(head_dim, n_kv_heads, page_size);
}

gguf_status gguf_kv_plan(const int32_t *ctx_len, const int32_t *new_len, int64_t n_requests,
                         const int32_t *free_pages, int64_t n_free, int32_t *block_table, int64_t ld_table,
                         int64_t width, int64_t page_size, int64_t n_tokens, int32_t *q_start, int32_t *kv_len,
                         int32_t *positions, int64_t *slots, int32_t *pages_used, int32_t *dev_status,
                         gguf_stream_t stream) {
    if (n_requests < 0 || n_free < 0 || n_tokens < 0 || width < 0)
        return report(GGUF_ERR_INVALID_ARG, "kv_plan: negative size");
    if (n_requests > 16384)
        return refuse(GGUF_ERR_SHAPE, "kv_plan: %lld requests (at most 16384)", (long long)n_requests);
    if (n_tokens > 0x7fffffff || n_free > 0x7fffffff || width > 0x7fffffff)
        return report(GGUF_ERR_SHAPE, "kv_plan: n_tokens, n_free and width must fit in 31 bits");
    if (ld_table < width) return refuse(GGUF_ERR_INVALID_ARG, "kv_plan: ld_table=%lld < width=%lld", (long long)ld_table, (long long)width);
    if (page_size < KV_TILE || page_size % KV_TILE || page_size > (1 << 20))
        return refuse(GGUF_ERR_SHAPE, "kv_plan: page_size=%lld is not a multiple of 16 up to 2^20", (long long)page_size);
    if (!q_start || !pages_used || (n_requests > 0 && (!ctx_len || !new_len || !kv_len)) ||
        (n_requests > 0 && width > 0 && !block_table) || (n_free > 0 && !free_pages) ||
        (n_tokens > 0 && (!positions || !slots)))
        return report(GGUF_ERR_INVALID_ARG, "kv_plan: null pointer");
    if (!at(ctx_len, 4) || !at(new_len, 4) || !at(free_pages, 4) || !at(block_table, 4) || !at(q_start, 4) ||
        !at(kv_len, 4) || !at(positions, 4) || !at(slots, 8) || !at(pages_used, 4) || !at(dev_status, 4))
        return report(GGUF_ERR_ALIGNMENT, "kv_plan: misaligned array");
    const KvPlan p{ctx_len, new_len, n_requests, free_pages, n_free, block_table, ld_table, width, page_size,
                   n_tokens, q_start, kv_len, positions, slots, pages_used, dev_status};
    return launched(launch_kv_plan(p, (cudaStream_t)stream), "kv_plan");
}

gguf_status gguf_qk_norm_rope(const gguf_qk_rope_args *a, gguf_stream_t stream) {
    if (!a) return report(GGUF_ERR_INVALID_ARG, "qk_norm_rope: null args");
    if (!float_type(a->xt)) return refuse(GGUF_ERR_UNSUPPORTED_TYPE, "qk_norm_rope: type %d is not F32/BF16/F16", a->xt);
    const bool store = a->cache != nullptr, keys = store || a->k_out != nullptr;
    const int64_t hk = keys ? a->n_kv_heads : 0, d = a->head_dim, es = float_size(a->xt);
    if (a->n_tokens < 0 || a->n_heads < 0 || a->n_positions < 0 || a->rot < 0)
        return report(GGUF_ERR_INVALID_ARG, "qk_norm_rope: negative size");
    gguf_status st = check_cache("qk_norm_rope", d, keys ? hk : 1, store ? a->page_size : KV_TILE, store ? a->n_pages : 0);
    if (st != GGUF_OK) return st;
    if (a->n_heads > 65535 || a->n_tokens > 0x7fffffff)
        return report(GGUF_ERR_SHAPE, "qk_norm_rope: at most 65535 heads and 2^31 - 1 tokens");
    if (a->rope_type != GGUF_ROPE_NORM && a->rope_type != GGUF_ROPE_NEOX)
        return refuse(GGUF_ERR_INVALID_ARG, "qk_norm_rope: rope_type %d", a->rope_type);
    if (a->rot % 16 || a->rot > d)
        return refuse(GGUF_ERR_SHAPE, "qk_norm_rope: rot=%lld is not a multiple of 16 up to head_dim", (long long)a->rot);
    if (a->ldq < a->n_heads * d || a->ldqo < a->n_heads * d || (keys && a->ldk < hk * d) ||
        (store && a->ldv < hk * d) || (a->k_out && a->ldko < hk * d))
        return report(GGUF_ERR_INVALID_ARG, "qk_norm_rope: a row stride is shorter than the row");
    if (a->n_tokens == 0 || a->n_heads + hk == 0) return GGUF_OK;
    if (!a->positions || (a->n_heads > 0 && (!a->q || !a->q_out)) || (keys && !a->k) || (store && (!a->v || !a->slots)) ||
        (a->rot > 0 && !a->cos_sin))
        return report(GGUF_ERR_INVALID_ARG, "qk_norm_rope: null pointer");
    if (!at(a->q, es) || !at(a->k, es) || !at(a->v, es) || !at(a->q_out, es) || !at(a->k_out, es) ||
        !at(a->positions, 4) || !at(a->slots, 8) || !at(a->dev_status, 4))
        return report(GGUF_ERR_ALIGNMENT, "qk_norm_rope: misaligned array");
    if (!at(a->q_norm, 16) || !at(a->k_norm, 16) || !at(a->cos_sin, 16) || !at(a->cache, 16))
        return report(GGUF_ERR_ALIGNMENT, "qk_norm_rope: q_norm, k_norm, cos_sin and cache must be 16-byte aligned");
    const QkRope p{a->q, a->k, a->v, a->ldq, a->ldk, a->ldv, a->n_tokens, a->n_heads, hk,
                   a->n_heads + hk, a->q_norm, a->k_norm, a->eps, a->positions,
                   a->cos_sin, a->rot > 0 ? a->n_positions : INT64_MAX, (int)a->rot, a->rope_type == GGUF_ROPE_NEOX, a->q_out, a->k_out,
                   a->ldqo, a->ldko, (uint8_t *)a->cache, a->n_pages, a->page_size, a->slots, a->dev_status};
    const bool vec = rows16(a->q, a->ldq, es) && rows16(keys ? a->k : nullptr, a->ldk, es) &&
                     rows16(store ? a->v : nullptr, a->ldv, es) && rows16(a->q_out, a->ldqo, es) &&
                     rows16(a->k_out, a->ldko, es);
    return launched(launch_qk_norm_rope(p, d, a->xt, vec, (cudaStream_t)stream), "qk_norm_rope");
}

gguf_status gguf_kv_get_rows(const void *cache, int64_t n_pages, int64_t page_size, int64_t n_kv_heads,
                             int64_t head_dim, const int64_t *slots, int64_t n, void *k, void *v, int ot,
                             gguf_stream_t stream) {
    if (!float_type(ot)) return refuse(GGUF_ERR_UNSUPPORTED_TYPE, "kv_get_rows: out type %d is not F32/BF16/F16", ot);
    gguf_status st = check_cache("kv_get_rows", head_dim, n_kv_heads, page_size, n_pages);
    if (st != GGUF_OK) return st;
    if (n < 0) return report(GGUF_ERR_INVALID_ARG, "kv_get_rows: negative size");
    if (n > 0x7fffffff || n * n_kv_heads > ((int64_t)1 << 33))
        return report(GGUF_ERR_SHAPE, "kv_get_rows: too many rows for one call");
    if (n == 0) return GGUF_OK;
    if (!slots || !k || !v || (n_pages > 0 && !cache)) return report(GGUF_ERR_INVALID_ARG, "kv_get_rows: null pointer");
    if (!at(cache, 16) || !at(slots, 8) || !at(k, float_size(ot)) || !at(v, float_size(ot)))
        return report(GGUF_ERR_ALIGNMENT, "kv_get_rows: misaligned cache, slots, k or v");
    const KvRows p{(const uint8_t *)cache, n_pages, page_size, n_kv_heads, slots, n, k, v};
    return launched(launch_kv_get_rows(p, head_dim, ot, at(k, 16) && at(v, 16), (cudaStream_t)stream), "kv_get_rows");
}

// Positions are below 2^31: a window as wide as that hides nothing, and first tokens past it are all tokens.  No request has
// more queries than the call.  With these bounds set here, sums of the three fit in 64 bits.
static Attn attn_of(const gguf_attn_args *a) {
    constexpr int64_t FAR = (int64_t)1 << 31;
    return Attn{a->q, a->qt, a->n_tokens, a->ldq, (const uint8_t *)a->cache, a->n_pages, a->page_size, a->block_table,
                a->ld_table, a->width, a->q_start, a->kv_len, a->n_requests, std::min(a->max_q_len, a->n_tokens), a->n_heads,
                a->n_kv_heads, a->scale, a->window < FAR ? a->window : 0, std::min(a->sinks, FAR), a->out, a->ldo, a->dev_status};
}

// the checks that the workspace size depends on
static gguf_status check_attn_sizes(const gguf_attn_args *a) {
    if (!a) return report(GGUF_ERR_INVALID_ARG, "paged_attention: null args");
    if (!float_type(a->qt)) return refuse(GGUF_ERR_UNSUPPORTED_TYPE, "paged_attention: type %d is not F32/BF16/F16", a->qt);
    gguf_status st = check_cache("paged_attention", a->head_dim, a->n_kv_heads, a->page_size, a->n_pages);
    if (st != GGUF_OK) return st;
    if (a->n_tokens < 0 || a->n_requests < 0 || a->width < 0 || a->window < 0 || a->sinks < 0)
        return report(GGUF_ERR_INVALID_ARG, "paged_attention: negative size");
    if (a->n_heads < 1 || a->n_heads > 65535 || a->n_heads % a->n_kv_heads)
        return refuse(GGUF_ERR_SHAPE, "paged_attention: n_heads=%lld is not a multiple of n_kv_heads=%lld (at most 65535)",
                      (long long)a->n_heads, (long long)a->n_kv_heads);
    if (a->n_tokens > 0x7fffffff || a->width > 0x7fffffff)
        return report(GGUF_ERR_SHAPE, "paged_attention: n_tokens and width must fit in 31 bits");
    if (a->n_requests > 16384)
        return refuse(GGUF_ERR_SHAPE, "paged_attention: %lld requests (at most 16384)", (long long)a->n_requests);
    if (a->max_q_len < 1) return report(GGUF_ERR_INVALID_ARG, "paged_attention: max_q_len must be positive");
    return GGUF_OK;
}

size_t gguf_paged_attention_ws_size(const gguf_attn_args *a) {
    if (check_attn_sizes(a) != GGUF_OK || a->n_tokens == 0 || a->n_requests == 0) return 0;
    return attn_ws_size(attn_of(a), a->head_dim);
}

gguf_status gguf_paged_attention(const gguf_attn_args *a, void *ws, size_t ws_bytes, gguf_stream_t stream) {
    gguf_status st = check_attn_sizes(a);
    if (st != GGUF_OK) return st;
    const int64_t row = a->n_heads * a->head_dim, es = float_size(a->qt);
    if (a->ldq < row || a->ldo < row || a->ld_table < a->width)
        return report(GGUF_ERR_INVALID_ARG, "paged_attention: a row stride is shorter than the row");
    if (!(a->scale > 0.0f) || a->scale > 3e38f) return report(GGUF_ERR_INVALID_ARG, "paged_attention: scale must be positive and finite");
    if (a->n_tokens == 0 || a->n_requests == 0) return GGUF_OK;
    // fp32 queries walk over the tokens in groups of 8 rows: a request's groups x heads x tiles of 16 tokens are counted
    // in 32 bits
    if (a->qt == GGUF_F32) {
        const double tiles = (double)a->width * (double)a->page_size / KV_TILE;
        const double groups = (double)std::min<int64_t>(a->max_q_len, a->n_tokens) * (double)(a->n_heads / a->n_kv_heads) / 8.0 + 1.0;
        if (tiles * groups * (double)a->n_kv_heads > 4.0e9)
            return report(GGUF_ERR_SHAPE, "paged_attention: too many fp32 queries over too wide a table for one call; split it");
    }
    if (!a->q || !a->out || !a->q_start || !a->kv_len || (a->n_pages > 0 && !a->cache) || (a->width > 0 && !a->block_table))
        return report(GGUF_ERR_INVALID_ARG, "paged_attention: null pointer");
    if (!at(a->q, es) || !at(a->out, es) || !at(a->cache, 16) || !at(a->block_table, 4) || !at(a->q_start, 4) ||
        !at(a->kv_len, 4) || !at(a->dev_status, 4))
        return report(GGUF_ERR_ALIGNMENT, "paged_attention: cache must be 16-byte aligned, the arrays by their elements");
    const Attn p = attn_of(a);
    const size_t need = attn_ws_size(p, a->head_dim);
    if (ws_bytes < need || (need > 0 && !ws))
        return refuse(GGUF_ERR_WORKSPACE, "paged_attention: workspace of %zu bytes < required %zu", ws_bytes, need);
    if (need > 0 && !at(ws, 16)) return report(GGUF_ERR_ALIGNMENT, "paged_attention: workspace must be 16-byte aligned");
    return launched(launch_attn(p, a->head_dim, ws, (cudaStream_t)stream), "paged_attention");
}

}  // extern "C"
