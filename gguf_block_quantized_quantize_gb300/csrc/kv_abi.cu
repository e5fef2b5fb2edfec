// C ABI of the paged Q4_0 cache operators: argument checks, then one launcher
// each.
#include <algorithm>

#include "abi_checks.h"
#include "common.cuh"
#include "internal.h"
#include "kv.cuh"

namespace gg {

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

// one position a token (axes null), or a position on each axis
static gguf_status qk_norm_rope(const gguf_qk_rope_args *a, const gguf_rope_axes *axes, const char *what, cudaStream_t stream) {
    if (!a) return refuse(GGUF_ERR_INVALID_ARG, "%s: null args", what);
    if (!float_type(a->xt)) return refuse(GGUF_ERR_UNSUPPORTED_TYPE, "%s: type %d is not F32/BF16/F16", what, a->xt);
    const bool store = a->cache != nullptr, keys = store || a->k_out != nullptr;
    const int64_t hk = keys ? a->n_kv_heads : 0, d = a->head_dim, es = float_size(a->xt);
    if (a->n_tokens < 0 || a->n_heads < 0 || a->n_positions < 0 || a->rot < 0)
        return refuse(GGUF_ERR_INVALID_ARG, "%s: negative size", what);
    gguf_status st = check_cache(what, d, keys ? hk : 1, store ? a->page_size : KV_TILE, store ? a->n_pages : 0);
    if (st != GGUF_OK) return st;
    if (a->n_heads > 65535 || a->n_tokens > 0x7fffffff)
        return refuse(GGUF_ERR_SHAPE, "%s: at most 65535 heads and 2^31 - 1 tokens", what);
    if (a->rope_type != GGUF_ROPE_NORM && a->rope_type != GGUF_ROPE_NEOX)
        return refuse(GGUF_ERR_INVALID_ARG, "%s: rope_type %d", what, a->rope_type);
    if (a->rot % 16 || a->rot > d)
        return refuse(GGUF_ERR_SHAPE, "%s: rot=%lld is not a multiple of 16 up to head_dim", what, (long long)a->rot);
    if (axes) {
        if (axes->n_axes < 1 || axes->n_axes > GGUF_MAX_AXES)
            return refuse(GGUF_ERR_SHAPE, "%s: %lld axes (1..%d)", what, (long long)axes->n_axes, GGUF_MAX_AXES);
        int64_t pairs = 0;
        for (int i = 0; i < axes->n_axes; i++) {
            if (axes->sections[i] < 0) return refuse(GGUF_ERR_INVALID_ARG, "%s: negative section", what);
            pairs += axes->sections[i];
        }
        if (pairs != a->rot / 2)
            return refuse(GGUF_ERR_SHAPE, "%s: the sections hold %lld pairs, rot=%lld has %lld", what, (long long)pairs, (long long)a->rot,
                          (long long)(a->rot / 2));
        if (axes->n_axes > 1 && axes->ld_positions != 0 && axes->ld_positions < a->n_tokens)
            return refuse(GGUF_ERR_INVALID_ARG, "%s: ld_positions=%lld < n_tokens", what, (long long)axes->ld_positions);
    }
    if (a->ldq < a->n_heads * d || a->ldqo < a->n_heads * d || (keys && a->ldk < hk * d) ||
        (store && a->ldv < hk * d) || (a->k_out && a->ldko < hk * d))
        return refuse(GGUF_ERR_INVALID_ARG, "%s: a row stride is shorter than the row", what);
    if (a->n_tokens == 0 || a->n_heads + hk == 0) return GGUF_OK;
    if (!a->positions || (a->n_heads > 0 && (!a->q || !a->q_out)) || (keys && !a->k) || (store && (!a->v || !a->slots)) ||
        (a->rot > 0 && !a->cos_sin))
        return refuse(GGUF_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!at(a->q, es) || !at(a->k, es) || !at(a->v, es) || !at(a->q_out, es) || !at(a->k_out, es) ||
        !at(a->positions, 4) || !at(a->slots, 8) || !at(a->dev_status, 4))
        return refuse(GGUF_ERR_ALIGNMENT, "%s: misaligned array", what);
    if (!at(a->q_norm, 16) || !at(a->k_norm, 16) || !at(a->cos_sin, 16) || !at(a->cache, 16))
        return refuse(GGUF_ERR_ALIGNMENT, "%s: q_norm, k_norm, cos_sin and cache must be 16-byte aligned", what);
    QkRope p{a->q, a->k, a->v, a->ldq, a->ldk, a->ldv, a->n_tokens, a->n_heads, hk,
             a->q_norm, a->k_norm, a->eps, a->positions,
                   a->cos_sin, a->rot > 0 ? a->n_positions : INT64_MAX, (int)a->rot, a->rope_type == GGUF_ROPE_NEOX, a->q_out, a->k_out,
                   a->ldqo, a->ldko, (uint8_t *)a->cache, a->n_pages, a->page_size, a->slots, a->dev_status, 1, 0, {}};
    if (axes) {
        p.n_axes = (int)axes->n_axes;
        p.ldpos = axes->ld_positions;
        int left[GGUF_MAX_AXES] = {}, on = 0;   // pairs that an axis has left; the axis of the next pair
        for (int i = 0; i < p.n_axes; i++) left[i] = axes->sections[i];
        for (int i = 0; i < a->rot / 2; i++) {
            while (left[on] == 0) on = (on + 1) % p.n_axes;
            p.axis_of[i / 8] |= (uint16_t)(on << (2 * (i % 8)));
            left[on]--;
            if (axes->interleaved) on = (on + 1) % p.n_axes;
        }
    }
    const bool vec = rows16(a->q, a->ldq, es) && rows16(keys ? a->k : nullptr, a->ldk, es) &&
                     rows16(store ? a->v : nullptr, a->ldv, es) && rows16(a->q_out, a->ldqo, es) &&
                     rows16(a->k_out, a->ldko, es);
    return launched(launch_qk_norm_rope(p, d, a->xt, vec, stream), what);
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
    return qk_norm_rope(a, nullptr, "qk_norm_rope", (cudaStream_t)stream);
}

gguf_status gguf_qk_norm_mrope(const gguf_qk_rope_args *a, const gguf_rope_axes *axes, gguf_stream_t stream) {
    if (!axes) return report(GGUF_ERR_INVALID_ARG, "qk_norm_mrope: null axes");
    return qk_norm_rope(a, axes, "qk_norm_mrope", (cudaStream_t)stream);
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
static gguf_status check_attn_sizes(const gguf_attn_args *a, const char *what) {
    if (!a) return refuse(GGUF_ERR_INVALID_ARG, "%s: null args", what);
    if (!float_type(a->qt)) return refuse(GGUF_ERR_UNSUPPORTED_TYPE, "%s: type %d is not F32/BF16/F16", what, a->qt);
    gguf_status st = check_cache(what, a->head_dim, a->n_kv_heads, a->page_size, a->n_pages);
    if (st != GGUF_OK) return st;
    if (a->n_tokens < 0 || a->n_requests < 0 || a->width < 0 || a->window < 0 || a->sinks < 0)
        return refuse(GGUF_ERR_INVALID_ARG, "%s: negative size", what);
    if (a->n_heads < 1 || a->n_heads > 65535 || a->n_heads % a->n_kv_heads)
        return refuse(GGUF_ERR_SHAPE, "%s: n_heads=%lld is not a multiple of n_kv_heads=%lld (at most 65535)", what,
                      (long long)a->n_heads, (long long)a->n_kv_heads);
    if (a->n_tokens > 0x7fffffff || a->width > 0x7fffffff)
        return refuse(GGUF_ERR_SHAPE, "%s: n_tokens and width must fit in 31 bits", what);
    if (a->n_requests > 16384)
        return refuse(GGUF_ERR_SHAPE, "%s: %lld requests (at most 16384)", what, (long long)a->n_requests);
    if (a->max_q_len < 1) return refuse(GGUF_ERR_INVALID_ARG, "%s: max_q_len must be positive", what);
    return GGUF_OK;
}

static gguf_status check_attn_rows(const gguf_attn_args *a, const char *what) {
    const int64_t row = a->n_heads * a->head_dim;
    if (a->ldq < row || a->ldo < row || a->ld_table < a->width)
        return refuse(GGUF_ERR_INVALID_ARG, "%s: a row stride is shorter than the row", what);
    if (!(a->scale > 0.0f) || a->scale > 3e38f) return refuse(GGUF_ERR_INVALID_ARG, "%s: scale must be positive and finite", what);
    return GGUF_OK;
}
static gguf_status check_attn_arrays(const gguf_attn_args *a, const void *ws, size_t ws_bytes, size_t need, const char *what) {
    const int64_t es = float_size(a->qt);
    if (!a->q || !a->out || (a->n_pages > 0 && !a->cache) || (a->width > 0 && !a->block_table))
        return refuse(GGUF_ERR_INVALID_ARG, "%s: null pointer", what);
    if (!at(a->q, es) || !at(a->out, es) || !at(a->cache, 16) || !at(a->block_table, 4) || !at(a->dev_status, 4))
        return refuse(GGUF_ERR_ALIGNMENT, "%s: cache must be 16-byte aligned, the arrays by their elements", what);
    if (ws_bytes < need || (need > 0 && !ws))
        return refuse(GGUF_ERR_WORKSPACE, "%s: workspace of %zu bytes < required %zu", what, ws_bytes, need);
    if (need > 0 && !at(ws, 16)) return refuse(GGUF_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", what);
    return GGUF_OK;
}

size_t gguf_paged_attention_ws_size(const gguf_attn_args *a) {
    if (check_attn_sizes(a, "paged_attention") != GGUF_OK || a->n_tokens == 0 || a->n_requests == 0) return 0;
    return attn_ws_size(attn_of(a), a->head_dim);
}

gguf_status gguf_paged_attention(const gguf_attn_args *a, void *ws, size_t ws_bytes, gguf_stream_t stream) {
    gguf_status st = check_attn_sizes(a, "paged_attention");
    if (st == GGUF_OK) st = check_attn_rows(a, "paged_attention");
    if (st != GGUF_OK) return st;
    if (a->n_tokens == 0 || a->n_requests == 0) return GGUF_OK;
    // fp32 queries walk over the tokens in groups of 8 rows: a request's groups x heads x tiles of 16 tokens are counted
    // in 32 bits
    if (a->qt == GGUF_F32) {
        const double tiles = (double)a->width * (double)a->page_size / KV_TILE;
        const double groups = (double)std::min<int64_t>(a->max_q_len, a->n_tokens) * (double)(a->n_heads / a->n_kv_heads) / 8.0 + 1.0;
        if (tiles * groups * (double)a->n_kv_heads > 4.0e9)
            return report(GGUF_ERR_SHAPE, "paged_attention: too many fp32 queries over too wide a table for one call; split it");
    }
    if (!a->q_start || !a->kv_len) return report(GGUF_ERR_INVALID_ARG, "paged_attention: null pointer");
    if (!at(a->q_start, 4) || !at(a->kv_len, 4)) return report(GGUF_ERR_ALIGNMENT, "paged_attention: misaligned q_start or kv_len");
    const Attn p = attn_of(a);
    st = check_attn_arrays(a, ws, ws_bytes, attn_ws_size(p, a->head_dim), "paged_attention");
    if (st != GGUF_OK) return st;
    return launched(launch_attn(p, a->head_dim, ws, (cudaStream_t)stream), "paged_attention");
}

// requests, groups and tokens of a plan, and the step that they belong to
static gguf_status check_plan_sizes(int64_t n_requests, int64_t n_groups, int64_t n_tokens, const char *what) {
    if (n_requests < 0 || n_groups < 0 || n_tokens < 0) return refuse(GGUF_ERR_INVALID_ARG, "%s: negative size", what);
    if (n_requests > 16384 || n_groups > 16384)
        return refuse(GGUF_ERR_SHAPE, "%s: %lld requests in %lld groups (at most 16384)", what, (long long)n_requests, (long long)n_groups);
    if (n_tokens > 0x7fffffff) return refuse(GGUF_ERR_SHAPE, "%s: n_tokens must fit in 31 bits", what);
    return GGUF_OK;
}

int64_t gguf_prefix_plan_bytes(int64_t n_requests, int64_t n_groups, int64_t n_tokens) {
    if (check_plan_sizes(n_requests, n_groups, n_tokens, "prefix_plan_bytes") != GGUF_OK) return -1;
    return prefix_plan_bytes(n_requests, n_groups, n_tokens);
}

gguf_status gguf_prefix_plan(const int32_t *q_start, const int32_t *kv_len, int64_t n_requests, const int32_t *group_start,
                             const int32_t *prefix_len, int64_t n_groups, int64_t page_size, int64_t n_tokens, void *plan,
                             size_t plan_bytes, gguf_stream_t stream) {
    const gguf_status st = check_plan_sizes(n_requests, n_groups, n_tokens, "prefix_plan");
    if (st != GGUF_OK) return st;
    if (page_size < KV_TILE || page_size % KV_TILE || page_size > (1 << 20))
        return refuse(GGUF_ERR_SHAPE, "prefix_plan: page_size=%lld is not a multiple of 16 up to 2^20", (long long)page_size);
    if (!plan || !q_start || (n_requests > 0 && !kv_len) || (n_groups > 0 && (!group_start || !prefix_len)))
        return report(GGUF_ERR_INVALID_ARG, "prefix_plan: null pointer");
    if (!at(q_start, 4) || !at(kv_len, 4) || !at(group_start, 4) || !at(prefix_len, 4) || !at(plan, 16))
        return report(GGUF_ERR_ALIGNMENT, "prefix_plan: the plan must be 16-byte aligned, the arrays by their elements");
    const int64_t need = prefix_plan_bytes(n_requests, n_groups, n_tokens);
    if (plan_bytes < (size_t)need)
        return refuse(GGUF_ERR_WORKSPACE, "prefix_plan: plan of %zu bytes < required %lld", plan_bytes, (long long)need);
    return launched(launch_prefix_plan(q_start, kv_len, n_requests, group_start, prefix_len, n_groups, page_size, n_tokens, plan,
                                       (cudaStream_t)stream), "prefix_plan");
}

static gguf_status check_prefix_sizes(const gguf_attn_args *a, int64_t n_groups) {
    gguf_status st = check_attn_sizes(a, "prefix_attention");
    if (st == GGUF_OK) st = check_plan_sizes(a->n_requests, n_groups, a->n_tokens, "prefix_attention");
    if (st != GGUF_OK) return st;
    // the tiles of all units are shared out over SMs and warps, whose parts are counted in 31 bits
    const double units = (double)a->n_tokens * (double)(a->n_heads / a->n_kv_heads) / 8.0 + (double)(a->n_requests + n_groups);
    if (units * (double)a->n_kv_heads * ((double)a->width * (double)(a->page_size / KV_TILE) + (double)PF_PAST) > 0x1p40)
        return report(GGUF_ERR_SHAPE, "prefix_attention: too many queries over too wide a table for one call; split it");
    if (a->n_tokens * a->n_heads > (1 << 30))   // records are counted in 31 bits, two a query row
        return refuse(GGUF_ERR_SHAPE, "prefix_attention: %lld tokens x %lld heads (at most 2^30)", (long long)a->n_tokens, (long long)a->n_heads);
    return GGUF_OK;
}

size_t gguf_prefix_attention_ws_size(const gguf_attn_args *a, int64_t n_groups) {
    if (check_prefix_sizes(a, n_groups) != GGUF_OK || a->n_tokens == 0 || a->n_requests == 0) return 0;
    return prefix_attn_ws_size(attn_of(a), n_groups, a->head_dim);
}

gguf_status gguf_prefix_attention(const gguf_attn_args *a, const void *plan, size_t plan_bytes, int64_t n_groups, void *ws,
                                  size_t ws_bytes, gguf_stream_t stream) {
    gguf_status st = check_prefix_sizes(a, n_groups);
    if (st == GGUF_OK) st = check_attn_rows(a, "prefix_attention");
    if (st != GGUF_OK) return st;
    if (a->n_tokens == 0 || a->n_requests == 0) return GGUF_OK;
    if (!plan) return report(GGUF_ERR_INVALID_ARG, "prefix_attention: null pointer");
    if (!at(plan, 16)) return report(GGUF_ERR_ALIGNMENT, "prefix_attention: the plan must be 16-byte aligned");
    const int64_t planned = prefix_plan_bytes(a->n_requests, n_groups, a->n_tokens);
    if (plan_bytes < (size_t)planned)
        return refuse(GGUF_ERR_WORKSPACE, "prefix_attention: plan of %zu bytes < required %lld", plan_bytes, (long long)planned);
    const Attn p = attn_of(a);
    st = check_attn_arrays(a, ws, ws_bytes, prefix_attn_ws_size(p, n_groups, a->head_dim), "prefix_attention");
    if (st != GGUF_OK) return st;
    return launched(launch_prefix_attn(p, plan, n_groups, a->head_dim, ws, (cudaStream_t)stream), "prefix_attention");
}

}  // extern "C"
