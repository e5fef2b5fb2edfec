// C ABI of gguf_block_norm: argument checks, then the launcher.
#include "abi_checks.h"
#include "common.cuh"

using namespace gg;

extern "C" {

gguf_status gguf_block_norm(const gguf_block_norm_args *a, gguf_stream_t stream) {
    if (!a) return report(GGUF_ERR_INVALID_ARG, "block_norm: null args");
    const bool has_x = a->x != nullptr, has_h = a->h != nullptr, gated = has_x && a->gate != nullptr;
    if (!float_type(a->xt) || !float_type(a->ht) || (a->ht != a->xt && a->ht != GGUF_F32))
        return refuse(GGUF_ERR_UNSUPPORTED_TYPE, "block_norm: types %d (x) and %d (h): F32/BF16/F16, h as x or F32", a->xt, a->ht);
    if ((a->z && !float_type(a->zt)) || (gated && a->gt != a->xt && a->gt != GGUF_F32))
        return refuse(GGUF_ERR_UNSUPPORTED_TYPE, "block_norm: types %d (z: F32/BF16/F16) and %d (gate: as x or F32)", a->zt, a->gt);
    if (a->n_tokens < 0 || a->k < 0) return report(GGUF_ERR_INVALID_ARG, "block_norm: negative size");
    if (a->n_tokens > 0x7fffffff || a->k < 1 || a->k > 32768)
        return refuse(GGUF_ERR_SHAPE, "block_norm: %lld tokens of %lld values (at most 2^31 - 1 of 1..32768)", (long long)a->n_tokens,
                      (long long)a->k);
    if (a->z_q8_1 && a->k % QK8) return refuse(GGUF_ERR_SHAPE, "block_norm: q8_1 rows need k=%lld to be a multiple of 32", (long long)a->k);
    auto kind = [](int n) { return n == GGUF_NORM_NONE || n == GGUF_NORM_RMS || n == GGUF_NORM_LAYER; };
    if (!kind(a->post_kind) || !kind(a->pre_kind)) return refuse(GGUF_ERR_INVALID_ARG, "block_norm: norm kinds %d, %d", a->post_kind, a->pre_kind);
    if (gated && (a->gate_act < GGUF_GATE_NONE || a->gate_act > GGUF_GATE_SILU))
        return refuse(GGUF_ERR_INVALID_ARG, "block_norm: gate_act %d", a->gate_act);
    if (!has_x && (a->gate || a->post_kind != GGUF_NORM_NONE)) return report(GGUF_ERR_INVALID_ARG, "block_norm: a gate or a norm of x without x");
    if (!(a->post_eps >= 0.0f) || !(a->pre_eps >= 0.0f)) return report(GGUF_ERR_INVALID_ARG, "block_norm: eps must not be negative");
    if ((has_x && a->ldx < a->k) || (has_h && a->ldh < a->k) || (gated && a->ldg != 0 && a->ldg < a->k) ||
        (a->h_out && a->ldho < a->k) || (a->z && a->ldz < a->k))
        return report(GGUF_ERR_INVALID_ARG, "block_norm: a row stride is shorter than the row");
    if (a->n_tokens == 0) return GGUF_OK;
    if ((!has_x && !has_h) || (!a->h_out && !a->z && !a->z_q8_1))
        return report(GGUF_ERR_INVALID_ARG, "block_norm: nothing to read, or nothing to write");
    const int64_t es = float_size(a->xt), eh = float_size(a->ht), eg = float_size(a->gt), ez = float_size(a->zt);
    if (!at(a->x, es) || !at(a->h, eh) || !at(a->h_out, eh) || (gated && !at(a->gate, eg)) || !at(a->z, a->z ? ez : 1) ||
        !at(a->z_q8_1, 4) || !at(a->post_w, 4) || !at(a->post_b, 4) || !at(a->pre_w, 4) || !at(a->pre_b, 4))
        return report(GGUF_ERR_ALIGNMENT, "block_norm: misaligned array");
    const BlockNorm p{a->x, a->h, gated ? a->gate : nullptr, a->ldx, a->ldh, a->ldg, a->gt, a->gate_act, a->n_tokens, a->k,
                      a->post_kind, a->pre_kind, a->post_w, a->post_b, a->pre_w, a->pre_b, a->post_eps, a->pre_eps, a->branch_scale,
                      a->residual_scale, a->h_out, a->ldho, a->z, a->zt, a->ldz, (uint8_t *)a->z_q8_1};
    const bool vec = rows16(a->x, a->ldx, es) && rows16(a->h, a->ldh, eh) && rows16(gated ? a->gate : nullptr, a->ldg, eg) &&
                     rows16(a->h_out, a->ldho, eh) && rows16(a->z, a->ldz, ez) && at(a->post_w, 16) && at(a->post_b, 16) &&
                     at(a->pre_w, 16) && at(a->pre_b, 16);
    return launched(launch_block_norm(p, a->xt, a->ht, vec, (cudaStream_t)stream), "block_norm");
}

}  // extern "C"
