// gguf_qk_norm_rope and gguf_kv_get_rows: what happens to a token's query, key
// and value rows between their products and the attention.
//
//   y = x / sqrt(mean(x^2) + eps) * w             (queries and keys, per head)
//   (a, b) -> (a cos - b sin, b cos + a sin)      (pairs of the first rot values)
//   queries to q_out; keys (and values, untouched) to Q4_0 in their cache slot:
//   d = fp16(the value of largest magnitude / -8), code = clamp(roundf(x / d) + 8, 0, 15).
//
// One pass: a group of D / 8 lanes holds a row, 8 values a lane, so the sum of
// squares and a block's extreme are a few shuffles, a rotation partner is in
// the lane itself or one shuffle away, and a lane's 8 key values are exactly
// one word of the packed tile.  A group walks over several rows of one token
// and keeps the token's cosines and sines in registers.  Products and sums of
// the rotation and of the code are rounded one by one (no fused multiply-add),
// so that the stored codes are those of the formula evaluated step by step.
//
// Bound: HBM for prompts (reads q, k, v; writes q and 4.5 bits per k and v
// value), latency for single tokens.
#include "common.cuh"
#include "internal.h"
#include "kv.cuh"

namespace gg {

constexpr int QR_THREADS = 256;

// 8 values at element offset `off` of x, 16-byte aligned (VEC) or element-aligned
template <int T, bool VEC>
__device__ __forceinline__ void ld8(const void *x, int64_t off, float (&v)[8]) {
    if constexpr (T == GGUF_F32) {
        const float *p = reinterpret_cast<const float *>(x) + off;
        if constexpr (VEC) {
            const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = p[i];
        }
    } else {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(x) + off;
        if constexpr (VEC) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[2 * i] = from16<T>(w[i] & 0xffff);
                v[2 * i + 1] = from16<T>(w[i] >> 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = from16<T>(p[i]);
        }
    }
}

template <int T>
__device__ __forceinline__ uint32_t to16(float f) { return T == GGUF_BF16 ? f2bf_rn(f) : f2h_rn(f); }

template <int T, bool VEC>
__device__ __forceinline__ void st8(void *x, int64_t off, const float (&v)[8]) {
    if constexpr (T == GGUF_F32) {
        float *p = reinterpret_cast<float *>(x) + off;
        if constexpr (VEC) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) p[i] = v[i];
        }
    } else {
        uint16_t *p = reinterpret_cast<uint16_t *>(x) + off;
        if constexpr (VEC) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; i++) w[i] = to16<T>(v[2 * i]) | (to16<T>(v[2 * i + 1]) << 16);
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) p[i] = (uint16_t)to16<T>(v[i]);
        }
    }
}

// codes of the lane's 8 values of a 32-value block (4 neighbouring lanes) and
// the block's fp16 scale; a block whose scale rounds to 0 stands for zeros
__device__ __forceinline__ uint16_t q4_block(const float (&v)[8], int lane, uint32_t mask, uint32_t (&code)[8]) {
    float big = v[0];
#pragma unroll
    for (int i = 1; i < 8; i++)
        if (fabsf(v[i]) > fabsf(big)) big = v[i];
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {   // of equal magnitudes, the value of the lowest index
        const float other = __shfl_xor_sync(mask, big, o);
        const float a = fabsf(other), b = fabsf(big);
        if (a > b || (a == b && (lane & o))) big = other;
    }
    const uint16_t dh = f2h_rn(__fmul_rn(big, -0.125f));
    const float d = h2f(dh);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int c = d != 0.0f ? (int)roundf(__fdiv_rn(v[i], d)) : 0;
        code[i] = (uint32_t)min(max(c + 8, 0), 15);
    }
    return dh;
}

template <int D, int T, bool VEC>
__global__ void __launch_bounds__(QR_THREADS) qk_norm_rope_kernel(const QkRope p, int groups) {
    constexpr int LPR = D / 8;   // lanes per row
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int l = lane % LPR;
    const uint32_t mask = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1) << (lane - l);
    const int64_t gid = ((int64_t)blockIdx.x * QR_THREADS + threadIdx.x) / LPR;
    const int64_t t = gid / groups;
    const int g0 = (int)(gid - t * groups);
    if (t >= p.n_tokens) return;   // whole groups of lanes
    const int64_t pos = p.pos[t];
    const int rot = p.rot, half = rot / 2;
    if (pos < 0 || pos >= p.n_pos) {   // a padding token (-1), or one past the table
        if (pos >= p.n_pos && p.status != nullptr && g0 == 0 && l == 0) atomicAdd(p.status, 1);
        return;
    }
    const bool turns = 8 * l < rot;
    // cosines and sines of the lane's values: 4 pairs inside the lane, or 8
    // values whose partners are half / 8 lanes away
    float cs[8], sn[8];
    if (turns) {
        const float *row = p.cos_sin + pos * rot;
        if (p.neox) {
            const int i = 8 * l < half ? 8 * l : 8 * l - half;
            ld8<GGUF_F32, true>(row, i, cs);
            ld8<GGUF_F32, true>(row, half + i, sn);
        } else {
            const float4 c = *reinterpret_cast<const float4 *>(row + 4 * l);
            const float4 s = *reinterpret_cast<const float4 *>(row + half + 4 * l);
            cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
            sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
        }
    }
    const int64_t slot = p.slots != nullptr ? p.slots[t] : -1;
    uint8_t *tile0 = nullptr;
    int tok = 0;
    if (p.cache != nullptr && slot >= 0) {
        const int64_t pg = slot / p.page;
        const int off = (int)(slot - pg * p.page);
        if (pg < p.n_pages) {
            tok = off % KV_TILE;
            tile0 = p.cache + pg * kv_page_bytes(D, p.hk, p.page) + off / KV_TILE * kv_tile_bytes(D);
        } else if (p.status != nullptr && g0 == 0 && l == 0) atomicAdd(p.status, 1);
    }
    const int64_t head_step = p.page / KV_TILE * kv_tile_bytes(D);
    const int rows = (int)p.rows;
    for (int r = g0; r < rows; r += groups) {
        const bool is_q = r < p.h, is_k = !is_q && r < p.h + p.hk;
        const int head = is_q ? r : is_k ? r - (int)p.h : r - (int)(p.h + p.hk);
        float v[8];
        ld8<T, VEC>(is_q ? p.q : is_k ? p.k : p.v, t * (is_q ? p.ldq : is_k ? p.ldk : p.ldv) + (int64_t)head * D + 8 * l, v);
        if (is_q || is_k) {
            const float *w = is_q ? p.qw : p.kw;
            if (w != nullptr) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; i++) ss = __fmaf_rn(v[i], v[i], ss);
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(mask, ss, o);
                const float inv = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.0f / D), p.eps));
                float wv[8];
                ld8<GGUF_F32, true>(w, 8 * l, wv);
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = __fmul_rn(__fmul_rn(v[i], inv), wv[i]);
            }
            if (p.neox) {
                const int hl = half / 8;
                const bool low = 8 * l < half;
                const int src = (lane - l) + (turns ? (low ? l + hl : l - hl) : l);
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; i++) o[i] = __shfl_sync(mask, v[i], src);
                if (turns) {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float a = __fmul_rn(v[i], cs[i]), b = __fmul_rn(o[i], sn[i]);
                        v[i] = low ? __fsub_rn(a, b) : __fadd_rn(a, b);
                    }
                }
            } else if (turns) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float a = v[2 * i], b = v[2 * i + 1];
                    v[2 * i] = __fsub_rn(__fmul_rn(a, cs[i]), __fmul_rn(b, sn[i]));
                    v[2 * i + 1] = __fadd_rn(__fmul_rn(b, cs[i]), __fmul_rn(a, sn[i]));
                }
            }
            if (is_q) {
                st8<T, VEC>(p.q_out, t * p.ldqo + (int64_t)head * D + 8 * l, v);
                continue;
            }
            if (p.k_out != nullptr) st8<T, VEC>(p.k_out, t * p.ldko + (int64_t)head * D + 8 * l, v);
        }
        if (tile0 == nullptr) continue;
        uint32_t code[8];
        const uint16_t d = q4_block(v, lane, mask, code);
        uint8_t *tile = tile0 + head * head_step;
        const int b = l / 4;
        if (is_k) {
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) w |= code[i] << (4 * (i >> 1) + 16 * (i & 1));
            *reinterpret_cast<uint32_t *>(tile + KvTile<D>::k_word(tok, b, l % 4)) = w;
            if (l % 4 == 0) *reinterpret_cast<uint16_t *>(tile + KvTile<D>::KS + KvTile<D>::scale(tok, b)) = d;
        } else {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 4; i++) w |= code[4 * j + i] << (4 * i);
                *reinterpret_cast<uint16_t *>(tile + KvTile<D>::v_half(tok, b, 2 * (l % 4) + j)) = (uint16_t)w;
            }
            if (l % 4 == 0) *reinterpret_cast<uint16_t *>(tile + KvTile<D>::VS + KvTile<D>::scale(tok, b)) = d;
        }
    }
}

template <int D, int T, bool VEC>
__global__ void __launch_bounds__(QR_THREADS) kv_get_rows_kernel(const KvRows p) {
    constexpr int LPR = D / 8;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t gid = ((int64_t)blockIdx.x * QR_THREADS + threadIdx.x) / LPR;
    const int l = threadIdx.x % LPR;
    const int64_t i = gid / (2 * p.hk);
    if (i >= p.n) return;
    const int r = (int)(gid - i * 2 * p.hk);
    const bool is_k = r < p.hk;
    const int head = is_k ? r : r - (int)p.hk;
    const int64_t slot = p.slots[i];
    const int64_t pg = slot < 0 ? -1 : slot / p.page;
    float v[8];
    if (pg < 0 || pg >= p.n_pages) {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = 0.0f;
    } else {
        const int off = (int)(slot - pg * p.page), tok = off % KV_TILE, b = l / 4;
        const uint8_t *tile = p.cache + pg * kv_page_bytes(D, p.hk, p.page) +
                              (head * (p.page / KV_TILE) + off / KV_TILE) * kv_tile_bytes(D);
        const float d = h2f(ld_u16(tile + (is_k ? KvTile<D>::KS : KvTile<D>::VS) + KvTile<D>::scale(tok, b)));
        if (is_k) {
            const uint32_t w = ld_u32(tile + KvTile<D>::k_word(tok, b, l % 4));
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = d * (float)((int)((w >> (4 * (j >> 1) + 16 * (j & 1))) & 15) - 8);
        } else {
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const uint32_t w = ld_u16(tile + KvTile<D>::v_half(tok, b, 2 * (l % 4) + x));
#pragma unroll
                for (int j = 0; j < 4; j++) v[4 * x + j] = d * (float)((int)((w >> (4 * j)) & 15) - 8);
            }
        }
    }
    st8<T, VEC>(is_k ? p.k : p.v, (i * p.hk + head) * D + 8 * l, v);
}

static cudaError_t launch_pdl(const void *kern, int64_t grid, cudaStream_t s, void **args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(QR_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

template <int D>
static const void *rope_kernel(int t, bool vec) {
    if (t == GGUF_F32) return vec ? (const void *)qk_norm_rope_kernel<D, GGUF_F32, true> : (const void *)qk_norm_rope_kernel<D, GGUF_F32, false>;
    if (t == GGUF_F16) return vec ? (const void *)qk_norm_rope_kernel<D, GGUF_F16, true> : (const void *)qk_norm_rope_kernel<D, GGUF_F16, false>;
    return vec ? (const void *)qk_norm_rope_kernel<D, GGUF_BF16, true> : (const void *)qk_norm_rope_kernel<D, GGUF_BF16, false>;
}

cudaError_t launch_qk_norm_rope(const QkRope &p, int64_t d, int xt, bool vec, cudaStream_t s) {
    const int64_t rows = p.rows;
    // a token's rows are shared out over as many groups as fill the GPU (1024
    // threads per SM), at least one and at most a row each
    const int64_t lpr = d / 8, full = (int64_t)device_info().sm_count * 1024 / lpr;
    int64_t groups = (full + p.n_tokens - 1) / p.n_tokens;
    groups = groups < 1 ? 1 : groups > rows ? rows : groups;
    const int64_t grid = (p.n_tokens * groups * lpr + QR_THREADS - 1) / QR_THREADS;
    const void *kern = d == 64 ? rope_kernel<64>(xt, vec) : d == 128 ? rope_kernel<128>(xt, vec) : rope_kernel<256>(xt, vec);
    QkRope a = p;
    int g = (int)groups;
    void *args[2] = {&a, &g};
    return launch_pdl(kern, grid, s, args);
}

template <int D>
static const void *rows_kernel(int t, bool vec) {
    if (t == GGUF_F32) return vec ? (const void *)kv_get_rows_kernel<D, GGUF_F32, true> : (const void *)kv_get_rows_kernel<D, GGUF_F32, false>;
    if (t == GGUF_F16) return vec ? (const void *)kv_get_rows_kernel<D, GGUF_F16, true> : (const void *)kv_get_rows_kernel<D, GGUF_F16, false>;
    return vec ? (const void *)kv_get_rows_kernel<D, GGUF_BF16, true> : (const void *)kv_get_rows_kernel<D, GGUF_BF16, false>;
}

cudaError_t launch_kv_get_rows(const KvRows &p, int64_t d, int ot, bool vec, cudaStream_t s) {
    const int64_t grid = (p.n * 2 * p.hk * (d / 8) + QR_THREADS - 1) / QR_THREADS;
    const void *kern = d == 64 ? rows_kernel<64>(ot, vec) : d == 128 ? rows_kernel<128>(ot, vec) : rows_kernel<256>(ot, vec);
    KvRows a = p;
    void *args[1] = {&a};
    return launch_pdl(kern, grid, s, args);
}

}  // namespace gg
