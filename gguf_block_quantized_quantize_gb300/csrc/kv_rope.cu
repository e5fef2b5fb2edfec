// gguf_qk_norm_rope, gguf_qk_norm_mrope and gguf_kv_get_rows: what happens to a token's query, key
// and value rows between their products and the attention.
//
//   y = x / sqrt(mean(x^2) + eps) * w             (queries and keys, per head)
//   (a, b) -> (a cos - b sin, b cos + a sin)      (pairs of the first rot values)
//                                                 (at pos, or each pair at the position of its axis)
//   queries to q_out; keys (and values, untouched) to Q4_0 in their cache slot:
//   d = fp16(the value of largest magnitude / -8), code = clamp(roundf(x / d) + 8, 0, 15).
//
// One pass.  Queries and keys: a group of D / 8 lanes holds a row, 8 values a
// lane, so the sum of squares and a block's extreme are a few shuffles, a
// rotation partner is in the lane itself or one shuffle away, and a lane's 8 key
// values are exactly one word of the packed tile.  A group takes a few rows of
// one token, queries or keys, two of them loaded ahead (one of fp32), and keeps the
// token's cosines and sines in registers.  Values: a warp takes one 32-value block of 8 tokens, so that the
// 16 bits that a tile keeps together of 4 values of one token lie next to those
// of the other tokens.  Products and sums of the rotation are rounded one by one
// (no fused multiply-add).  Codes are exactly those of the fp32 keys that k_out
// shows for fp32 inputs; the norm's sum of squares is taken lane by lane, so a key
// value on the border of two codes may take the neighbour of the code that another
// order of that sum gives.
//
// Bound: HBM for prompts (reads q, k, v; writes q and 4.5 bits per k and v
// value), latency for single tokens.  Measured in a captured graph, one axis and
// three: 1 token, 32 + 8 + 8 heads of 128, bf16 2.8 and 3.3 us; 2048 tokens 17.4 and
// 19.9 us (the bytes take 6.7), 4096 tokens 29.1 and 31.6 us, 2048 in fp32 21.5 and
// 24.6; 2048 tokens, 16 + 2 + 2 heads of 256, 12.3 and 14.3 us.  Between: the issue of
// some 31 instructions a value (59 % of the slots) at eight warps a scheduler, and the
// chain load, sum, rotate, round, store.  With queries and keys in one loop and four rows
// loaded ahead the registers spilled (284 bytes of loads a thread) and each four rows
// fetched their token's angles anew: 2048 tokens 20.4 and 23.3 us, 4096 38.3 and 43.9.
#include <algorithm>

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
// two values rounded to 16 bits, the first in the low half
template <int T>
__device__ __forceinline__ uint32_t pair16(float a, float b) {
    uint32_t w;
    if constexpr (T == GGUF_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}

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
            for (int i = 0; i < 4; i++) w[i] = pair16<T>(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) p[i] = (uint16_t)to16<T>(v[i]);
        }
    }
}

// codes of the lane's 8 values of a 32-value block (the lanes that differ in
// bits `step` and 2 `step`, later ones holding later values) and the block's
// fp16 scale; a block whose scale rounds to 0 stands for zeros
__device__ __forceinline__ uint16_t q4_block(const float (&v)[8], int lane, uint32_t mask, int step, uint32_t (&code)[8]) {
    float big = v[0];
#pragma unroll
    for (int i = 1; i < 8; i++)
        if (fabsf(v[i]) > fabsf(big)) big = v[i];
#pragma unroll
    for (int k = 0; k < 2; k++) {   // of equal magnitudes, the value of the lowest index
        const int o = step << k;
        const float other = __shfl_xor_sync(mask, big, o);
        const float a = fabsf(other), b = fabsf(big);
        if (a > b || (a == b && (lane & o))) big = other;
    }
    const uint16_t dh = f2h_rn(__fmul_rn(big, -0.125f));
    const float d = h2f(dh), inv = d != 0.0f ? __frcp_rn(d) : 0.0f;
    // roundf(x / d): x * (1 / d) is within 2^-22 of it relatively (|x / d| < 12.1, so within 2^-18), which decides
    // the rounding unless the quotient lies that near to a half: then the division itself does.  Adding 1.5 * 2^23 + 8
    // leaves the rounded quotient + 8 in the low bits.
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float q = fmaxf(__fmul_rn(v[i], inv), -8.0f), r = __fadd_rn(q, 12582920.0f);
        near |= fabsf(__fsub_rn(q, __fsub_rn(r, 12582920.0f))) > 0.5f - 0x1p-17f;
        code[i] = min(__float_as_uint(r) & 31u, 15u);
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int c = d != 0.0f ? (int)roundf(__fdiv_rn(v[i], d)) : 0;
            code[i] = (uint32_t)min(max(c + 8, 0), 15);
        }
    }
    return dh;
}

// rows of q, k or v of 8 values per lane, before they become floats
template <int T>
struct Raw8 {
    uint4 w[T == GGUF_F32 ? 2 : 1];
    template <bool VEC>
    __device__ __forceinline__ void load(const void *x, int64_t off) {
        if constexpr (VEC) {
            const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(x) + off * (T == GGUF_F32 ? 4 : 2));
            w[0] = p[0];
            if constexpr (T == GGUF_F32) w[1] = p[1];
        } else if constexpr (T == GGUF_F32) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(x) + off;
            w[0] = make_uint4(p[0], p[1], p[2], p[3]);
            w[1] = make_uint4(p[4], p[5], p[6], p[7]);
        } else {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(x) + off;
            w[0] = make_uint4(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16, p[4] | (uint32_t)p[5] << 16,
                              p[6] | (uint32_t)p[7] << 16);
        }
    }
    __device__ __forceinline__ void floats(float (&v)[8]) const {
        const uint32_t a[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (T == GGUF_F32) {
                v[i] = __uint_as_float(a[i]);
                v[4 + i] = __uint_as_float(i == 0 ? w[1].x : i == 1 ? w[1].y : i == 2 ? w[1].z : w[1].w);
            } else {
                v[2 * i] = from16<T>(a[i] & 0xffff);
                v[2 * i + 1] = from16<T>(a[i] >> 16);
            }
        }
    }
};

// the positions of a token on its axes; -1: left out (padding: negative on some axis, or past the table: then `past` is set)
template <int AXES>
__device__ __forceinline__ bool token_positions(const QkRope &p, int64_t t, int64_t (&pos)[AXES], bool &past) {
    bool there = true;
    past = false;
#pragma unroll
    for (int a = 0; a < AXES; a++) {
        pos[a] = a == 0 || a < p.n_axes ? p.pos[a * p.ldpos + t] : 0;
        there &= pos[a] >= 0;
        past |= pos[a] >= p.n_pos;
    }
    past &= there;
    return there && !past;
}
// N cosines and sines of pairs i .. of a token, a pair's from the row of its axis
template <int AXES, int N>
__device__ __forceinline__ void angles(const QkRope &p, const int64_t (&pos)[AXES], int i, float (&cs)[8], float (&sn)[8]) {
    const int half = p.rot / 2;
    const uint32_t of = AXES == 1 ? 0 : (uint32_t)p.axis_of[i >> 3] >> (2 * (i & 7));   // 2 bits a pair
#pragma unroll
    for (int a = 0; a < AXES; a++) {
        uint32_t mine = 0;   // the pairs on this axis
#pragma unroll
        for (int x = 0; x < N; x++) mine |= ((of >> (2 * x)) & 3) == a ? 1u << x : 0u;
        if (AXES > 1 && mine == 0) continue;
        const float *row = p.cos_sin + pos[a] * p.rot + i;
        float c[N], s[N];
#pragma unroll
        for (int x = 0; x < N; x += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(row + x), v = *reinterpret_cast<const float4 *>(row + half + x);
            c[x] = u.x; c[x + 1] = u.y; c[x + 2] = u.z; c[x + 3] = u.w;
            s[x] = v.x; s[x + 1] = v.y; s[x + 2] = v.z; s[x + 3] = v.w;
        }
#pragma unroll
        for (int x = 0; x < N; x++)
            if (AXES == 1 || (mine >> x) & 1) { cs[x] = c[x]; sn[x] = s[x]; }
    }
}

// the tile (of KV head 0) and the token in it of a slot; null: nothing to store
template <int D>
__device__ __forceinline__ uint8_t *slot_tile(const QkRope &p, int64_t slot, int &tok) {
    tok = 0;
    if (slot < 0) return nullptr;
    const int64_t pg = (uint64_t)slot >> 32 ? slot / p.page : (int64_t)((uint32_t)slot / (uint32_t)p.page);
    if (pg >= p.n_pages) return nullptr;
    const int off = (int)(slot - pg * p.page);
    tok = off % KV_TILE;
    return p.cache + pg * kv_page_bytes(D, p.hk, p.page) + off / KV_TILE * kv_tile_bytes(D);
}

template <int T> constexpr int QR_ROWS = T == GGUF_F32 ? 1 : 2;   // rows that a group loads together

// Blocks [0, q_end): groups of D / 8 lanes, q_groups per token, over the rows of q; up to k_end: k_groups per token over the
// rows of k; the blocks after them: a warp per 8 tokens and 32-value block of v.
struct RopeCut {
    int q_groups, k_groups, q_end, k_end;
};

// a group's rows of one token: g0, g0 + groups, .. of the queries, or of the keys
template <int D, int T, bool VEC, int AXES, bool KEYS>
__device__ __forceinline__ void rope_rows(const QkRope &p, int64_t gid, int groups) {
    constexpr int LPR = D / 8, ES = T == GGUF_F32 ? 4 : 2;   // lanes per row
    const int lane = threadIdx.x & 31, l = lane % LPR;
    const uint32_t mask = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1) << (lane - l);
    const int64_t t = (uint64_t)gid >> 32 ? gid / groups : (int64_t)((uint32_t)gid / (uint32_t)groups);
    const int g0 = (int)(gid - t * groups);
    if (t >= p.n_tokens) return;   // whole groups of lanes
    const int rot = p.rot, half = rot / 2, rows = (int)(KEYS ? p.hk : p.h);
    const uint8_t *from = reinterpret_cast<const uint8_t *>(KEYS ? p.k : p.q) + (t * (KEYS ? p.ldk : p.ldq) + 8 * l) * ES;
    Raw8<T> raw[QR_ROWS<T>];
#pragma unroll
    for (int i = 0; i < QR_ROWS<T>; i++) {
        const int r = g0 + i * groups;
        if (r < rows) raw[i].template load<VEC>(from + r * (D * ES), 0);
    }
    int64_t pos[AXES];
    bool past;
    const bool there = token_positions<AXES>(p, t, pos, past);
    // (counted by the queries' first group, or the keys' where there are no queries)
    const bool counts = g0 == 0 && l == 0 && p.status != nullptr && (!KEYS || p.h == 0);
    if (!there) {   // a padding token (-1), or one past the table
        if (past && counts) atomicAdd(p.status, 1);
        return;
    }
    const bool turns = 8 * l < rot, low = 8 * l < half;
    // cosines and sines of the lane's values: 4 pairs inside the lane, or 8
    // values whose partners are half / 8 lanes away
    float cs[8], sn[8];
    if (turns) {
        if (p.neox) {
            angles<AXES, 8>(p, pos, low ? 8 * l : 8 * l - half, cs, sn);
#pragma unroll
            for (int x = 0; x < 8; x++) sn[x] = low ? -sn[x] : sn[x];
        } else {
            angles<AXES, 4>(p, pos, 4 * l, cs, sn);
        }
    }
    const float *w = KEYS ? p.kw : p.qw;
    float wv[8];
    if (w != nullptr) ld8<GGUF_F32, true>(w, 8 * l, wv);
    const int hl = half / 8, src = (lane - l) + (turns ? (low ? l + hl : l - hl) : l);
    uint8_t *tile = nullptr, *to = nullptr;
    int64_t head_step = 0;
    if constexpr (KEYS) {
        int tok = 0;
        const int64_t slot = p.cache != nullptr ? p.slots[t] : -1;
        tile = slot >= 0 ? slot_tile<D>(p, slot, tok) : nullptr;
        if (slot >= 0 && tile == nullptr && g0 == 0 && l == 0 && p.status != nullptr) atomicAdd(p.status, 1);
        head_step = p.page / KV_TILE * kv_tile_bytes(D);
        if (tile != nullptr) tile += KvTile<D>::k_word(tok, l / 4, l % 4);   // the lane's word of head 0
        if (tile != nullptr && l % 4 == 0) to = tile - KvTile<D>::k_word(tok, l / 4, 0) + KvTile<D>::KS + KvTile<D>::scale(tok, l / 4);
    } else {
        to = reinterpret_cast<uint8_t *>(p.q_out) + (t * p.ldqo + 8 * l) * ES;
    }
    for (int r0 = g0; r0 < rows; r0 += QR_ROWS<T> * groups) {
#pragma unroll
        for (int i = 0; i < QR_ROWS<T>; i++) {
            const int r = r0 + i * groups;
            if (r >= rows) break;
            float v[8];
            raw[i].floats(v);
            if (w != nullptr) {
                float ss = 0.0f;
#pragma unroll
                for (int x = 0; x < 8; x++) ss = __fmaf_rn(v[x], v[x], ss);
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(mask, ss, o);
                const float inv = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.0f / D), p.eps));
#pragma unroll
                for (int x = 0; x < 8; x++) v[x] = __fmul_rn(__fmul_rn(v[x], inv), wv[x]);
            }
            if (p.neox) {
                float o[8];
#pragma unroll
                for (int x = 0; x < 8; x++) o[x] = __shfl_sync(mask, v[x], src);
                if (turns) {   // the low values' sines are negative here
#pragma unroll
                    for (int x = 0; x < 8; x++) v[x] = __fadd_rn(__fmul_rn(v[x], cs[x]), __fmul_rn(o[x], sn[x]));
                }
            } else if (turns) {
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    const float a = v[2 * x], b = v[2 * x + 1];
                    v[2 * x] = __fsub_rn(__fmul_rn(a, cs[x]), __fmul_rn(b, sn[x]));
                    v[2 * x + 1] = __fadd_rn(__fmul_rn(b, cs[x]), __fmul_rn(a, sn[x]));
                }
            }
            if constexpr (!KEYS) st8<T, VEC>(to + r * (D * ES), 0, v);
            else {
                if (p.k_out != nullptr) st8<T, VEC>(p.k_out, t * p.ldko + (int64_t)r * D + 8 * l, v);
                if (tile == nullptr) continue;
                uint32_t code[8];
                const uint16_t d = q4_block(v, lane, mask, 1, code);
                uint32_t word = 0;
#pragma unroll
                for (int x = 0; x < 8; x++) word |= code[x] << (4 * (x >> 1) + 16 * (x & 1));
                *reinterpret_cast<uint32_t *>(tile + r * head_step) = word;
                if (to != nullptr) *reinterpret_cast<uint16_t *>(to + r * head_step) = d;
            }
        }
#pragma unroll
        for (int i = 0; i < QR_ROWS<T>; i++) {   // the next rows
            const int r = r0 + (QR_ROWS<T> + i) * groups;
            if (r < rows) raw[i].template load<VEC>(from + r * (D * ES), 0);
        }
    }
}

template <int D, int T, bool VEC, int AXES>
__global__ void __launch_bounds__(QR_THREADS, 4) qk_norm_rope_kernel(const QkRope p, const RopeCut cut) {
    constexpr int LPR = D / 8, NB = D / 32;   // lanes per row, blocks per row
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    if ((int)blockIdx.x >= cut.k_end) {
        const int64_t w = ((int64_t)(blockIdx.x - cut.k_end) * QR_THREADS + threadIdx.x) >> 5;   // 8 tokens, head, block
        const int l4 = lane >> 3, b = (int)(w % NB);
        const int64_t hw = w / NB, t8 = (uint64_t)hw >> 32 ? hw / p.hk : (int64_t)((uint32_t)hw / (uint32_t)p.hk), t = t8 * 8 + (lane & 7);
        const int head = (int)(hw - t8 * p.hk);
        const bool in = t < p.n_tokens;
        Raw8<T> raw;
        float v[8] = {};
        int tok = 0;
        uint8_t *tile = nullptr;
        if (in) {
            raw.template load<VEC>(p.v, t * p.ldv + (int64_t)head * D + 32 * b + 8 * l4);
            const int64_t slot = p.slots[t];
            int64_t pos[AXES];
            bool past;
            raw.floats(v);
            if (token_positions<AXES>(p, t, pos, past)) tile = slot_tile<D>(p, slot, tok);
        }
        uint32_t code[8];
        const uint16_t d = q4_block(v, lane, 0xffffffffu, 8, code);
        if (tile == nullptr) return;
        tile += head * (p.page / KV_TILE * kv_tile_bytes(D));
#pragma unroll
        for (int j = 0; j < 2; j++)
            *reinterpret_cast<uint16_t *>(tile + KvTile<D>::v_half(tok, b, 2 * l4 + j)) =
                (uint16_t)(code[4 * j] | code[4 * j + 1] << 4 | code[4 * j + 2] << 8 | code[4 * j + 3] << 12);
        if (l4 == 0) *reinterpret_cast<uint16_t *>(tile + KvTile<D>::VS + KvTile<D>::scale(tok, b)) = d;
        return;
    }
    if ((int)blockIdx.x < cut.q_end)
        rope_rows<D, T, VEC, AXES, false>(p, ((int64_t)blockIdx.x * QR_THREADS + threadIdx.x) / LPR, cut.q_groups);
    else
        rope_rows<D, T, VEC, AXES, true>(p, ((int64_t)(blockIdx.x - cut.q_end) * QR_THREADS + threadIdx.x) / LPR, cut.k_groups);
}

// gguf_kv_get_rows: values d * (c - 8) of slots.  16 slots side by side in the lanes, so that the lanes share the sectors
// of a tile that holds them all (with a slot's head per group of lanes 18 us, so 5.4 us: 2048 slots, 8 bf16 heads of 128;
// the bytes take 1.6).
template <int D, int T, bool VEC>
__global__ void __launch_bounds__(QR_THREADS) kv_get_rows_kernel(const KvRows p) {
    constexpr int LPR = D / 8;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t id = (int64_t)blockIdx.x * QR_THREADS + threadIdx.x;
    const int l = (int)(id / 16 % LPR);
    const int64_t rest = id / (16 * LPR);
    const int r = (int)(rest % (2 * p.hk));
    const int64_t i = rest / (2 * p.hk) * 16 + id % 16;
    if (i >= p.n) return;
    const bool is_k = r < p.hk;
    const int head = is_k ? r : r - (int)p.hk;
    const int64_t slot = p.slots[i];
    const int64_t pg = slot < 0 ? -1 : (uint64_t)slot >> 32 ? slot / p.page : (int64_t)((uint32_t)slot / (uint32_t)p.page);
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
            const uint32_t w = ld_u16(tile + KvTile<D>::v_half(tok, b, 2 * (l % 4))) |
                               (uint32_t)ld_u16(tile + KvTile<D>::v_half(tok, b, 2 * (l % 4) + 1)) << 16;
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = d * (float)((int)((w >> (4 * j)) & 15) - 8);
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

template <int D, int AXES>
static const void *rope_kernel(int t, bool vec) {
    if (t == GGUF_F32) return vec ? (const void *)qk_norm_rope_kernel<D, GGUF_F32, true, AXES> : (const void *)qk_norm_rope_kernel<D, GGUF_F32, false, AXES>;
    if (t == GGUF_F16) return vec ? (const void *)qk_norm_rope_kernel<D, GGUF_F16, true, AXES> : (const void *)qk_norm_rope_kernel<D, GGUF_F16, false, AXES>;
    return vec ? (const void *)qk_norm_rope_kernel<D, GGUF_BF16, true, AXES> : (const void *)qk_norm_rope_kernel<D, GGUF_BF16, false, AXES>;
}
// one position a token, or up to four
template <int D>
static const void *rope_kernel(int t, bool vec, int axes) { return axes == 1 ? rope_kernel<D, 1>(t, vec) : rope_kernel<D, 4>(t, vec); }

cudaError_t launch_qk_norm_rope(const QkRope &p, int64_t d, int xt, bool vec, cudaStream_t s) {
    // A group per row for few tokens; once that fills the GPU (2048 threads per SM, 512 where a group is a whole warp: 2048
    // tokens, 16 + 2 heads of 256, 14.7 and 12.3 us; 32 + 8 of 128 17.3 and 19.5 us) up to eight rows per group, which share the
    // token's angles (4096 tokens, 32 + 8 heads of 128, on three axes: 36 us with four rows, 31.4 with eight).
    const int64_t lpr = d / 8, full = (int64_t)device_info().sm_count * (d == 256 ? 512 : 2048) / lpr, all = p.h + p.hk;
    auto groups_of = [&](int64_t rows) -> int64_t {
        if (rows == 0) return 0;
        const int64_t fill = (full * rows / all + p.n_tokens - 1) / p.n_tokens;   // its share of the threads
        return std::max<int64_t>(1, std::min(rows, std::max((rows + 7) / 8, fill)));
    };
    auto blocks = [&](int64_t groups) { return (p.n_tokens * groups * lpr + QR_THREADS - 1) / QR_THREADS; };
    const int64_t qg = groups_of(p.h), kg = groups_of(p.hk);
    const int64_t v_warps = p.cache != nullptr ? (p.n_tokens + 7) / 8 * p.hk * (d / 32) : 0;
    const int64_t q_end = blocks(qg), k_end = q_end + blocks(kg), grid = k_end + (v_warps * 32 + QR_THREADS - 1) / QR_THREADS;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    const void *kern = d == 64 ? rope_kernel<64>(xt, vec, p.n_axes) : d == 128 ? rope_kernel<128>(xt, vec, p.n_axes) : rope_kernel<256>(xt, vec, p.n_axes);
    QkRope a = p;
    RopeCut cut{(int)qg, (int)kg, (int)q_end, (int)k_end};
    void *args[2] = {&a, &cut};
    return launch_pdl(kern, grid, s, args);
}

template <int D>
static const void *rows_kernel(int t, bool vec) {
    if (t == GGUF_F32) return vec ? (const void *)kv_get_rows_kernel<D, GGUF_F32, true> : (const void *)kv_get_rows_kernel<D, GGUF_F32, false>;
    if (t == GGUF_F16) return vec ? (const void *)kv_get_rows_kernel<D, GGUF_F16, true> : (const void *)kv_get_rows_kernel<D, GGUF_F16, false>;
    return vec ? (const void *)kv_get_rows_kernel<D, GGUF_BF16, true> : (const void *)kv_get_rows_kernel<D, GGUF_BF16, false>;
}

cudaError_t launch_kv_get_rows(const KvRows &p, int64_t d, int ot, bool vec, cudaStream_t s) {
    const int64_t grid = ((p.n + 15) / 16 * 16 * 2 * p.hk * (d / 8) + QR_THREADS - 1) / QR_THREADS;
    const void *kern = d == 64 ? rows_kernel<64>(ot, vec) : d == 128 ? rows_kernel<128>(ot, vec) : rows_kernel<256>(ot, vec);
    KvRows a = p;
    void *args[1] = {&a};
    return launch_pdl(kern, grid, s, args);
}

}  // namespace gg
