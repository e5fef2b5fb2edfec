// Attention of few query rows over the paged Q4_0 cache (single tokens, and a
// few tokens at once): each cached byte is read once per group of RG query
// rows that share its KV head, so HBM is the bound: 36 bytes per 32 values of
// head size and token.
//
// Work: the tiles (16 tokens of one head) that the units (request, KV head,
// group of RG rows) see, in one sequence, unit by unit.  It is cut evenly over
// the CTAs and, within a CTA, over the warps, whatever the requests' lengths;
// the cut is made on the device, from the lengths, so a captured graph serves
// any lengths.  A warp keeps an online softmax of the unit it is in; pieces of
// a unit are joined in the CTA through shared memory and, where a unit runs
// over several CTAs, by a second small launch, always in the same order.
//
// A warp's tile: its 18 * D contiguous bytes come by one bulk copy into the
// warp's own ring of stages, several tiles ahead.  Scores and outputs are
// warp-level 16x8x16 matrix products with the codes as operands:
//   S = Q K^T  A = 16 query rows, B = 8 keys.  The 4-bit code c is put into the
//              mantissa of 16 (one shift, one and-or for two values), which is
//              the exact number 16 + c; the accumulator starts from -24 sum(q),
//              so it ends as sum q (c - 8) of one 32-value block, and the
//              block's scale is applied to it in fp32.
//   O^T = V^T P^T  A = 16 values of a head, B = 8 query rows; the accumulator of
//              S is the B operand of O^T as it stands.  v = d * (c - 8) is
//              rounded to fp16 (2^-12 of it at most) and p = 2^(s - max + 10)
//              likewise; sums and statistics are fp32.
// fp32 queries use three bf16 parts of q, and high and low fp16 parts of p and
// v, for fp32 accuracy.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "kv.cuh"
#include "tc.cuh"

namespace gg {

constexpr float AD_PBITS = 10.0f;   // probabilities are held times 2^10 (at most 1024): small ones keep their bits in fp16

template <int D, int QT, int NT>
struct AdCfg {
    static constexpr int RG = 8 * NT;                       // query rows of a unit
    static constexpr int WARPS = (D == 256 || NT == 2 || QT == GGUF_F32) ? 8 : 16;
    static constexpr int STAGES = NT == 2 ? 8 : 4;
    static constexpr int RING = STAGES * KvTile<D>::BYTES;  // bytes per warp, a multiple of 128
    static constexpr int SLOT = RG * (D + 2) * 4;           // one partial result: O, then max and sum per row
    static_assert(SLOT <= RING, "a warp's last partial result reuses its ring");
    static constexpr int SMEM = WARPS * (RING + SLOT);
};

// what the requests look like to the kernels of one call
struct AdShape {
    Attn p;
    int32_t min_rows, max_rows;   // requests with more than min_rows and at most max_rows query rows per KV head are taken
    int32_t vec;                  // rows of q and out start on 16 bytes
    float *part;                  // CTA-level partial results, two slots per CTA
    int32_t *meta;                // per CTA: units that continue past it (see attn_combine_kernel)
    int *err;                     // error word: a wait for a copy was given up
};

// one request: its queries and the tiles that they see together
struct AdReq {
    int32_t rows0;        // first query token
    int32_t q;            // query tokens
    int32_t pos0;         // position of the first
    int32_t nt, n_sink, w_tile;   // tiles: n_sink first ones, then from w_tile on
};
__device__ __forceinline__ AdReq ad_request(const AdShape &a, int r) {
    AdReq o;
    const Attn &p = a.p;
    const int G = (int)(p.h / p.hk);
    o.rows0 = p.q_start[r];
    const int64_t q = min((int64_t)p.q_start[r + 1] - o.rows0, p.max_q);
    const bool mine = o.rows0 >= 0 && q > 0 && q * G > a.min_rows && q * G <= a.max_rows && o.rows0 + q <= p.n_tokens;
    o.q = mine ? (int32_t)q : 0;
    o.nt = o.n_sink = o.w_tile = 0;
    const int32_t kv = p.kv_len[r];
    o.pos0 = kv - (p.q_start[r + 1] - o.rows0);
    const int32_t last = o.pos0 + o.q - 1;
    if (o.q > 0 && last >= 0) {
        const int32_t end = last / KV_TILE + 1;
        o.nt = end;
        if (p.window > 0) {
            const int64_t w0 = (int64_t)o.pos0 - p.window + 1;
            o.w_tile = w0 > 0 ? (int32_t)(w0 / KV_TILE) : 0;
            o.n_sink = (int32_t)min((p.sinks + KV_TILE - 1) / KV_TILE, (int64_t)o.w_tile);
            o.nt = o.n_sink + end - o.w_tile;
        }
    }
    return o;
}
__device__ __forceinline__ int64_t ad_tiles(const AdShape &a, const AdReq &q, int rg) {
    const int G = (int)(a.p.h / a.p.hk);
    return (int64_t)q.nt * ((q.q * G + rg - 1) / rg) * a.p.hk;
}

__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t o) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(m), "r"(o));   // (x & m) | o
    return r;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) { return h2u(__floats2half2_rn(lo, hi)); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 16 + code of nibble i of both halves of w, as two fp16 / bf16 numbers
template <int I>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
    constexpr int SH = 4 * I - 6;
    return and_or(SH < 0 ? w << (SH < 0 ? -SH : 0) : w >> (SH > 0 ? SH : 0), 0x03C003C0u, 0x4C004C00u);
}
template <int I>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
    constexpr int SH = 4 * I - 3;
    return and_or(SH < 0 ? w << (SH < 0 ? -SH : 0) : w >> (SH > 0 ? SH : 0), 0x00780078u, 0x41804180u);
}
// 1024 + code, one operation fewer for the lowest nibble
template <int I>
__device__ __forceinline__ __half2 codes_1024(uint32_t w) { return u2h(and_or(w >> (4 * I), 0x000F000Fu, 0x64006400u)); }

// N consecutive words of shared memory as vector loads
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; i++) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    } else {
        static_assert(N == 2, "2, 4 or 8 words");
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    }
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     tc::smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

// four consecutive outputs
template <int QT>
__device__ __forceinline__ void store4(void *out, int64_t i, bool vec, float a, float b, float c, float d) {
    if constexpr (QT == GGUF_F32) {
        float *o = reinterpret_cast<float *>(out) + i;
        if (vec) *reinterpret_cast<float4 *>(o) = make_float4(a, b, c, d);
        else { o[0] = a; o[1] = b; o[2] = c; o[3] = d; }
    } else {
        uint16_t *o = reinterpret_cast<uint16_t *>(out) + i;
        const uint16_t h[4] = {QT == GGUF_BF16 ? f2bf_rn(a) : f2h_rn(a), QT == GGUF_BF16 ? f2bf_rn(b) : f2h_rn(b),
                               QT == GGUF_BF16 ? f2bf_rn(c) : f2h_rn(c), QT == GGUF_BF16 ? f2bf_rn(d) : f2h_rn(d)};
        if (vec) *reinterpret_cast<uint2 *>(o) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        else { o[0] = h[0]; o[1] = h[1]; o[2] = h[2]; o[3] = h[3]; }
    }
}

// where a walk over the sequence of tiles stands
struct AdCursor {
    int r, u, tile;   // request, unit within it, tile within the unit
    AdReq q;
};
__device__ __forceinline__ void ad_next_request(const AdShape &a, AdCursor &c) {
    do {
        c.r++;
        if (c.r >= a.p.R) return;
        c.q = ad_request(a, c.r);
    } while (c.q.nt == 0);
}
template <int RG>
__device__ __forceinline__ void ad_advance(const AdShape &a, AdCursor &c) {
    if (++c.tile < c.q.nt) return;
    c.tile = 0;
    const int G = (int)(a.p.h / a.p.hk);
    if (++c.u < (c.q.q * G + RG - 1) / RG * (int)a.p.hk) return;
    c.u = 0;
    ad_next_request(a, c);
}
// first token of a tile
__device__ __forceinline__ int ad_token(const AdCursor &c) {
    return (c.tile < c.q.n_sink ? c.tile : c.q.w_tile + c.tile - c.q.n_sink) * KV_TILE;
}
// page entry that a cursor's tile needs; -1 past the table
__device__ __forceinline__ int32_t ad_page(const AdShape &a, const AdCursor &c) {
    if (c.r >= a.p.R) return -1;
    const uint32_t pi = (uint32_t)ad_token(c) / (uint32_t)a.p.page;
    return pi < a.p.width ? a.p.table[c.r * a.p.ld + pi] : -1;
}

template <int D, int QT, int NT>
__global__ void __launch_bounds__(AdCfg<D, QT, NT>::WARPS * 32) attn_decode_kernel(const AdShape a) {
    using C = AdCfg<D, QT, NT>;
    using L = KvTile<D>;
    constexpr int RG = C::RG, NB = L::NB, BW = L::BW, NC = L::NC, ST = C::STAGES;
    constexpr int QP = QT == GGUF_F32 ? 3 : 1;   // bf16 parts of a query value
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[C::WARPS][ST];
    __shared__ int64_t chunk_end[C::WARPS * 32];
    __shared__ int64_t warp_sum[C::WARPS];
    // what each warp leaves at its end: 1 a piece of a unit that began before the warp, which 2 goes on past the
    // warp; 4 the first piece of a unit that goes on past the warp
    __shared__ int32_t left[C::WARPS], left_r[C::WARPS], left_u[C::WARPS];
    __shared__ int64_t left_end[C::WARPS];
    const Attn &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, q4 = lane & 3;
    uint8_t *ring = smem + warp * C::RING;
    if (lane == 0)
        for (int i = 0; i < ST; i++) tc::mbar_init(&bars[warp][i], 1);
    tc::fence_barrier_init();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // tiles of all requests: thread t holds those of requests [t * per, (t + 1) * per)
    constexpr int NTHR = C::WARPS * 32;
    const int R = (int)p.R, per = (R + NTHR - 1) / NTHR;
    int64_t mine = 0;
    for (int r = tid * per; r < min(R, (tid + 1) * per); r++) mine += ad_tiles(a, ad_request(a, r), RG);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; w++) incl += warp_sum[w];
    chunk_end[tid] = incl;
    __syncthreads();
    const int64_t total = chunk_end[NTHR - 1];
    const int64_t per_cta = (total + gridDim.x - 1) / gridDim.x;
    const int64_t cta0 = min(total, (int64_t)blockIdx.x * per_cta), cta1 = min(total, cta0 + per_cta);
    const int64_t per_warp = (cta1 - cta0 + C::WARPS - 1) / C::WARPS;
    const int64_t t0 = min(cta1, cta0 + warp * per_warp), t1 = min(cta1, t0 + per_warp);

    int flags = 0, open_r = 0, open_u = 0;
    int64_t open_end = 0;
    if (t0 < t1) {
        // the request, unit and tile of t0
        AdCursor cur;
        {
            int lo = -1, hi = NTHR - 1;   // first chunk that ends past t0
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (chunk_end[mid] > t0) hi = mid;
                else lo = mid;
            }
            int64_t before = hi > 0 ? chunk_end[hi - 1] : 0;
            cur.r = hi * per;
            for (;; cur.r++) {   // it is there: t0 < total
                cur.q = ad_request(a, cur.r);
                const int64_t n = ad_tiles(a, cur.q, RG);
                if (before + n > t0) break;
                before += n;
            }
            const int64_t off = t0 - before;
            cur.u = (int)(off / cur.q.nt);
            cur.tile = (int)(off - (int64_t)cur.u * cur.q.nt);
        }
        const int G = (int)(p.h / p.hk);
        const float sl = p.scale * 1.44269504088896341f;
        AdCursor ahead = cur;
        int64_t n_ahead = t0;      // next tile to ask for
        uint32_t bad = 0;          // stages whose tile has no page
        int32_t pg = ad_page(a, ahead);
        auto ask = [&](int stage) {
            const int tok = ad_token(ahead);
            const bool ok = pg >= 0 && pg < p.n_pages;
            bad = ok ? bad & ~(1u << stage) : bad | (1u << stage);
            if (lane == 0) {
                if (ok) {
                    const int head = ahead.u % (int)p.hk;
                    const uint32_t off = (uint32_t)tok % (uint32_t)p.page;
                    const uint8_t *src = p.cache + pg * kv_page_bytes(D, p.hk, p.page) +
                                         (head * (p.page / KV_TILE) + off / KV_TILE) * (int64_t)L::BYTES;
                    tc::mbar_arrive_expect_tx(&bars[warp][stage], L::BYTES);
                    bulk_load(ring + stage * L::BYTES, src, L::BYTES, &bars[warp][stage]);
                } else {
                    tc::mbar_arrive(&bars[warp][stage]);
                    if (p.status != nullptr) atomicAdd(p.status, 1);
                }
            }
            n_ahead++;
            if (n_ahead < t1) {
                ad_advance<RG>(a, ahead);
                pg = ad_page(a, ahead);
            }
        };
        for (int i = 0; i < ST && n_ahead < t1; i++) ask(i);

        uint32_t qa[QP][NB][2][NT][2];   // A fragments of the queries
        float corr[NB][NT];              // -24 sum of the row's block
        float o[NB][2][NT][4];
        float m[NT], lsum[NT];
        int pos[NT];                     // position of the rows g and g + 8; -1 for a row that is not there
        int pos_lo = 0, pos_hi = 0;
        bool fresh = true, dead = false;
        int stage = 0;
        uint32_t phase = 0;
        for (int64_t t = t0; t < t1; t++) {
            if (fresh) {   // a unit begins: its query rows
                const int row0 = cur.u / (int)p.hk * RG, head0 = cur.u % (int)p.hk * G;
                const int rows = cur.q.q * G;
                pos_lo = cur.q.pos0 + row0 / G;
                pos_hi = cur.q.pos0 + (min(rows, row0 + RG) - 1) / G;
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    const int row = row0 + g + 8 * n;
                    const bool there = row < rows;
                    pos[n] = there ? cur.q.pos0 + row / G : -1;
                    m[n] = -INFINITY;
                    lsum[n] = 0.0f;
                    const int64_t at = there ? (cur.q.rows0 + row / G) * p.ldq + (int64_t)(head0 + row % G) * D : 0;
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        float s = 0.0f;
                        uint32_t w[QP][4];
                        if constexpr (QT != GGUF_F32) {
                            const uint16_t *src = reinterpret_cast<const uint16_t *>(p.q) + at + 32 * b + 8 * q4;
                            uint32_t *x = w[0];
                            if (!there) x[0] = x[1] = x[2] = x[3] = 0;
                            else if (a.vec) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(src);
                                x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; i++) x[i] = src[2 * i] | (uint32_t)src[2 * i + 1] << 16;
                            }
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                s += QT == GGUF_BF16 ? bf2f(x[i] & 0xffff) + bf2f(x[i] >> 16) : h2f(x[i] & 0xffff) + h2f(x[i] >> 16);
                        } else {
                            const float *src = reinterpret_cast<const float *>(p.q) + at + 32 * b + 8 * q4;
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                float x[2] = {there ? src[2 * i] : 0.0f, there ? src[2 * i + 1] : 0.0f};
#pragma unroll
                                for (int part = 0; part < QP; part++) {   // what the part before left over
                                    const uint32_t lo = f2bf_rn(x[0]), hi = f2bf_rn(x[1]);
                                    w[part][i] = lo | hi << 16;
                                    x[0] -= bf2f((uint16_t)lo);
                                    x[1] -= bf2f((uint16_t)hi);
                                }
                            }
                        }
                        s += __shfl_xor_sync(0xffffffffu, s, 1);
                        s += __shfl_xor_sync(0xffffffffu, s, 2);
                        corr[b][n] = -24.0f * s;
#pragma unroll
                        for (int part = 0; part < QP; part++)
#pragma unroll
                            for (int k = 0; k < 2; k++)
#pragma unroll
                                for (int i = 0; i < 2; i++) qa[part][b][k][n][i] = w[part][2 * k + i];
#pragma unroll
                        for (int j = 0; j < 2; j++)
#pragma unroll
                            for (int i = 0; i < 4; i++) o[b][j][n][i] = 0.0f;
                    }
                }
                fresh = false;
            }
            bool ok = false;
            if (t < n_ahead) {
                ok = tc::mbar_wait(&bars[warp][stage], phase);
                if (!__all_sync(0xffffffffu, ok)) {   // given up: ask for no more, wait for what is under way
                    if (lane == 0 && a.err != nullptr) atomicOr(a.err, 1);
                    dead = true;
                    ok = false;
                }
                ok = ok && !((bad >> stage) & 1);
            }
            const uint8_t *tile = ring + stage * L::BYTES;
            if (ok) {
                // ---- scores of 16 tokens: n-tile e holds tokens 8e + 2 q4, + 1
                float s[2][NT == 2 ? 4 : 2];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    uint32_t ds[NB];
                    lds_words<NB>(tile + L::KS + 4 * (4 * e + q4) * NB, ds);
#pragma unroll
                    for (int i = 0; i < (NT == 2 ? 4 : 2); i++) s[e][i] = 0.0f;
#pragma unroll
                    for (int c = 0; c < NC; c++) {
                        uint32_t w[BW];
                        lds_words<BW>(tile + 4 * ((e * NC + c) * 32 + lane) * BW, w);
#pragma unroll
                        for (int x = 0; x < BW; x++) {
                            const int b = c * BW + x;
                            float acc[4];
                            acc[0] = acc[1] = QT == GGUF_F32 ? 0.0f : corr[b][0];
                            acc[2] = acc[3] = QT == GGUF_F32 || NT == 1 ? 0.0f : corr[b][NT - 1];
                            uint32_t cb[4];
                            if constexpr (QT == GGUF_F16) {
                                cb[0] = codes_f16<0>(w[x]); cb[1] = codes_f16<1>(w[x]);
                                cb[2] = codes_f16<2>(w[x]); cb[3] = codes_f16<3>(w[x]);
                            } else {
                                cb[0] = codes_bf16<0>(w[x]); cb[1] = codes_bf16<1>(w[x]);
                                cb[2] = codes_bf16<2>(w[x]); cb[3] = codes_bf16<3>(w[x]);
                            }
                            if constexpr (QT == GGUF_F32) {   // the exact c - 8, so that nothing large cancels
#pragma unroll
                                for (int i = 0; i < 4; i++) {
                                    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&cb[i]),
                                                                     __float2bfloat162_rn(24.0f));
                                    cb[i] = *reinterpret_cast<const uint32_t *>(&v);
                                }
                            }
#pragma unroll
                            for (int part = 0; part < QP; part++)
#pragma unroll
                                for (int k = 0; k < 2; k++) {
                                    const uint32_t a1 = NT == 2 ? qa[part][b][k][NT - 1][0] : 0u;
                                    const uint32_t a3 = NT == 2 ? qa[part][b][k][NT - 1][1] : 0u;
                                    if constexpr (QT == GGUF_F16)
                                        mma_f16_16816(acc, qa[part][b][k][0][0], a1, qa[part][b][k][0][1], a3, cb[2 * k], cb[2 * k + 1]);
                                    else
                                        mma_bf16_16816(acc, qa[part][b][k][0][0], a1, qa[part][b][k][0][1], a3, cb[2 * k], cb[2 * k + 1]);
                                }
                            const float2 d = __half22float2(u2h(ds[b]));
#pragma unroll
                            for (int i = 0; i < (NT == 2 ? 4 : 2); i++)
                                s[e][i] = fmaf(acc[i], i & 1 ? d.y : d.x, s[e][i]);
                        }
                    }
                }
                // ---- what is not seen; scores in units of log2
                const int tok = ad_token(cur);
                const bool whole = tok + KV_TILE - 1 <= pos_lo &&
                                   (p.window <= 0 || tok > pos_hi - p.window || tok + KV_TILE <= p.sinks);
                uint32_t keep[2] = {0xffffffffu, 0xffffffffu};   // value scales of tokens that some row sees
#pragma unroll
                for (int e = 0; e < 2; e++)
#pragma unroll
                    for (int i = 0; i < (NT == 2 ? 4 : 2); i++) s[e][i] *= sl;
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        keep[e] = 0;
#pragma unroll
                        for (int j = 0; j < 2; j++) {
                            const int at = tok + 8 * e + 2 * q4 + j;
                            const bool in = p.window <= 0 || at < p.sinks;
                            if (at <= pos_hi && (in || at > pos_lo - p.window)) keep[e] |= 0xffffu << (16 * j);
#pragma unroll
                            for (int n = 0; n < NT; n++)
                                if (!(at <= pos[n] && (in || at > pos[n] - p.window))) s[e][2 * n + j] = -INFINITY;
                        }
                    }
                }
                // ---- online softmax
                uint32_t pb[NT][2], pl[NT][2];
                bool grew = false;
                float alpha[NT];
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    float mx = fmaxf(fmaxf(s[0][2 * n], s[0][2 * n + 1]), fmaxf(s[1][2 * n], s[1][2 * n + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float mn = fmaxf(m[n], mx);
                    alpha[n] = 1.0f;
                    if (mn > m[n]) {
                        alpha[n] = ex2(m[n] - mn);   // 0 from -inf
                        grew = true;
                    }
                    m[n] = mn;
                    const float base = mn == -INFINITY ? 0.0f : AD_PBITS - mn;
                    float pr[2][2];
#pragma unroll
                    for (int e = 0; e < 2; e++)
#pragma unroll
                        for (int j = 0; j < 2; j++) pr[e][j] = ex2(s[e][2 * n + j] + base);
                    lsum[n] = fmaf(lsum[n], alpha[n], (pr[0][0] + pr[0][1]) + (pr[1][0] + pr[1][1]));
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        pb[n][e] = pack_h2(pr[e][0], pr[e][1]);
                        if constexpr (QT == GGUF_F32) {
                            const float2 hi = __half22float2(u2h(pb[n][e]));
                            pl[n][e] = pack_h2(pr[e][0] - hi.x, pr[e][1] - hi.y);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int n = 0; n < NT; n++) {   // the columns of O^T: rows 2 q4, 2 q4 + 1
                        const float a0 = __shfl_sync(0xffffffffu, alpha[n], 8 * q4);
                        const float a1 = __shfl_sync(0xffffffffu, alpha[n], 8 * q4 + 4);
#pragma unroll
                        for (int b = 0; b < NB; b++)
#pragma unroll
                            for (int j = 0; j < 2; j++) {
                                o[b][j][n][0] *= a0; o[b][j][n][1] *= a1;
                                o[b][j][n][2] *= a0; o[b][j][n][3] *= a1;
                            }
                    }
                }
                // ---- outputs
                uint32_t dv[2][NB];
#pragma unroll
                for (int e = 0; e < 2; e++) lds_words<NB>(tile + L::VS + 4 * (4 * e + q4) * NB, dv[e]);
                if (!whole) {
#pragma unroll
                    for (int b = 0; b < NB; b++) { dv[0][b] &= keep[0]; dv[1][b] &= keep[1]; }
                }
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    uint32_t w[2][BW];
#pragma unroll
                    for (int e = 0; e < 2; e++) lds_words<BW>(tile + L::VC + 4 * ((e * NC + c) * 32 + lane) * BW, w[e]);
#pragma unroll
                    for (int x = 0; x < BW; x++) {
                        const int b = c * BW + x;
                        const __half2 off = u2h(0x64086408u);   // 1032
                        __half2 v[2][4];
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            v[e][0] = __hsub2(codes_1024<0>(w[e][x]), off);
                            v[e][1] = __hsub2(codes_1024<1>(w[e][x]), off);
                            v[e][2] = __hsub2(codes_1024<2>(w[e][x]), off);
                            v[e][3] = __hsub2(codes_1024<3>(w[e][x]), off);
                        }
#pragma unroll
                        for (int j = 0; j < 2; j++) {
                            const __half2 d0 = u2h(dv[0][b]), d1 = u2h(dv[1][b]);
                            const __half2 f0 = __hmul2(v[0][2 * j], d0), f1 = __hmul2(v[0][2 * j + 1], d0);
                            const __half2 f2 = __hmul2(v[1][2 * j], d1), f3 = __hmul2(v[1][2 * j + 1], d1);
#pragma unroll
                            for (int n = 0; n < NT; n++)
                                mma_f16_16816(o[b][j][n], h2u(f0), h2u(f1), h2u(f2), h2u(f3), pb[n][0], pb[n][1]);
                            if constexpr (QT == GGUF_F32) {
                                const __half2 l0 = __hfma2(v[0][2 * j], d0, __hneg2(f0));
                                const __half2 l1 = __hfma2(v[0][2 * j + 1], d0, __hneg2(f1));
                                const __half2 l2 = __hfma2(v[1][2 * j], d1, __hneg2(f2));
                                const __half2 l3 = __hfma2(v[1][2 * j + 1], d1, __hneg2(f3));
#pragma unroll
                                for (int n = 0; n < NT; n++) {
                                    mma_f16_16816(o[b][j][n], h2u(l0), h2u(l1), h2u(l2), h2u(l3), pb[n][0], pb[n][1]);
                                    mma_f16_16816(o[b][j][n], h2u(f0), h2u(f1), h2u(f2), h2u(f3), pl[n][0], pl[n][1]);
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();   // the stage is free
            if (n_ahead < t1 && !dead) ask(stage);
            if (++stage == ST) { stage = 0; phase ^= 1; }

            // ---- the unit's or the warp's end
            const bool unit_end = cur.tile == cur.q.nt - 1;
            if (unit_end || t == t1 - 1) {
                const bool began = t - cur.tile >= t0;   // with this warp
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    lsum[n] += __shfl_xor_sync(0xffffffffu, lsum[n], 1);
                    lsum[n] += __shfl_xor_sync(0xffffffffu, lsum[n], 2);
                }
                if (unit_end && began) {   // a whole unit
                    const int row0 = cur.u / (int)p.hk * RG, head0 = cur.u % (int)p.hk * G, rows = cur.q.q * G;
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int j = 0; j < 2; j++) {
                            const float l = __shfl_sync(0xffffffffu, lsum[n], 8 * q4 + 4 * j);
                            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                            const int row = row0 + 8 * n + 2 * q4 + j;
                            if (row < rows) {
                                const int64_t at = (cur.q.rows0 + row / G) * p.ldo + (int64_t)(head0 + row % G) * D;
#pragma unroll
                                for (int b = 0; b < NB; b++)
                                    store4<QT>(p.out, at + 32 * b + 4 * g, a.vec, o[b][0][n][j] * inv, o[b][0][n][2 + j] * inv,
                                               o[b][1][n][j] * inv, o[b][1][n][2 + j] * inv);
                            }
                        }
                } else {
                    // a unit from before the warp leaves its piece beside the ring; one that goes on past the warp
                    // ends with the warp's last tile, and takes the ring, where no copy is under way any more
                    flags |= began ? 4 : unit_end ? 1 : 3;
                    if (began) { open_r = cur.r; open_u = cur.u; open_end = t - cur.tile + cur.q.nt; }
                    float *dst = reinterpret_cast<float *>(began ? ring : smem + C::WARPS * C::RING + warp * C::SLOT);
#pragma unroll
                    for (int n = 0; n < NT; n++) {
#pragma unroll
                        for (int j = 0; j < 2; j++)
#pragma unroll
                            for (int b = 0; b < NB; b++)
                                *reinterpret_cast<float4 *>(dst + (8 * n + 2 * q4 + j) * D + 32 * b + 4 * g) =
                                    make_float4(o[b][0][n][j], o[b][0][n][2 + j], o[b][1][n][j], o[b][1][n][2 + j]);
                        if (q4 == 0) {
                            dst[RG * D + 2 * (8 * n + g)] = m[n];
                            dst[RG * D + 2 * (8 * n + g) + 1] = lsum[n];
                        }
                    }
                }
                fresh = true;
            }
            if (t + 1 < t1) ad_advance<RG>(a, cur);
        }
    }
    if (lane == 0) {
        left[warp] = flags;
        left_r[warp] = open_r;
        left_u[warp] = open_u;
        left_end[warp] = open_end;
    }
    __syncthreads();

    // ---- the CTA's pieces: a chain is the piece that opens a unit (or the first warp's piece of a unit from the CTA
    // before) and the pieces of the warps after it
    const int G = (int)(p.h / p.hk);
    int chain = -1;          // the warp that opened the chain, -1 none; `orphan`: it came from the CTA before
    bool orphan = false;
    auto piece = [&](int w, bool first) {
        return reinterpret_cast<const float *>(first ? smem + w * C::RING : smem + C::WARPS * C::RING + w * C::SLOT);
    };
    auto join = [&](int end, bool open) {   // pieces of warps chain .. end
        const bool ring1 = !orphan;          // the first piece lies in the ring
        for (int it = tid; it < RG * D / 4; it += NTHR) {
            const int row = it / (D / 4), col = it % (D / 4) * 4;
            float mx = -INFINITY;
            for (int w = chain; w <= end; w++) mx = fmaxf(mx, piece(w, ring1 && w == chain)[RG * D + 2 * row]);
            const float base = mx == -INFINITY ? 0.0f : mx;
            float l = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int w = chain; w <= end; w++) {
                const float *src = piece(w, ring1 && w == chain);
                const float f = ex2(src[RG * D + 2 * row] - base);
                const float4 x = *reinterpret_cast<const float4 *>(src + row * D + col);
                l = fmaf(f, src[RG * D + 2 * row + 1], l);
                v.x = fmaf(f, x.x, v.x); v.y = fmaf(f, x.y, v.y); v.z = fmaf(f, x.z, v.z); v.w = fmaf(f, x.w, v.w);
            }
            if (!orphan && !open) {
                const AdReq q = ad_request(a, left_r[chain]);
                const int u = left_u[chain], at_row = u / (int)p.hk * RG + row;
                if (at_row < q.q * G) {
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    store4<QT>(p.out, (q.rows0 + at_row / G) * p.ldo + (int64_t)(u % (int)p.hk * G + at_row % G) * D + col,
                               a.vec, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                }
            } else {
                float *dst = a.part + (int64_t)(2 * blockIdx.x + (orphan ? 0 : 1)) * (C::SLOT / 4);
                *reinterpret_cast<float4 *>(dst + row * D + col) = v;
                if (col == 0) {
                    dst[RG * D + 2 * row] = mx;
                    dst[RG * D + 2 * row + 1] = l;
                }
            }
        }
    };
    int follow = 0, meta_r = 0, meta_u = 0;
    for (int w = 0; w < C::WARPS; w++) {
        const int f = left[w];
        if (f & 1) {
            if (chain < 0) { chain = w; orphan = true; }
            if (!(f & 2)) {
                join(w, false);
                chain = -1;
            }
        }
        if (f & 4) { chain = w; orphan = false; }
        if (chain >= 0 && (w == C::WARPS - 1 || left[w + 1] == 0)) {   // the CTA's last piece
            join(w, true);
            if (!orphan) {
                follow = (int)((left_end[chain] - cta1 + per_cta - 1) / per_cta);
                meta_r = left_r[chain];
                meta_u = left_u[chain];
            }
            break;
        }
    }
    if (tid == 0) {
        a.meta[4 * blockIdx.x] = follow;
        a.meta[4 * blockIdx.x + 1] = meta_r;
        a.meta[4 * blockIdx.x + 2] = meta_u;
    }
    // ---- queries that see no token
    for (int r = blockIdx.x * C::WARPS + warp; r < R; r += gridDim.x * C::WARPS) {
        const AdReq q = ad_request(a, r);
        if (q.nt > 0) continue;
        const int64_t n = (int64_t)q.q * p.h * (D / 4);
        for (int64_t i = lane; i < n; i += 32)
            store4<QT>(p.out, (q.rows0 + i / (p.h * (D / 4))) * p.ldo + i % (p.h * (D / 4)) * 4, a.vec, 0.0f, 0.0f, 0.0f, 0.0f);
    }
}

// Units that run over several CTAs of attn_decode_kernel: CTA c (blockIdx.x)
// joins the unit that CTA c opened and did not finish (meta[c] = {CTAs after c
// that hold pieces, request, unit}) for one query row (blockIdx.y), pieces in
// the order of the CTAs.
constexpr int AC_THREADS = 256;
constexpr int AC_MAX = 1024;   // CTAs of attn_decode_kernel at most
template <int D, int QT, int NT>
__global__ void __launch_bounds__(AC_THREADS) attn_combine_kernel(const AdShape a) {
    using C = AdCfg<D, QT, NT>;
    constexpr int COLS = D / 4, LANES = AC_THREADS / COLS;
    __shared__ float wt[AC_MAX], red[AC_THREADS / 32], red_l[AC_THREADS / 32];
    __shared__ float4 sum[AC_THREADS];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Attn &p = a.p;
    const int c = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
    const int n = a.meta[4 * c] + 1;
    if (n == 1) return;
    const AdReq q = ad_request(a, a.meta[4 * c + 1]);
    const int u = a.meta[4 * c + 2], G = (int)(p.h / p.hk), at_row = u / (int)p.hk * C::RG + row;
    if (at_row >= q.q * G) return;
    auto slot = [&](int k) { return a.part + (int64_t)(2 * (c + k) + (k == 0 ? 1 : 0)) * (C::SLOT / 4); };
    float mx = -INFINITY;
    for (int k = tid; k < n; k += AC_THREADS) mx = fmaxf(mx, slot(k)[C::RG * D + 2 * row]);
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (tid % 32 == 0) red[tid / 32] = mx;
    __syncthreads();
    for (int i = 0; i < AC_THREADS / 32; i++) mx = fmaxf(mx, red[i]);
    const float base = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f;
    for (int k = tid; k < n; k += AC_THREADS) {
        const float f = ex2(slot(k)[C::RG * D + 2 * row] - base);
        wt[k] = f;
        l = fmaf(f, slot(k)[C::RG * D + 2 * row + 1], l);
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (tid % 32 == 0) red_l[tid / 32] = l;
    __syncthreads();
    const int col = tid % COLS;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k = tid / COLS; k < n; k += LANES) {
        const float f = wt[k];
        const float4 x = *reinterpret_cast<const float4 *>(slot(k) + row * D + 4 * col);
        v.x = fmaf(f, x.x, v.x); v.y = fmaf(f, x.y, v.y); v.z = fmaf(f, x.z, v.z); v.w = fmaf(f, x.w, v.w);
    }
    sum[tid] = v;
    __syncthreads();
    if (tid >= COLS) return;
    l = 0.0f;
    for (int i = 0; i < AC_THREADS / 32; i++) l += red_l[i];
    for (int i = 1; i < LANES; i++) {
        const float4 x = sum[i * COLS + tid];
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    store4<QT>(p.out, (q.rows0 + at_row / G) * p.ldo + (int64_t)(u % (int)p.hk * G + at_row % G) * D + 4 * col, a.vec,
               v.x * inv, v.y * inv, v.z * inv, v.w * inv);
}

template <int D, int QT, int NT>
static cudaError_t attn_decode_run(const AdShape &a, int ctas, cudaStream_t s) {
    using C = AdCfg<D, QT, NT>;
    cudaError_t err = cudaSuccess;
    const void *kern = (const void *)attn_decode_kernel<D, QT, NT>;
    if (kernel_occupancy(kern, C::WARPS * 32, C::SMEM, &err) == 0) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::WARPS * 32);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, QT, NT>, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)ctas, C::RG);
    cfg.blockDim = dim3(AC_THREADS);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn_combine_kernel<D, QT, NT>, a);
}

}  // namespace gg
