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
// warp's own ring of stages; two tiles are treated at a time.  Scores and
// outputs are warp-level 16x8x16 matrix products with the codes as operands:
//   S^T = K Q^T    A = 16 keys, B = 8 query rows.  One and-or puts two 4-bit codes
//                  c into the mantissas of 1024: the numbers 1024 + c, or from the
//                  odd nibbles 1024 + 16 c, whose query values are held / 16.  The
//                  accumulator starts from what the offsets add up to, negated, so
//                  it ends as sum q (c - 8) of one 32-value block, and the block's
//                  scale is applied to it in fp32.
//   O^T = V^T P^T  A = 16 values of a head over 16 tokens, B = 8 query rows: the
//                  accumulators of S^T, transposed 8 x 8 in registers.  v = d (c - 8)
//                  is rounded to fp16 (2^-12 of it at most) and p = 2^(s - max + 10)
//                  likewise; sums and statistics are fp32.
// 16-bit query rows are scaled by a power of two to a largest value in [2^8,
// 2^9), which fp16 holds exactly (bf16 values below 2^-15 of the row's largest
// lose bits).  fp32 queries use three bf16 parts of q, the exact c - 8, and
// high and low fp16 parts of p and v, for fp32 accuracy.
//
// Measured, with 8 rows a unit: 32 requests of up to 8192 tokens (32 query heads, 8
// KV heads of 128) 51.7 us, 3.7 TB/s; 4 of 131072 (16 heads, 2 of 256) 60.0 us, 3.6
// TB/s; 64 with a window of 4096 (32, 8 of 64) 48.8 us, 3.1 TB/s; 1 of 333 (fp32)
// 10.9 us.  What bounds it now: no unit is full (issue slots 59 %, DRAM 48 %, tensor
// pipe 20 %).  Three computing warps a scheduler, as many as the registers allow,
// wait in the chain of a step (scores, maxima by shuffles, probabilities, outputs),
// beside a unit's start and join (3500 cycles) and the second launch (about 4 us).
// With 4 heads per KV head a single token fills half of a unit's 8 rows.  Spills a
// thread: 96 bytes of stores and 56 of loads with heads of 128 (144 / 104 with 16
// rows), 32 / 16 of 64, 112 / 88 of 256, 248 / 204 of 256 in fp32.
//
// fp32 queries of any number come here, 8 rows a unit: 32 requests of 8192 tokens
// 112 us, a prompt of 1024 tokens 282 us, of 2048 1050 us, of 8192 15.9 ms (bf16 in
// the prompt kernel: 42, 71 and 662 us).
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "kv.cuh"
#include "tc.cuh"

namespace gg {

constexpr float AD_PBITS = 10.0f;   // probabilities are held times 2^10 (at most 1024): small ones keep their bits in fp16

constexpr int ad_warps(int d, bool f32, int nt) { return d == 256 || nt == 2 || f32 ? 8 : 12; }
template <int D, int QT, int NT>
struct AdCfg {
    static constexpr int RG = 8 * NT;                       // query rows of a unit
    // warps that compute; one more warpgroup holds the warp that asks for the copies, and gives registers to them
    static constexpr int WARPS = ad_warps(D, QT == GGUF_F32, NT);
    static constexpr int THREADS = WARPS * 32 + 128;
    static constexpr int REGS = WARPS == 8 ? 224 : 152, REGS_COPY = 56;   // sums of a launch at 168 and 128
    static constexpr int TP = D == 256 && QT == GGUF_F32 ? 1 : D == 64 && NT == 1 && QT != GGUF_F32 ? 4 : 2;   // tiles at a time
    static constexpr int STEP = TP * KvTile<D>::BYTES;
    static constexpr int STAGES = NT == 2 || TP == 1 ? 4 : D == 256 ? 2 : 3;   // as the shared memory allows
    static constexpr int RING = STAGES * STEP;              // bytes per warp, a multiple of 128
    static constexpr int SLOT = RG * (D + 2) * 4;           // one partial result: O, then max and sum per row
    static_assert(SLOT <= RING, "a warp's last partial result reuses its ring");
    static constexpr int SMEM = WARPS * (RING + SLOT);
};

// a / b of non-negative numbers, mostly small ones
__device__ __forceinline__ int64_t ad_div(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// An entry of the plan of gguf_prefix_attention (attn_prefix.cu): queries that see tiles of one row of the block table.
// Entry r < R: the queries of request r and its own tiles; entry R + g: those of all requests of group g and the tiles
// that the group shares.
struct PfEntry {
    int32_t rows0, q;          // first query token, query tokens
    int32_t tile0, tile1;      // tiles, before the window
    int32_t pos_min, pos_max;  // of the queries
    int32_t row;               // row of the block table
    int32_t group;             // of a request: its group's entry, -1 for none
};
// gguf_prefix_attention: what its kernels have beside AdShape's members.  A query row (token and head) has a record of
// PfStride<D> floats for its request's own tiles and, n_tokens x heads records later, one for its group's: output, maximum
// and sum of the first piece of its unit, the slot of the next piece and how many follow (as int32).  The rest of the unit's
// tiles went to the warps (decode kernel) or CTAs (prefill kernel) that follow in the sequence; each has one slot, of rows
// like records, for a unit that began before it.
struct PfShape {
    const int32_t *plan;       // header, entries, of each token its position, and its request and group (pf_pack), q_start, kv_len
    int32_t n_entries, chained;   // chained: the decode kernel follows the prefill kernel of the call; one by one, the other way round
    int32_t parts, pieces;     // slots of the decode kernel, of the prefill kernel
    int32_t tiles;             // that an entry has at most, whatever its lengths say
    float *records;
};
constexpr int PF_HEADER = 8, PF_MAGIC = 0x50465831;   // {magic, requests, groups, tokens, page size, short, 0, 0}; short: 1 where the
                                                      // first request of some group is shorter than what the group shares
// where q_start and kv_len lie in a plan, in words
__host__ __device__ __forceinline__ int64_t pf_lengths_at(int64_t R, int64_t NG, int64_t n_tokens) {
    return PF_HEADER + (R + NG) * (int64_t)(sizeof(PfEntry) / 4) + 2 * n_tokens;
}
template <int D> struct PfStride { static constexpr int64_t value = D + 4; };   // 16-byte steps

// the unit that a CTA began and did not end: the CTAs after it that hold pieces of it (0: there is none), its
// request's first query token, its first head, its first row; how many rows
struct AdMeta {
    int32_t follow, rows0, head0, row0, rows, pad[3];
};
// what the requests look like to the kernels of one call
struct AdShape {
    Attn p;
    int32_t min_rows, max_rows;   // requests with more than min_rows and at most max_rows query rows per KV head are taken
    int32_t vec;                  // rows of q and out start on 16 bytes
    int32_t G, hk;                // query heads per KV head, KV heads
    int32_t G_shift;              // G = 1 << G_shift, or -1
    int32_t tpp, tpp_shift;       // tiles per page, likewise
    int64_t page_bytes;
    int32_t max_splits;           // prefill: the pieces that a row block's tokens may be cut into at most (1: no join),
    int32_t *item_base;           // with the row blocks before each request, their rows, the pieces and the first that is cut,
    float *pieces;                // and the partial results, [row block][piece][row][max, sum, D values]
    int32_t whole;                // each CTA takes one whole unit (few short ones), and nothing is left to join
    float *part;                  // CTA-level partial results, two slots per CTA
    AdMeta *meta;                 // per CTA: the unit that goes on past it
    PfShape pf;                   // gguf_prefix_attention; else (and but for the plan, one by one) zeros
    int *err;                     // error word: a wait for a copy was given up
};

__host__ __device__ __forceinline__ int ad_token_of_row(const AdShape &a, int row) { return a.G_shift >= 0 ? row >> a.G_shift : row / a.G; }
// one request: its queries and the tiles that they see together
struct AdReq {
    int32_t rows0;        // first query token
    int32_t q;            // query tokens
    int32_t pos0;         // position of the first
    int32_t nt, n_sink, w_tile;   // tiles: n_sink first ones, from s_tile on, then from w_tile on
    int32_t row, pos_max;         // (PRE) row of the block table, the last position of a query
    int32_t s_tile;               // (PRE; else 0)
};
// FED: of gguf_prefix_attention one by one, of at most a.pf.tiles tiles
template <bool FED>
__device__ __forceinline__ AdReq ad_request(const AdShape &a, int r) {
    AdReq o;
    const Attn &p = a.p;
    const int G = a.G;
    o.rows0 = p.q_start[r];
    // of a request that is longer than max_q, or reaches past the rows of q, the first queries (their positions follow from
    // its whole length)
    const int64_t q = min(min((int64_t)p.q_start[r + 1] - o.rows0, p.max_q), p.n_tokens - o.rows0);
    const bool mine = o.rows0 >= 0 && q > 0 && q * G > a.min_rows && q * G <= a.max_rows;
    o.q = mine ? (int32_t)q : 0;
    o.row = r;
    o.pos_max = o.s_tile = 0;
    o.nt = o.n_sink = o.w_tile = 0;
    const int32_t kv = p.kv_len[r];
    o.pos0 = kv - (p.q_start[r + 1] - o.rows0);
    const int32_t last = o.pos0 + o.q - 1;
    if (o.q > 0 && last >= 0) {
        const int32_t end = FED ? min(last / KV_TILE + 1, a.pf.tiles) : last / KV_TILE + 1;
        o.nt = end;
        if (p.window > 0) {
            const int64_t w0 = (int64_t)o.pos0 - p.window + 1;
            o.w_tile = w0 > 0 ? (int32_t)(w0 / KV_TILE) : 0;
            if (FED) o.w_tile = min(o.w_tile, end);
            o.n_sink = (int32_t)min((p.sinks + KV_TILE - 1) / KV_TILE, (int64_t)o.w_tile);
            o.nt = o.n_sink + end - o.w_tile;
        }
    }
    return o;
}
// the same of an entry of the plan; what is not a plan of this call has no queries
__device__ __forceinline__ const PfEntry *pf_entries(const PfShape &f) { return reinterpret_cast<const PfEntry *>(f.plan + PF_HEADER); }
__device__ __forceinline__ int2 pf_token(const PfShape &f, int64_t t) {
    return reinterpret_cast<const int2 *>(pf_entries(f) + f.n_entries)[t];
}
// a request and its group (-1: none) in one word; -1: no request
__device__ __forceinline__ int pf_pack(int r, int g) { return r < 0 ? -1 : r | (g + 1) << 16; }
__device__ __forceinline__ int2 pf_unpack(int w) { return w < 0 ? make_int2(-1, -1) : make_int2(w & 0xffff, (w >> 16) - 1); }
__device__ __forceinline__ bool pf_plan_fits(const AdShape &a) {
    const int4 h = *reinterpret_cast<const int4 *>(a.pf.plan);
    return h.x == PF_MAGIC && h.y == (int32_t)a.p.R && h.z == a.pf.n_entries - (int32_t)a.p.R && h.w == (int32_t)a.p.n_tokens &&
           a.pf.plan[4] == (int32_t)a.p.page;
}
__device__ __forceinline__ AdReq pf_request(const AdShape &a, int e) {
    AdReq o;
    const Attn &p = a.p;
    const int4 u = reinterpret_cast<const int4 *>(pf_entries(a.pf) + e)[0], v = reinterpret_cast<const int4 *>(pf_entries(a.pf) + e)[1];
    o.rows0 = u.x;
    const int32_t tile0 = max(u.z, 0);
    int32_t tile1 = max(min(u.w, a.pf.tiles), tile0);
    o.q = u.y;
    o.pos_max = v.y;
    if (e < p.R && u.y > p.max_q) {   // the first max_q of a request's queries (the join leaves out the others of a group's)
        o.q = (int32_t)p.max_q;
        o.pos_max = v.x + o.q - 1;
        tile1 = max(min(tile1, o.pos_max >= 0 ? o.pos_max / KV_TILE + 1 : 0), tile0);
    }
    const int64_t rows = (int64_t)o.q * a.G;
    const bool mine = u.x >= 0 && u.y > 0 && (int64_t)u.x + u.y <= p.n_tokens && rows > a.min_rows && rows <= a.max_rows &&
                      v.z >= 0 && v.z < p.R;
    o.q = mine ? o.q : 0;
    o.pos0 = v.x;
    o.row = v.z;
    o.n_sink = 0;
    o.s_tile = o.w_tile = tile0;
    if (p.window > 0) {   // of the tiles from tile0 on (0 for a group): those that the sinks reach, then what the first query sees from
        const int64_t lo = (int64_t)v.x - p.window + 1;
        o.w_tile = max(lo > 0 ? (int32_t)min(lo / KV_TILE, (int64_t)tile1) : 0, tile0);
        o.n_sink = (int32_t)min(max((p.sinks + KV_TILE - 1) / KV_TILE - tile0, (int64_t)0), (int64_t)(o.w_tile - tile0));
    }
    o.nt = o.q > 0 ? o.n_sink + tile1 - o.w_tile : 0;
    return o;
}
template <bool PRE, bool FED>
__device__ __forceinline__ AdReq ad_request_of(const AdShape &a, int r) {
    if constexpr (PRE) return pf_request(a, r);
    else return ad_request<FED>(a, r);
}
template <bool PRE>
__device__ __forceinline__ int ad_requests(const AdShape &a) { return PRE ? a.pf.n_entries : (int)a.p.R; }

// the tile of the request's i-th one, and whether it is the first of its page among them (a page that is not there counts once)
__device__ __forceinline__ int ad_tile(const AdReq &q, int i) { return i < q.n_sink ? q.s_tile + i : q.w_tile + i - q.n_sink; }
__device__ __forceinline__ bool ad_starts_page(const AdShape &a, const AdReq &q, int i) {
    return i == 0 || ad_tile(q, i) / a.tpp != ad_tile(q, i - 1) / a.tpp;
}
// The row of the block table that a group's tiles are read through: that of its first request (q.row), which lists them if
// the last of them begins among its tokens, else that of the request whose query stands last, of several the first.
// By the lanes of `mask` together, of which the caller is the i-th of n.  Asked for only where the plan says that some first
// request is short: elsewhere the lengths' load need not come before the table's.
__device__ __forceinline__ int pf_row(const AdShape &a, const AdReq &q, int i, int n, uint32_t mask) {
    const int32_t *lens = a.pf.plan + pf_lengths_at(a.p.R, a.pf.n_entries - a.p.R, a.p.n_tokens) + a.p.R + 1;
    if ((int64_t)ad_tile(q, q.nt - 1) * KV_TILE < lens[q.row]) return q.row;
    uint32_t r = 0x7fffffff;
    for (int t = i; t < q.q; t += n) {
        const int2 at = pf_token(a.pf, q.rows0 + t);
        if (at.x == q.pos_max) r = min(r, (uint32_t)pf_unpack(at.y).x);
    }
    r = __reduce_min_sync(mask, r);
    return r < (uint32_t)a.p.R ? (int)r : q.row;
}
// its units: groups of rg query rows x KV heads
__device__ __forceinline__ int64_t ad_units(const AdShape &a, const AdReq &q, int rg) {
    return (int64_t)((q.q * a.G + rg - 1) / rg) * a.hk;
}
// d = A B + c of the warp-level 16x8x16 product, fp16 or (BF) bf16 operands
template <bool BF>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                          float c1, float c2, float c3) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// the 8 x 8 matrix of 16-bit values whose row lane / 4 holds the lane's pair, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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
// codes of nibble I of both halves of w as two fp16 numbers: 1024 + c (even I) or 1024 + 16 c (odd I)
template <int I>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
    return and_or(I < 2 ? w : w >> 8, I & 1 ? 0x00F000F0u : 0x000F000Fu, 0x64006400u);
}
// c - 8 of nibble I of both halves, exact
template <int I>
__device__ __forceinline__ __half2 signed_f16(uint32_t w) {
    const __half2 x = u2h(codes_f16<I>(w));
    return I & 1 ? __hfma2(x, u2h(0x2C002C00u), u2h(0xD480D480u))   // x / 16 - 72
                 : __hsub2(x, u2h(0x64086408u));                    // x - 1032
}
// the same as two bf16 numbers (from 16 + c)
template <int I>
__device__ __forceinline__ uint32_t signed_bf16(uint32_t w) {
    constexpr int SH = 4 * I - 3;
    const uint32_t x = and_or(SH < 0 ? w << (SH < 0 ? -SH : 0) : w >> (SH > 0 ? SH : 0), 0x00780078u, 0x41804180u);
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&x), __float2bfloat162_rn(24.0f));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// a power of two that takes the largest magnitude of a row of queries into [2^8, 2^9)
__device__ __forceinline__ float q_scale_up(float mx) {
    const uint32_t e = max(__float_as_uint(mx) >> 23, 16u);
    return __uint_as_float(mx == 0.0f ? 127u << 23 : min(262u - e, 254u) << 23);
}

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

using tc::bulk_load;

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
// the next unit with tiles
template <int RG, bool PRE, bool FED>
__device__ __forceinline__ void ad_next_unit(const AdShape &a, AdCursor &c) {
    c.tile = 0;
    if (++c.u < (c.q.q * a.G + RG - 1) / RG * a.hk) return;
    c.u = 0;
    do {
        if (++c.r >= ad_requests<PRE>(a)) return;
        c.q = ad_request_of<PRE, FED>(a, c.r);
    } while (c.q.nt == 0);
}

__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(tc::smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

// PRE: a launch of gguf_prefix_attention, whose units leave records and slots instead of outputs.  FED: a launch of its requests
// one by one, whose q_start and kv_len lie in the plan: none is taken where that is of other sizes.  (Asked by every launch it
// cost calls of 8 us 0.2.)
template <int D, int QT, int NT, bool PRE, bool FED>
__global__ void __launch_bounds__(AdCfg<D, QT, NT>::THREADS, 1) attn_decode_kernel(const AdShape a) {
    using C = AdCfg<D, QT, NT>;
    using L = KvTile<D>;
    constexpr int RG = C::RG, NB = L::NB, BW = L::BW, NC = L::NC, ST = C::STAGES, TP = C::TP;
    constexpr int QP = QT == GGUF_F32 ? 3 : 1;   // bf16 parts of a query value
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[C::WARPS][ST], freed[C::WARPS][ST];
    __shared__ uint32_t absent[C::WARPS][ST];   // tiles of a stage that have no page
    using At = std::conditional_t<PRE, int64_t, int32_t>;
    __shared__ int32_t start_r[C::WARPS];
    __shared__ At start_at[C::WARPS];   // where a warp starts: request, tile of the request's
    __shared__ int64_t warp_sum[C::THREADS / 32];
    __shared__ int32_t cta_tiles, blind;   // blind: some queries see no token
    __shared__ int32_t abort_word;
    volatile int32_t *abort_flag = &abort_word;
    // what each warp leaves at its end: 1 a piece of a unit that began before the warp, which 2 goes on past the
    // warp; 4 the first piece of a unit that goes on past the warp
    __shared__ int32_t left[C::WARPS], left_row[C::WARPS], left_u[C::WARPS], left_rows[C::WARPS];   // first query, unit, rows
    __shared__ int64_t left_end[C::WARPS];
    const Attn &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, q4 = lane & 3;
    if (tid < C::WARPS)
        for (int i = 0; i < ST; i++) { tc::mbar_init(&full[tid][i], 1); tc::mbar_init(&freed[tid][i], 1); }
    if (tid == 0) abort_word = blind = 0;
    tc::fence_barrier_init();
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // (the prefill kernel before it let this one start when all that came before the call was complete; it takes other
    // entries and writes other records, so there is nothing of it to wait for until the end)
    if (!PRE || !a.pf.chained) asm volatile("griddepcontrol.wait;" ::: "memory");

    // The cut.  Thread t holds requests [t * per, (t + 1) * per) of the sequence of tiles (or of units, where a CTA
    // takes one whole unit) and, once the sum of what comes before is known, writes down where the warps start whose
    // first tile lies in them.
    constexpr int NTHR = C::THREADS;
    const bool lost = FED && !pf_plan_fits(a);
    const int R = ad_requests<PRE>(a), per = (R + NTHR - 1) / NTHR, r0 = tid * per, r1 = lost ? r0 : min(R, r0 + per);
    if (lost && blockIdx.x == 0 && tid == 0 && p.status != nullptr) atomicAdd(p.status, 1);
    AdReq rq{};
    int64_t mine = 0;
    bool fits = true;   // (the entries are there to be read in any case)
    if constexpr (PRE) fits = pf_plan_fits(a);
    for (int r = r0; r < r1; r++) {
        rq = ad_request_of<PRE, FED>(a, r);
        if (PRE && !fits) rq.q = rq.nt = 0;
        mine += ad_units(a, rq, RG) * (!PRE && a.whole ? 1 : rq.nt);
        if (!PRE && rq.q > 0 && rq.nt == 0) blind = 1;   // (every writer writes the same)
    }
    int64_t before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) warp_sum[warp] = before;
    if (tid == 0) cta_tiles = 0;
    __syncthreads();
    before -= mine;
    int64_t total = 0;
    if constexpr (PRE) {   // (every warp adds up the warps' sums, a lane each)
        const int64_t one = lane < NTHR / 32 ? warp_sum[lane] : 0;
        int64_t upto = one;
#pragma unroll
        for (int o = 1; o < NTHR / 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        total = __shfl_sync(0xffffffffu, upto, NTHR / 32 - 1);
        before += __shfl_sync(0xffffffffu, upto - one, warp);
    } else {
#pragma unroll
        for (int w = 0; w < NTHR / 32; w++) {
            if (w < warp) before += warp_sum[w];
            total += warp_sum[w];
        }
    }
    // (PRE: the same for every warp, and a step's tiles at least)
    const int64_t even = PRE ? max((int64_t)TP, ad_div(total + gridDim.x * C::WARPS - 1, gridDim.x * C::WARPS)) : 0;
    const int64_t share = PRE ? even * C::WARPS : a.whole ? 1 : ad_div(total + gridDim.x - 1, gridDim.x);
    int64_t cta0 = min(total, (int64_t)blockIdx.x * share), cta1 = min(total, cta0 + share);
    int64_t per_warp = PRE ? even : ad_div(cta1 - cta0 + C::WARPS - 1, C::WARPS);
    for (int r = r0; r < r1; r++) {
        if (per > 1) {
            rq = ad_request_of<PRE, FED>(a, r);
            if (PRE && !fits) rq.q = rq.nt = 0;
        }
        const int64_t units = ad_units(a, rq, RG), n = units * (!PRE && a.whole ? 1 : rq.nt);
        if (before < cta1 && before + n > cta0) {
            if (!PRE && a.whole) {   // the CTA's unit: its tiles over the warps
                const int share_w = (rq.nt + C::WARPS - 1) / C::WARPS, first = (int)(cta0 - before) * rq.nt;
#pragma unroll
                for (int w = 0; w < C::WARPS; w++) {
                    start_r[w] = r;
                    start_at[w] = first + w * share_w;
                }
                cta_tiles = rq.nt;
            } else {   // (a request has less than 2^31 tiles in all its units)
                const int64_t skip = cta0 - before;
#pragma unroll
                for (int w = 0; w < C::WARPS; w++) {
                    const int64_t at = skip + w * per_warp;
                    if (at >= 0 && at < n) {
                        start_r[w] = r;
                        start_at[w] = (At)at;
                    }
                }
            }
        }
        before += n;
    }
    __syncthreads();
    if (!PRE && a.whole) {
        cta0 = 0;
        cta1 = cta_tiles;
        per_warp = (cta1 + C::WARPS - 1) / C::WARPS;
    }
    auto start_of = [&](int w) {
        AdCursor c;
        c.r = start_r[w];
        c.q = ad_request_of<PRE, FED>(a, c.r);
        if constexpr (PRE) c.u = (int)ad_div(start_at[w], c.q.nt);
        else c.u = (int)((uint32_t)start_at[w] / (uint32_t)c.q.nt);
        c.tile = (int)(start_at[w] - (At)c.u * c.q.nt);
        return c;
    };
    const int64_t per_cta = share;

    if (warp >= C::WARPS) {
        // ================= copies: 8 lanes ask for those of one computing warp, a step of TP tiles of a unit at a
        // time, a tile each; they hold the 16 table entries from page `base` on, the later 8 on their way early
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_COPY));
        constexpr int GW = C::WARPS / 4;   // warps that one of the four asks for: every scheduler bears the same load
        const bool mine8 = (lane >> 3) < GW;
        const int who = mine8 ? (warp - C::WARPS) * GW + (lane >> 3) : 0, l8 = lane & 7;
        const int64_t t0 = min(cta1, cta0 + who * per_warp), t1 = min(cta1, t0 + per_warp);
        int tiles = mine8 ? (int)min(t1 - t0, (int64_t)0x7fffffff) : 0;   // to ask for
        int unit = 0;                 // of them, those of the unit
        int stage = 0, uses = 0;      // next stage, and how often the ring has gone round
        const bool any_short = PRE && a.pf.plan[5] != 0;
        int base = 0, of = -1, rows_of = 0;   // the table entries: first page, and request; (PRE) the table's row
        int32_t now8 = -1, next8 = -1;
        const uint32_t tpp = (uint32_t)a.tpp;
        const int shift = a.tpp_shift;
        AdCursor feed{};
        if (tiles > 0) feed = start_of(who);
        const uint8_t *head = nullptr;   // the unit's head in page 0
        uint64_t idle_since = 0;
        // the lanes stay together: a step is taken by all groups whose stage is free
        for (;;) {
            bool go = tiles > 0 && (uses == 0 || mbar_test(&freed[who][stage], (uint32_t)(uses - 1) & 1u));
            go = __shfl_sync(0xffffffffu, go, lane & 24);
            if (!__any_sync(0xffffffffu, go)) {
                if (!__any_sync(0xffffffffu, tiles > 0 && !*abort_flag)) break;
                const uint64_t now = tc::globaltimer();
                if (idle_since == 0) idle_since = now;
                if (__any_sync(0xffffffffu, now - idle_since > tc::kWaitLimitNs)) { *abort_flag = 1; break; }
                __nanosleep(100);
                continue;
            }
            idle_since = 0;
            if (go && unit == 0) {
                if (feed.tile == feed.q.nt) ad_next_unit<RG, PRE, FED>(a, feed);
                unit = min(tiles, feed.q.nt - feed.tile);
                if (PRE && of != feed.r) rows_of = !any_short || feed.r < p.R ? feed.q.row : pf_row(a, feed.q, l8, 8, 0xffu << (lane & 24));
                head = p.cache + (int64_t)(feed.u % a.hk) * tpp * L::BYTES;
            }
            __syncwarp();
            const int cnt = min(TP, unit), i = feed.tile + max(min(l8, cnt - 1), 0);
            const int at = ad_tile(feed.q, i);
            const int page_at = shift >= 0 ? at >> shift : (int)((uint32_t)at / tpp), in_page = at - page_at * (int)tpp;
            const int first = __shfl_sync(0xffffffffu, page_at, lane & 24);
            const int32_t *row = p.table + (PRE ? rows_of : feed.r) * p.ld;
            if (go && (of != feed.r || first < base || first >= base + 8)) {
                const bool slide = of == feed.r && first >= base + 8 && first < base + 16;
                base = slide ? base + 8 : first & ~7;
                now8 = slide ? next8 : base + l8 < p.width ? row[base + l8] : -1;
                next8 = base + 8 + l8 < p.width ? row[base + 8 + l8] : -1;
                of = feed.r;
            }
            __syncwarp();
            const int d = page_at - base;
            const int32_t e0 = __shfl_sync(0xffffffffu, now8, (lane & 24) | (d & 7));
            const int32_t e1 = __shfl_sync(0xffffffffu, next8, (lane & 24) | (d & 7));
            int32_t pg = d < 8 ? e0 : e1;
            // a step may reach from the first tokens into the window: then the entry is read on the spot
            if (go && (d < 0 || d >= 16)) pg = page_at < p.width ? row[page_at] : -1;
            const bool ok = go && l8 < cnt && pg >= 0 && pg < p.n_pages;
            const uint32_t have = (__ballot_sync(0xffffffffu, ok) >> (lane & 24)) & 0xffu;
            if (go && l8 == 0) {
                const uint32_t none = ~have & ((1u << cnt) - 1);
                absent[who][stage] = none;
                tc::mbar_arrive_expect_tx(&full[who][stage], (uint32_t)__popc(have) * L::BYTES);
            }
            // counted by the request's first unit
            if (go && l8 < cnt && !ok && feed.u == 0 && p.status != nullptr && ad_starts_page(a, feed.q, i)) atomicAdd(p.status, 1);
            __syncwarp();
            if (ok)
                bulk_load(smem + who * C::RING + stage * C::STEP + l8 * L::BYTES,
                          head + pg * a.page_bytes + in_page * L::BYTES, L::BYTES, &full[who][stage]);
            if (go) {
                feed.tile += cnt;
                tiles -= cnt;
                unit -= cnt;
                if (++stage == ST) { stage = 0; uses++; }
            }
        }
        const int step = uses * ST + stage;
        if (*abort_flag && mine8)   // copies that are under way land before the CTA exits
            for (int i = max(0, step - ST); i < step; i++) tc::mbar_wait(&full[who][i % ST], (uint32_t)(i / ST) & 1u);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS));
    constexpr int NCOMP = C::WARPS * 32;
    auto join_warps = [] { asm volatile("bar.sync 1, %0;" ::"n"(NCOMP) : "memory"); };
    uint8_t *ring = smem + warp * C::RING;
    const int64_t t0 = min(cta1, cta0 + warp * per_warp), t1 = min(cta1, t0 + per_warp);
    int flags = 0, open_row = 0, open_rows = 0, open_u = 0;
    int64_t open_end = 0;
    if (t0 < t1) {
        AdCursor cur = start_of(warp);
        const int G = a.G;
        const float log2_scale = p.scale * 1.44269504088896341f;
        bool dead = false;
        int left_tiles = (int)min(t1 - t0, (int64_t)0x7fffffff), stage = 0;
        uint32_t phase = 0;
        while (left_tiles > 0) {
            // ---- a unit, or the part of it that is the warp's: its query rows
            const int group = cur.u / a.hk, row0 = group * RG, head0 = (cur.u - group * a.hk) * G, rows = cur.q.q * G;
            int pos_lo = cur.q.pos0 + ad_token_of_row(a, row0), pos_hi = cur.q.pos0 + ad_token_of_row(a, min(rows, row0 + RG) - 1);
            if constexpr (PRE) {   // rows of several requests: the first and the last position among them
                const int pos = pf_token(a.pf, cur.q.rows0 + ad_token_of_row(a, min(rows, row0 + RG) - 1 - lane % min(RG, rows - row0))).x;
                pos_lo = __reduce_min_sync(0xffffffffu, pos);
                pos_hi = __reduce_max_sync(0xffffffffu, pos);
            }
            uint32_t qb[QP][NB][2][NT][2];   // B fragments of the queries: row g, values 8 q4 .. of each block
            float corr[NB][NT][4];           // what the code offsets add to rows 2 q4, + 1 (twice: an accumulator), negated
            float sl[NT][2];                 // scores to log2 units
            float o[NB][2][NT][4];
            float m[NT][2], lsum[NT][2];
#pragma unroll
            for (int n = 0; n < NT; n++) {
                const int row = row0 + g + 8 * n;
                const bool there = row < rows;
                const int tk = ad_token_of_row(a, row);
                const int64_t at = there ? (cur.q.rows0 + tk) * p.ldq + (int64_t)(head0 + row - tk * G) * D : 0;
                if constexpr (QT != GGUF_F32) {
                    uint32_t w[NB][4];
                    float mx = 0.0f;
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        const uint16_t *from = reinterpret_cast<const uint16_t *>(p.q) + at + 32 * b + 8 * q4;
                        if (!there) w[b][0] = w[b][1] = w[b][2] = w[b][3] = 0;
                        else if (a.vec) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(from);
                            w[b][0] = v.x; w[b][1] = v.y; w[b][2] = v.z; w[b][3] = v.w;
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; i++) w[b][i] = from[2 * i] | (uint32_t)from[2 * i + 1] << 16;
                        }
#pragma unroll
                        for (int i = 0; i < 4; i++) mx = fmaxf(mx, fmaxf(fabsf(from16<QT>(w[b][i] & 0xffff)), fabsf(from16<QT>(w[b][i] >> 16))));
                    }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float up = q_scale_up(mx), inv = 1.0f / up;
#pragma unroll
                    for (int j = 0; j < 2; j++) sl[n][j] = log2_scale * __shfl_sync(0xffffffffu, inv, 8 * q4 + 4 * j);
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        float s = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; i++) {   // pair i belongs to nibble i of the key's word
                            const float x = up * from16<QT>(w[b][i] & 0xffff), y = up * from16<QT>(w[b][i] >> 16);
                            const float f = i & 1 ? 0.0625f : 1.0f;
                            qb[0][b][i >> 1][n][i & 1] = pack_h2(x * f, y * f);
                            s = fmaf(i & 1 ? -72.0f : -1032.0f, x + y, s);
                        }
                        s += __shfl_xor_sync(0xffffffffu, s, 1);
                        s += __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
                        for (int j = 0; j < 4; j++) corr[b][n][j] = __shfl_sync(0xffffffffu, s, 8 * q4 + 4 * (j & 1) + (j >> 1));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 2; j++) sl[n][j] = log2_scale;
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        const float *from = reinterpret_cast<const float *>(p.q) + at + 32 * b + 8 * q4;
                        corr[b][n][0] = corr[b][n][1] = corr[b][n][2] = corr[b][n][3] = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            float x = there ? from[2 * i] : 0.0f, y = there ? from[2 * i + 1] : 0.0f;
#pragma unroll
                            for (int part = 0; part < QP; part++) {   // what the part before left over
                                const uint32_t lo = f2bf_rn(x), hi = f2bf_rn(y);
                                qb[part][b][i >> 1][n][i & 1] = lo | hi << 16;
                                x -= bf2f((uint16_t)lo);
                                y -= bf2f((uint16_t)hi);
                            }
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    m[n][j] = -INFINITY;
                    lsum[n][j] = 0.0f;
                }
#pragma unroll
                for (int b = 0; b < NB; b++)
#pragma unroll
                    for (int j = 0; j < 2; j++)
#pragma unroll
                        for (int i = 0; i < 4; i++) o[b][j][n][i] = 0.0f;
            }
            const bool began = cur.tile == 0;
            const int seg_end = min(cur.q.nt, cur.tile + left_tiles);
            left_tiles -= seg_end - cur.tile;
            // tiles that every row sees whole: below full_sink, and from full_lo to full_hi
            int full_sink = 0, full_lo = 0, full_hi = pos_lo < 0 ? 0 : (pos_lo + 1) / KV_TILE;
            if (PRE && p.window <= 0) full_hi -= cur.q.w_tile;
            if (p.window > 0) {
                full_sink = (int)min((int64_t)cur.q.n_sink, p.sinks / KV_TILE);
                if constexpr (PRE) full_sink = (int)min((int64_t)cur.q.n_sink, max(p.sinks / KV_TILE - cur.q.s_tile, (int64_t)0));
                const int64_t lo = (int64_t)pos_hi - p.window + 1;   // first token that the last row sees
                const int lo_tile = lo > 0 ? (int)((lo + KV_TILE - 1) / KV_TILE) : 0, shift = cur.q.n_sink - cur.q.w_tile;
                full_lo = max(lo_tile + shift, cur.q.n_sink);
                full_hi += shift;
            }
            while (cur.tile < seg_end) {
                // ---- up to TP tiles
                const uint8_t *tile0 = ring + stage * C::STEP;
                uint32_t use = 0;
                if (!dead) {
                    if (__all_sync(0xffffffffu, tc::mbar_wait(&full[warp][stage], phase)))
                        use = ~absent[warp][stage] & ((1u << min(TP, seg_end - cur.tile)) - 1);
                    else {   // given up: no tile counts any more
                        if (lane == 0 && a.err != nullptr) atomicOr(a.err, 1);
                        *abort_flag = 1;
                        dead = true;
                    }
                }
                // ---- scores: tokens g and g + 8 of a tile, rows 2 q4 and 2 q4 + 1
                float s[TP][NT][4];
#pragma unroll
                for (int x = 0; x < TP; x++) {
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int i = 0; i < 4; i++) s[x][n][i] = 0.0f;
                    uint32_t ds[2][NB];
#pragma unroll
                    for (int e = 0; e < 2; e++) lds_words<NB>(tile0 + x * L::BYTES + L::KS + 4 * (4 * e + (g >> 1)) * NB, ds[e]);
#pragma unroll
                    for (int c = 0; c < NC; c++) {
                        uint32_t w[2][BW];
#pragma unroll
                        for (int e = 0; e < 2; e++) lds_words<BW>(tile0 + x * L::BYTES + 4 * ((e * NC + c) * 32 + lane) * BW, w[e]);
#pragma unroll
                        for (int i = 0; i < BW; i++) {
                            const int b = c * BW + i;
                            uint32_t k0[4], k1[4];
                            if constexpr (QT != GGUF_F32) {
                                k0[0] = codes_f16<0>(w[0][i]); k0[1] = codes_f16<0>(w[1][i]);
                                k0[2] = codes_f16<1>(w[0][i]); k0[3] = codes_f16<1>(w[1][i]);
                                k1[0] = codes_f16<2>(w[0][i]); k1[1] = codes_f16<2>(w[1][i]);
                                k1[2] = codes_f16<3>(w[0][i]); k1[3] = codes_f16<3>(w[1][i]);
                            } else {
                                k0[0] = signed_bf16<0>(w[0][i]); k0[1] = signed_bf16<0>(w[1][i]);
                                k0[2] = signed_bf16<1>(w[0][i]); k0[3] = signed_bf16<1>(w[1][i]);
                                k1[0] = signed_bf16<2>(w[0][i]); k1[1] = signed_bf16<2>(w[1][i]);
                                k1[2] = signed_bf16<3>(w[0][i]); k1[3] = signed_bf16<3>(w[1][i]);
                            }
                            const float2 d = __half22float2(u2h(__byte_perm(ds[0][b], ds[1][b], (g & 1) ? 0x7632 : 0x5410)));
#pragma unroll
                            for (int n = 0; n < NT; n++) {
                                float acc[4];
                                mma_16816<QT == GGUF_F32>(acc, k0, qb[0][b][0][n][0], qb[0][b][0][n][1], corr[b][n][0],
                                                          corr[b][n][1], corr[b][n][2], corr[b][n][3]);
                                mma_16816<QT == GGUF_F32>(acc, k1, qb[0][b][1][n][0], qb[0][b][1][n][1], acc[0], acc[1], acc[2], acc[3]);
#pragma unroll
                                for (int part = 1; part < QP; part++) {
                                    mma_16816<true>(acc, k0, qb[part][b][0][n][0], qb[part][b][0][n][1], acc[0], acc[1], acc[2], acc[3]);
                                    mma_16816<true>(acc, k1, qb[part][b][1][n][0], qb[part][b][1][n][1], acc[0], acc[1], acc[2], acc[3]);
                                }
                                s[x][n][0] = fmaf(acc[0], d.x, s[x][n][0]);
                                s[x][n][1] = fmaf(acc[1], d.x, s[x][n][1]);
                                s[x][n][2] = fmaf(acc[2], d.y, s[x][n][2]);
                                s[x][n][3] = fmaf(acc[3], d.y, s[x][n][3]);
                            }
                        }
                    }
                }
                // ---- what is not seen
                const int i1 = cur.tile + TP;
                const bool whole = use == (1u << TP) - 1 && (i1 <= full_sink || (cur.tile >= full_lo && i1 <= full_hi));
                uint32_t keep[TP][2];   // value scales of tokens that some row sees
                if (!whole) {
                    int pos[NT][2];   // positions of rows 2 q4, + 1; -1 for a row that is not there
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int j = 0; j < 2; j++) {
                            const int row = row0 + 8 * n + 2 * q4 + j;
                            pos[n][j] = row >= rows ? -1 : PRE ? pf_token(a.pf, cur.q.rows0 + ad_token_of_row(a, row)).x
                                                               : cur.q.pos0 + ad_token_of_row(a, row);
                        }
#pragma unroll
                    for (int x = 0; x < TP; x++) {
                        const bool there = (use >> x) & 1;
                        const int tok = ad_tile(cur.q, cur.tile + x) * KV_TILE;
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            keep[x][e] = 0;
#pragma unroll
                            for (int j = 0; j < 2; j++) {
                                const int at = tok + 8 * e + 2 * q4 + j;
                                if (there && at <= pos_hi && (p.window <= 0 || at < p.sinks || at > pos_lo - p.window))
                                    keep[x][e] |= 0xffffu << (16 * j);
                            }
                            const int at = tok + 8 * e + g;
                            const bool in = p.window <= 0 || at < p.sinks;
#pragma unroll
                            for (int n = 0; n < NT; n++)
#pragma unroll
                                for (int j = 0; j < 2; j++)
                                    if (!(there && at <= pos[n][j] && (in || at > pos[n][j] - p.window))) s[x][n][2 * e + j] = -INFINITY;
                        }
                    }
                }
                // ---- online softmax
                uint32_t pb[TP][NT][2], pl[TP][NT][2];
                bool grew = false;
                float alpha[NT][2];
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int x = 0; x < TP; x++) mx = fmaxf(mx, fmaxf(s[x][n][j], s[x][n][2 + j]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float mn = fmaxf(m[n][j], mx * sl[n][j]);
                        alpha[n][j] = 1.0f;
                        if (mn > m[n][j]) {
                            alpha[n][j] = ex2(m[n][j] - mn);   // 0 from -inf
                            grew = true;
                        }
                        m[n][j] = mn;
                        const float base = mn == -INFINITY ? 0.0f : AD_PBITS - mn;
                        lsum[n][j] *= alpha[n][j];
#pragma unroll
                        for (int x = 0; x < TP; x++) {
                            s[x][n][j] = ex2(fmaf(s[x][n][j], sl[n][j], base));
                            s[x][n][2 + j] = ex2(fmaf(s[x][n][2 + j], sl[n][j], base));
                            lsum[n][j] += s[x][n][j] + s[x][n][2 + j];
                        }
                    }
#pragma unroll
                for (int x = 0; x < TP; x++)
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const uint32_t hi = pack_h2(s[x][n][2 * e], s[x][n][2 * e + 1]);
                            pb[x][n][e] = transpose8(hi);
                            if constexpr (QT == GGUF_F32) {
                                const float2 f = __half22float2(u2h(hi));
                                pl[x][n][e] = transpose8(pack_h2(s[x][n][2 * e] - f.x, s[x][n][2 * e + 1] - f.y));
                            }
                        }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int b = 0; b < NB; b++)
#pragma unroll
                            for (int j = 0; j < 2; j++)
#pragma unroll
                                for (int i = 0; i < 4; i++) o[b][j][n][i] *= alpha[n][i & 1];
                }
                // ---- outputs
#pragma unroll
                for (int x = 0; x < TP; x++) {
                    uint32_t dv[2][NB];
#pragma unroll
                    for (int e = 0; e < 2; e++) lds_words<NB>(tile0 + x * L::BYTES + L::VS + 4 * (4 * e + q4) * NB, dv[e]);
                    if (!whole) {
#pragma unroll
                        for (int b = 0; b < NB; b++) { dv[0][b] &= keep[x][0]; dv[1][b] &= keep[x][1]; }
                    }
#pragma unroll
                    for (int c = 0; c < NC; c++) {
                        uint32_t w[2][BW];
#pragma unroll
                        for (int e = 0; e < 2; e++) lds_words<BW>(tile0 + x * L::BYTES + L::VC + 4 * ((e * NC + c) * 32 + lane) * BW, w[e]);
#pragma unroll
                        for (int i = 0; i < BW; i++) {
                            const int b = c * BW + i;
                            const __half2 d0 = u2h(dv[0][b]), d1 = u2h(dv[1][b]);
                            const __half2 v[2][4] = {{signed_f16<0>(w[0][i]), signed_f16<1>(w[0][i]), signed_f16<2>(w[0][i]), signed_f16<3>(w[0][i])},
                                                     {signed_f16<0>(w[1][i]), signed_f16<1>(w[1][i]), signed_f16<2>(w[1][i]), signed_f16<3>(w[1][i])}};
#pragma unroll
                            for (int j = 0; j < 2; j++) {
                                const __half2 f[4] = {__hmul2(v[0][2 * j], d0), __hmul2(v[0][2 * j + 1], d0),
                                                      __hmul2(v[1][2 * j], d1), __hmul2(v[1][2 * j + 1], d1)};
                                const uint32_t fa[4] = {h2u(f[0]), h2u(f[1]), h2u(f[2]), h2u(f[3])};
#pragma unroll
                                for (int n = 0; n < NT; n++) {
                                    float(&oo)[4] = o[b][j][n];
                                    if constexpr (PRE && QT == GGUF_F32) {
                                        // The matrix unit cuts its sums off towards zero: added up in it, the outputs of a
                                        // long prefix shrink by about 2^-24 with every tile (7.6e-6 of them at 60 x 16000
                                        // tokens).  So a tile's products, the small ones first, and then one rounded sum.
                                        const uint32_t la[4] = {h2u(__hfma2(v[0][2 * j], d0, __hneg2(f[0]))), h2u(__hfma2(v[0][2 * j + 1], d0, __hneg2(f[1]))),
                                                                h2u(__hfma2(v[1][2 * j], d1, __hneg2(f[2]))), h2u(__hfma2(v[1][2 * j + 1], d1, __hneg2(f[3])))};
                                        float t[4];
                                        mma_16816<false>(t, la, pb[x][n][0], pb[x][n][1], 0.0f, 0.0f, 0.0f, 0.0f);
                                        mma_16816<false>(t, fa, pl[x][n][0], pl[x][n][1], t[0], t[1], t[2], t[3]);
                                        mma_16816<false>(t, fa, pb[x][n][0], pb[x][n][1], t[0], t[1], t[2], t[3]);
#pragma unroll
                                        for (int e = 0; e < 4; e++) oo[e] += t[e];
                                        continue;
                                    }
                                    mma_16816<false>(oo, fa, pb[x][n][0], pb[x][n][1], oo[0], oo[1], oo[2], oo[3]);
                                    if constexpr (QT == GGUF_F32) {
                                        const uint32_t la[4] = {h2u(__hfma2(v[0][2 * j], d0, __hneg2(f[0]))), h2u(__hfma2(v[0][2 * j + 1], d0, __hneg2(f[1]))),
                                                                h2u(__hfma2(v[1][2 * j], d1, __hneg2(f[2]))), h2u(__hfma2(v[1][2 * j + 1], d1, __hneg2(f[3])))};
                                        mma_16816<false>(oo, la, pb[x][n][0], pb[x][n][1], oo[0], oo[1], oo[2], oo[3]);
                                        mma_16816<false>(oo, fa, pl[x][n][0], pl[x][n][1], oo[0], oo[1], oo[2], oo[3]);
                                    }
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&freed[warp][stage]);
                cur.tile = min(cur.tile + TP, seg_end);
                if (++stage == ST) { stage = 0; phase ^= 1; }
            }

            // ---- the unit's or the warp's end
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int j = 0; j < 2; j++)
#pragma unroll
                    for (int i = 4; i < 32; i <<= 1) lsum[n][j] += __shfl_xor_sync(0xffffffffu, lsum[n][j], i);
            const bool unit_end = cur.tile == cur.q.nt;
            if constexpr (PRE) {   // rows of a unit that began here: their records; of one from the warp before: the warp's slot
                const int64_t at = (cur.q.rows0 + (cur.r >= p.R ? p.n_tokens : 0)) * p.h + head0;
                const int mine = blockIdx.x * C::WARPS + warp;
                float *slot = a.part + (int64_t)mine * (RG * PfStride<D>::value);
                const int follow = (int)ad_div(cur.q.nt - seg_end + per_warp - 1, per_warp);
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const int row = row0 + 8 * n + 2 * q4 + j;
                        if (row < rows) {
                            const int tk = ad_token_of_row(a, row);
                            float *to = began ? a.pf.records + (at + tk * p.h + row - tk * G) * PfStride<D>::value : slot + (row - row0) * PfStride<D>::value;
#pragma unroll
                            for (int b = 0; b < NB; b++)
                                *reinterpret_cast<float4 *>(to + 32 * b + 4 * g) =
                                    make_float4(o[b][0][n][j], o[b][0][n][2 + j], o[b][1][n][j], o[b][1][n][2 + j]);
                            if (g == 0) *reinterpret_cast<float4 *>(to + D) = make_float4(m[n][j], lsum[n][j], __int_as_float(mine + 1), __int_as_float(follow));
                        }
                    }
            } else if (unit_end && began) {   // a whole unit
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const float inv = lsum[n][j] == 0.0f ? 0.0f : 1.0f / lsum[n][j];
                        const int row = row0 + 8 * n + 2 * q4 + j;
                        if (row < rows) {
                            const int tk = ad_token_of_row(a, row);
                            const int64_t at = (cur.q.rows0 + tk) * p.ldo + (int64_t)(head0 + row - tk * G) * D;
#pragma unroll
                            for (int b = 0; b < NB; b++)
                                store4<QT>(p.out, at + 32 * b + 4 * g, a.vec, o[b][0][n][j] * inv, o[b][0][n][2 + j] * inv,
                                           o[b][1][n][j] * inv, o[b][1][n][2 + j] * inv);
                        }
                    }
            } else {
                // a unit from before the warp leaves its piece beside the ring; one that goes on past the warp ends
                // with the warp's last tile, and takes the ring, where no copy is under way any more
                flags |= began ? 4 : unit_end ? 1 : 3;
                if (began) { open_row = cur.q.rows0; open_rows = rows; open_u = cur.u; open_end = t1 + cur.q.nt - cur.tile; }
                __syncwarp();
                float *dst = reinterpret_cast<float *>(began ? ring : smem + C::WARPS * C::RING + warp * C::SLOT);
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int j = 0; j < 2; j++) {
#pragma unroll
                        for (int b = 0; b < NB; b++)
                            *reinterpret_cast<float4 *>(dst + (8 * n + 2 * q4 + j) * D + 32 * b + 4 * g) =
                                make_float4(o[b][0][n][j], o[b][0][n][2 + j], o[b][1][n][j], o[b][1][n][2 + j]);
                        if (g == 0) {
                            dst[RG * D + 2 * (8 * n + 2 * q4 + j)] = m[n][j];
                            dst[RG * D + 2 * (8 * n + 2 * q4 + j) + 1] = lsum[n][j];
                        }
                    }
            }
            if (left_tiles > 0) ad_next_unit<RG, PRE, FED>(a, cur);
        }
    }
    if constexpr (PRE) {   // what follows this launch may count on the prefill kernel's records too
        if (a.pf.chained) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    if (lane == 0) {
        left[warp] = flags;
        left_row[warp] = open_row;
        left_rows[warp] = open_rows;
        left_u[warp] = open_u;
        left_end[warp] = open_end;
    }
    join_warps();

    // ---- the CTA's pieces: a chain is the piece that opens a unit (or the first warp's piece of a unit from the CTA
    // before) and the pieces of the warps after it
    const int G = a.G;
    int chain = -1;          // the warp that opened the chain, -1 none; `orphan`: it came from the CTA before
    bool orphan = false;
    auto piece = [&](int w, bool first) {
        return reinterpret_cast<const float *>(first ? smem + w * C::RING : smem + C::WARPS * C::RING + w * C::SLOT);
    };
    auto join = [&](int end, bool open) {   // pieces of warps chain .. end
        const bool ring1 = !orphan;          // the first piece lies in the ring
        for (int it = tid; it < RG * D / 4; it += NCOMP) {
            const int row = it / (D / 4), col = it % (D / 4) * 4;
            float mx = -INFINITY;
#pragma unroll 4
            for (int w = chain; w <= end; w++) mx = fmaxf(mx, piece(w, ring1 && w == chain)[RG * D + 2 * row]);
            const float base = mx == -INFINITY ? 0.0f : mx;
            float l = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int w = chain; w <= end; w++) {
                const float *src = piece(w, ring1 && w == chain);
                const float2 ml = *reinterpret_cast<const float2 *>(src + RG * D + 2 * row);
                const float4 x = *reinterpret_cast<const float4 *>(src + row * D + col);
                const float f = ex2(ml.x - base);
                l = fmaf(f, ml.y, l);
                v.x = fmaf(f, x.x, v.x); v.y = fmaf(f, x.y, v.y); v.z = fmaf(f, x.z, v.z); v.w = fmaf(f, x.w, v.w);
            }
            if (!orphan && !open) {
                const int u = left_u[chain], group = u / a.hk, at_row = group * RG + row;
                if (at_row < left_rows[chain]) {
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    const int tk = ad_token_of_row(a, at_row);
                    store4<QT>(p.out, (int64_t)(left_row[chain] + tk) * p.ldo + (int64_t)((u - group * a.hk) * G + at_row - tk * G) * D + col,
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
    int follow = 0, opener = 0;
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
                opener = chain;
            }
            break;
        }
    }
    if (tid == 0 && !a.whole) {
        AdMeta m{};
        if (follow > 0) {
            const int u = left_u[opener], row0 = u / a.hk * RG;
            m = AdMeta{follow, left_row[opener], u % a.hk * G, row0, min(left_rows[opener] - row0, RG), {}};
        }
        a.meta[blockIdx.x] = m;
    }
    // ---- queries that see no token
    for (int r = blockIdx.x * C::WARPS + warp; blind && r < R; r += gridDim.x * C::WARPS) {
        const AdReq q = ad_request<FED>(a, r);
        if (q.nt > 0) continue;
        const int64_t n = (int64_t)q.q * p.h * (D / 4);
        for (int64_t i = lane; i < n; i += 32)
            store4<QT>(p.out, (q.rows0 + i / (p.h * (D / 4))) * p.ldo + i % (p.h * (D / 4)) * 4, a.vec, 0.0f, 0.0f, 0.0f, 0.0f);
    }
}

// Units that run over several CTAs of attn_decode_kernel: CTA c (blockIdx.x)
// joins the unit that CTA c opened and did not finish for one query row
// (blockIdx.y).  A thread takes four columns of every LANES-th piece, with a
// maximum and sum of its own, so that all loads are under way at once; the
// threads' results are joined in a fixed order.
constexpr int AC_THREADS = 256;
template <int D, int QT, int NT>
__global__ void __launch_bounds__(AC_THREADS) attn_combine_kernel(const AdShape a) {
    using C = AdCfg<D, QT, NT>;
    constexpr int COLS = D / 4, LANES = AC_THREADS / COLS;
    __shared__ float4 sum[LANES][COLS];
    __shared__ float2 stat[LANES];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Attn &p = a.p;
    const int c = blockIdx.x, row = blockIdx.y, col = threadIdx.x % COLS, k0 = threadIdx.x / COLS;
    const AdMeta m = a.meta[c];
    if (m.follow == 0 || row >= m.rows) return;
    const int n = m.follow + 1;
    float mx = -INFINITY, l = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int k = k0; k < n; k += LANES) {
        const float *src = a.part + (int64_t)(2 * (c + k) + (k == 0 ? 1 : 0)) * (C::SLOT / 4);
        const float4 x = *reinterpret_cast<const float4 *>(src + row * D + 4 * col);
        const float2 ml = *reinterpret_cast<const float2 *>(src + C::RG * D + 2 * row);
        const float mn = fmaxf(mx, ml.x), base = mn == -INFINITY ? 0.0f : mn;
        const float f = ex2(mx - base), h = ex2(ml.x - base);
        mx = mn;
        l = fmaf(l, f, ml.y * h);
        v.x = fmaf(v.x, f, x.x * h); v.y = fmaf(v.y, f, x.y * h);
        v.z = fmaf(v.z, f, x.z * h); v.w = fmaf(v.w, f, x.w * h);
    }
    sum[k0][col] = v;
    if (col == 0) stat[k0] = make_float2(mx, l);
    __syncthreads();
    if (threadIdx.x >= COLS) return;
    for (int i = 0; i < LANES; i++) mx = fmaxf(mx, stat[i].x);
    const float base = mx == -INFINITY ? 0.0f : mx;
    l = 0.0f;
    v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < LANES; i++) {
        const float h = ex2(stat[i].x - base);
        const float4 x = sum[i][col];
        l = fmaf(stat[i].y, h, l);
        v.x = fmaf(x.x, h, v.x); v.y = fmaf(x.y, h, v.y); v.z = fmaf(x.z, h, v.z); v.w = fmaf(x.w, h, v.w);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int G = a.G, at = m.row0 + row;
    store4<QT>(p.out, (m.rows0 + at / G) * p.ldo + (int64_t)(m.head0 + at % G) * D + 4 * col, a.vec, v.x * inv, v.y * inv,
               v.z * inv, v.w * inv);
}

template <int D, int QT, int NT>
static cudaError_t attn_decode_run(const AdShape &shape, int ctas, cudaStream_t s) {
    using C = AdCfg<D, QT, NT>;
    AdShape a = shape;
    // Few units of few tiles: a CTA each, and the second launch is saved (about 4 us).  The table's width bounds the
    // tiles: 2048 tokens are 128 tiles, 11 to 16 per warp, about 4 us.  (8 requests of 333 tokens, 32 heads of 128: 9.6 us
    // with a table of their width, 12.2 us with one of 32768 tokens.)
    const int64_t most_rows = std::min<int64_t>(a.max_rows, a.G * a.p.max_q);
    const int64_t units = a.p.R * a.p.hk * ((most_rows + C::RG - 1) / C::RG);
    const int64_t span = a.p.window > 0 ? std::min(a.p.width * a.p.page, a.p.window + a.p.sinks + a.p.max_q + 3 * KV_TILE)
                                        : a.p.width * a.p.page;
    a.whole = units <= ctas && span <= 2048;
    if (a.whole) ctas = (int)units;
    cudaError_t err = cudaSuccess;
    const void *kern = a.pf.plan ? (const void *)attn_decode_kernel<D, QT, NT, false, true> : (const void *)attn_decode_kernel<D, QT, NT, false, false>;
    if (kernel_occupancy(kern, C::THREADS, C::SMEM, &err) == 0) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[1] = {&a};
    cudaError_t e = cudaLaunchKernelExC(&cfg, kern, args);
    if (e != cudaSuccess || a.whole) return e;
    cfg.gridDim = dim3((unsigned)ctas, C::RG);
    cfg.blockDim = dim3(AC_THREADS);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn_combine_kernel<D, QT, NT>, a);
}

// the launch of gguf_prefix_attention
template <int D, int QT, int NT>
static cudaError_t attn_prefix_decode_run(const AdShape &a, int ctas, cudaStream_t s) {
    using C = AdCfg<D, QT, NT>;
    cudaError_t err = cudaSuccess;
    if (kernel_occupancy((const void *)attn_decode_kernel<D, QT, NT, true, false>, C::THREADS, C::SMEM, &err) == 0) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, QT, NT, true, false>, a);
}

}  // namespace gg
