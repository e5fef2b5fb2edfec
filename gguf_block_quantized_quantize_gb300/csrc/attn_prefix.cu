// gguf_prefix_plan and gguf_prefix_attention: attention of a batch whose requests
// share long prefixes, group by group, over the paged Q4_0 cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = 2^(s_ij - m),   j over [0, P) and [P, pos_i]
//
// The sums over the two ranges are taken apart, each with a maximum of its own,
// and joined: (m, l, O) + (m', l', O') = (M, 2^(m-M) l + 2^(m'-M) l', 2^(m-M) O +
// 2^(m'-M) O').  So the queries of all requests of a group stand together as the
// rows of one matrix against the group's P shared tokens, which come from memory
// once for all of them and are unpacked once for every 256 of the rows (128 with
// heads of 256, 8 or 16 in the kernel of few rows); only what a request has of its
// own is walked over per request.
//
// An entry of the plan is a set of consecutive queries and a range of tiles of one
// row of the block table: one for each request (its own tiles) and one for each
// group (the shared ones, through one request's row).  Entries with more than
// `few` query rows per KV head go to the tensor-core kernel of prompts
// (attn_prefill.cuh), the others to the kernel of few rows (attn_decode.cuh), each in
// a mode that cuts all its tiles evenly over the CTAs, takes every row's position
// from the plan, and leaves (m, l, O) in fp32: a record per query row for the first
// piece of its unit, a slot per warp or CTA for a unit that goes on from the one before.  The
// second kernel starts as the first one's CTAs end, without waiting for its results.
// The join takes a warp per query row; its record says where the other pieces lie.
//
// Measured in a captured graph, without the plan (3 to 4 us, once a step), and request
// by request: 32 x (8192 + 512) tokens, 32 / 8 heads of 128, bf16 39 and 69 us; 256 x
// (32768 + 128) 183 and 1690 us (0.74 PFLOP/s); 16 x 3.5 queries x (20000 + 400), heads of
// 64, fp16 50 and 82 us.  What bounds it: with many queries the tensor-core kernel (157 of
// the 183 us), whose matrix unit is 35 % active: its products read keys, values and Q from
// shared memory, which unpacking fills as well (4200 cycles a block of 128 tokens and 256
// rows; the products alone take 2600).  With few, latency: three kernels (19, 13.5 and 8 us
// by themselves) of 4 blocks, 3 tiles a warp and 20 pieces a row.  Spills a thread (stores /
// loads): tensor-core kernel 164 / 204 bytes with heads of 128, 84 / 92 of 64, 24 / 52 of
// 256; few rows 48 / 84 at most, fp32 with heads of 256 174 / 192.
#include <algorithm>

#include "attn_decode.cuh"
#include "attn_prefix.h"

namespace gg {

int *tg_error_word();   // the library's device error word (mmq.cu)

// ---------------------------------------------------------------- plan

struct PfPlanArgs {
    const int32_t *q_start, *kv_len;
    int64_t R;
    const int32_t *group_start, *prefix_len;
    int64_t NG, page, n_tokens;
    int32_t *plan;
};
// the last i in [0, n) with a[i] <= x, or -1 (a does not decrease)
__device__ __forceinline__ int64_t last_up_to(const int32_t *a, int64_t n, int64_t x) {
    int64_t lo = -1, hi = n;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}
// the arrays of requests and groups, in shared memory where they fit: a search of 9 steps takes 300 cycles there, 5000 in the
// L2, and what it finds is there too
constexpr int PF_HELD = 2048;
struct PfGroup {
    int64_t s, e;    // its requests
    int32_t tiles;   // shared ones
};
__device__ __forceinline__ PfGroup pf_group(const PfPlanArgs &p, int64_t g) {
    PfGroup o;
    o.s = max((int64_t)p.group_start[g], (int64_t)0);
    o.e = min((int64_t)p.group_start[g + 1], p.R);
    // whole pages: the one that a prefix ends in holds tokens of a request's own, and is its own
    const uint32_t page = (uint32_t)p.page;
    o.tiles = o.e - o.s >= 2 ? (int32_t)((uint32_t)max(p.prefix_len[g], 0) / page * (page / KV_TILE)) : 0;
    return o;
}
// the group with which a request shares tiles, or -1
__device__ __forceinline__ int pf_group_of(const PfPlanArgs &p, int64_t r) {
    if (p.NG == 0) return -1;   // (and there may be no arrays)
    const int64_t g = last_up_to(p.group_start, p.NG + 1, r);
    if (g < 0 || g >= p.NG) return -1;
    const PfGroup in = pf_group(p, g);
    return r >= in.s && r < in.e && in.tiles > 0 ? (int)g : -1;
}
// the queries of requests s .. e - 1 that the call's arrays hold
__device__ __forceinline__ void pf_queries(const PfPlanArgs &p, int64_t s, int64_t e, PfEntry &o) {
    const int64_t a = p.q_start[s], b = min((int64_t)p.q_start[e], p.n_tokens);
    o.rows0 = (int32_t)max(a, (int64_t)0);
    o.q = a >= 0 && b > a ? (int32_t)(b - a) : 0;
}

// Independent parts, over all CTAs: a thread per token, a thread per request, a warp per group, and the header by a CTA of its
// own.  Latency-bound: a token's request is a binary search of q_start, a group's positions a loop of its requests by 32.
constexpr int PF_THREADS = 256;
__global__ void __launch_bounds__(PF_THREADS) prefix_plan_kernel(const PfPlanArgs args) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ int32_t held[4][PF_HELD];
    PfPlanArgs p = args;
    if (p.R < PF_HELD) {
        for (int i = threadIdx.x; i <= p.R; i += PF_THREADS) {
            held[0][i] = p.q_start[i];
            if (i < p.R) held[1][i] = p.kv_len[i];
        }
        p.q_start = held[0];
        p.kv_len = held[1];
    }
    if (p.NG > 0 && p.NG < PF_HELD) {
        for (int i = threadIdx.x; i <= p.NG; i += PF_THREADS) {
            held[2][i] = p.group_start[i];
            if (i < p.NG) held[3][i] = p.prefix_len[i];
        }
        p.group_start = held[2];
        p.prefix_len = held[3];
    }
    __syncthreads();
    const int64_t id = (int64_t)blockIdx.x * PF_THREADS + threadIdx.x;
    PfEntry *entries = reinterpret_cast<PfEntry *>(p.plan + PF_HEADER);
    if (blockIdx.x == gridDim.x - 1) {   // the header
        bool is_short = false;   // some group's first request does not reach the end of what the group shares
        for (int64_t g = threadIdx.x; g < p.NG; g += PF_THREADS) {
            const PfGroup in = pf_group(p, g);
            is_short |= in.tiles > 0 && p.kv_len[in.s] < (int64_t)in.tiles * KV_TILE;
        }
        is_short = __syncthreads_or(is_short);
        const int32_t h[PF_HEADER] = {PF_MAGIC, (int32_t)p.R, (int32_t)p.NG, (int32_t)p.n_tokens, (int32_t)p.page, is_short, 0, 0};
        if (threadIdx.x == 0)
            for (int i = 0; i < PF_HEADER; i++) p.plan[i] = h[i];
        return;
    }
    int32_t *starts = p.plan + pf_lengths_at(p.R, p.NG, p.n_tokens);   // what a call takes whose requests go one by one
    if (id <= p.R) starts[id] = p.q_start[id];
    if (id < p.R) starts[p.R + 1 + id] = p.kv_len[id];
    if (id < p.n_tokens) {
        const int64_t r = last_up_to(p.q_start, p.R + 1, id);
        int2 o = make_int2(-1, -1);
        if (r >= 0 && r < p.R) {
            o.x = (int)(p.kv_len[r] - ((int64_t)p.q_start[r + 1] - id));
            o.y = pf_pack((int)r, pf_group_of(p, r));
        }
        reinterpret_cast<int2 *>(entries + p.R + p.NG)[id] = o;
    }
    if (id < p.R) {
        PfEntry o{};
        pf_queries(p, id, id + 1, o);
        o.pos_min = (int32_t)max(p.kv_len[id] - ((int64_t)p.q_start[id + 1] - p.q_start[id]), (int64_t)INT32_MIN / 2);
        o.pos_max = o.pos_min + o.q - 1;
        const int g = pf_group_of(p, id);
        o.group = -1;
        if (g >= 0) {
            o.tile0 = pf_group(p, g).tiles;
            o.group = (int32_t)(p.R + g);
        }
        o.tile1 = max(o.tile0, o.q > 0 && o.pos_max >= 0 ? o.pos_max / KV_TILE + 1 : 0);
        o.row = (int32_t)id;
        entries[id] = o;
    }
    const int64_t g = id >> 5;
    if (g < p.NG) {   // whole warps
        const PfGroup in = pf_group(p, g);
        PfEntry o{};
        if (in.tiles > 0) {
            pf_queries(p, in.s, in.e, o);
            int lo = INT32_MAX, hi = INT32_MIN;
            for (int64_t r = in.s + (threadIdx.x & 31); r < in.e; r += 32) {
                PfEntry one{};
                pf_queries(p, r, r + 1, one);
                if (one.q == 0) continue;
                const int first = (int)max(p.kv_len[r] - ((int64_t)p.q_start[r + 1] - p.q_start[r]), (int64_t)INT32_MIN / 2);
                lo = min(lo, first);
                hi = max(hi, first + one.q - 1);
            }
            o.pos_min = __reduce_min_sync(0xffffffffu, lo);
            o.pos_max = __reduce_max_sync(0xffffffffu, hi);
            o.tile1 = o.q > 0 && o.pos_max >= 0 ? min(in.tiles, o.pos_max / KV_TILE + 1) : 0;
            o.row = (int32_t)in.s;
        }
        o.group = -1;
        if ((threadIdx.x & 31) == 0) entries[p.R + g] = o;
    }
}

int64_t prefix_plan_bytes(int64_t R, int64_t NG, int64_t n_tokens) {
    return 4 * (pf_lengths_at(R, NG, n_tokens) + 2 * R + 1);
}

static cudaError_t launch_chained(const void *kern, int64_t grid, int threads, cudaStream_t s, void **args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

cudaError_t launch_prefix_plan(const int32_t *q_start, const int32_t *kv_len, int64_t R, const int32_t *group_start,
                               const int32_t *prefix_len, int64_t NG, int64_t page, int64_t n_tokens, void *plan, cudaStream_t s) {
    PfPlanArgs a{q_start, kv_len, R, group_start, prefix_len, NG, page, n_tokens, (int32_t *)plan};
    const int64_t most = std::max<int64_t>(std::max(R + 1, n_tokens), 32 * NG);
    void *args[1] = {&a};
    return launch_chained((const void *)prefix_plan_kernel, (most + PF_THREADS - 1) / PF_THREADS + 1, PF_THREADS, s, args);
}

// ---------------------------------------------------------------- join

// a query row's pieces of one entry: the record, then n - 1 slots
struct PfPieces {
    const float *first, *slot;
    int64_t step;
    int n;
    __device__ __forceinline__ const float *at(int i) const { return i == 0 ? first : slot + (i - 1) * step; }
};
// next: what the record says of them; it was written if the entry has queries and tiles
template <int D>
__device__ __forceinline__ PfPieces pf_pieces(const AdShape &a, const AdReq &q, const float *record, float2 next, int64_t t, int head,
                                              int few, int rg) {
    constexpr int64_t RS = PfStride<D>::value;
    PfPieces x{};
    if (q.nt == 0 || t < q.rows0 || t >= (int64_t)q.rows0 + q.q) return x;
    const bool tc = (int64_t)q.q * a.G > few;
    const int rows = tc ? (D == 256 ? 128 : 256) : rg;   // of a unit, a power of two: the prefill kernel's (ApCfg), or rg
    const int in = ((int)(t - q.rows0) * a.G + head % a.G) & (rows - 1);
    // (a kernel that gave up a wait leaves records unwritten: no slot is read that is not there)
    const int slots = tc ? a.pf.pieces : a.pf.parts, slot = min(max(__float_as_int(next.x), 0), slots);
    x.first = record;
    x.n = 1 + min(max(__float_as_int(next.y), 0), slots - slot);
    x.step = rows * RS;
    x.slot = (tc ? a.pieces : a.part) + slot * x.step + in * RS;
    return x;
}

// Pieces a warp takes at a time where query rows are many (more than 16 warps an SM): 4 leave registers for twice the warps,
// 256 requests of 32 heads 10 us, and 14 us with 8.  Where they are few nothing hides a warp's loads but its own: 8.
constexpr int JOIN_MANY = 4;
// Bound: the pieces' bytes, from the L2 mostly, and for few pieces the chain token, entry, pieces.  A warp per query row
// takes AT_ONCE pieces at a time, so that their loads are under way together.
template <int D, int QT, int AT_ONCE>
__global__ void __launch_bounds__(PF_THREADS) prefix_join_kernel(const AdShape a, const int few, const int rg) {
    constexpr int W = D == 64 ? 2 : 4, PL = D / 32 / W;   // values per load, loads per lane
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Attn &p = a.p;
    const int64_t w = ((int64_t)blockIdx.x * PF_THREADS + threadIdx.x) >> 5, t = (uint64_t)w >> 31 ? w / p.h : (int64_t)((uint32_t)w / (uint32_t)p.h);
    const int head = (int)(w - t * p.h), lane = threadIdx.x & 31;
    if (t >= p.n_tokens) return;
    constexpr int64_t RS = PfStride<D>::value;
    const float *own = a.pf.records + (t * p.h + head) * RS, *shared = own + p.n_tokens * p.h * RS;
    const float2 own_next = *reinterpret_cast<const float2 *>(own + D + 2), shared_next = *reinterpret_cast<const float2 *>(shared + D + 2);
    const int2 at_rg = pf_unpack(pf_token(a.pf, t).y);
    if (!pf_plan_fits(a)) {
        if (w == 0 && lane == 0 && p.status != nullptr) atomicAdd(p.status, 1);
        return;
    }
    const int r = at_rg.x, ge = (int)p.R + at_rg.y;
    if (r < 0 || r >= p.R) return;
    const bool grouped = ge >= p.R && ge < a.pf.n_entries;
    const AdReq q0 = pf_request(a, r), q1 = pf_request(a, grouped ? ge : r);
    if (t - q0.rows0 >= q0.q) return;   // past the request's max_q first queries
    PfPieces x[2];
    x[0] = pf_pieces<D>(a, q0, own, own_next, t, head, few, rg);
    x[1] = PfPieces{};
    if (grouped) x[1] = pf_pieces<D>(a, q1, shared, shared_next, t, head, few, rg);
    const int n = x[0].n + x[1].n;
    float mx = -INFINITY, l = 0.0f, v[PL * W];
#pragma unroll
    for (int i = 0; i < PL * W; i++) v[i] = 0.0f;
    for (int i0 = 0; i0 < n; i0 += AT_ONCE) {
        float2 ml[AT_ONCE];
        float u[AT_ONCE][PL * W];
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) {
            const int k = i0 + i;
            ml[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int c = 0; c < PL * W; c++) u[i][c] = 0.0f;
            if (k < n) {
                const float *src = k < x[0].n ? x[0].at(k) : x[1].at(k - x[0].n);
                ml[i] = *reinterpret_cast<const float2 *>(src + D);
#pragma unroll
                for (int c = 0; c < PL; c++) {
                    if constexpr (W == 4) *reinterpret_cast<float4 *>(&u[i][4 * c]) = *reinterpret_cast<const float4 *>(src + 4 * lane + 128 * c);
                    else *reinterpret_cast<float2 *>(&u[i][0]) = *reinterpret_cast<const float2 *>(src + 2 * lane);
                }
            }
        }
        float mn = mx;
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) mn = fmaxf(mn, ml[i].x);
        const float base = mn == -INFINITY ? 0.0f : mn, f0 = ex2(mx - base);
        mx = mn;
        l *= f0;
#pragma unroll
        for (int c = 0; c < PL * W; c++) v[c] *= f0;
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) {
            const float f = ex2(ml[i].x - base);
            l = fmaf(f, ml[i].y, l);
#pragma unroll
            for (int c = 0; c < PL * W; c++) v[c] = fmaf(f, u[i][c], v[c]);
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t at = t * p.ldo + (int64_t)head * D + W * lane;
#pragma unroll
    for (int c = 0; c < PL; c++) {
        float u[W];
#pragma unroll
        for (int i = 0; i < W; i++) u[i] = l == 0.0f ? 0.0f : v[W * c + i] * inv;
        if constexpr (W == 4) store4<QT>(p.out, at + 128 * c, a.vec, u[0], u[1], u[2], u[3]);
        else
#pragma unroll
            for (int i = 0; i < W; i++) store_out(p.out, QT, at + i, u[i]);
    }
}

template <int D, int AT_ONCE>
static const void *join_kernel(int qt) {
    return qt == GGUF_F32 ? (const void *)prefix_join_kernel<D, GGUF_F32, AT_ONCE>
         : qt == GGUF_F16 ? (const void *)prefix_join_kernel<D, GGUF_F16, AT_ONCE> : (const void *)prefix_join_kernel<D, GGUF_BF16, AT_ONCE>;
}
template <int D>
static const void *join_kernel(int qt, bool many) { return many ? join_kernel<D, JOIN_MANY>(qt) : join_kernel<D, 8>(qt); }

// ---------------------------------------------------------------- what a call runs

struct PfRun {
    bool alone;        // the requests go one by one, through the kernels of gguf_paged_attention
    int ctas;
    bool tc;           // the tensor-core kernel runs
    int few, rg;       // entries of at most `few` query rows per KV head, in units of rg rows, go to the other one
    size_t part, pieces, bytes;   // offsets in the workspace behind the records, and its size
};
static PfRun prefix_run(const Attn &p, int64_t NG, int64_t d) {
    PfRun x{};
    x.ctas = std::min(device_info().sm_count, 1024);
    const int64_t G = p.h / p.hk;
    // Units of 16 rows where a request alone has more than 8 (heads of 256 and fp32 queries have no such units).  The
    // tensor-core kernel takes what is more than a unit: 2800 cycles for 128 tokens and up to 128 rows, against 1500 for
    // each 8 rows and 2100 for each 16.
    x.rg = p.qt != GGUF_F32 && d != 256 && G * p.max_q > 8 ? 16 : 8;
    x.tc = p.qt != GGUF_F32 && p.n_tokens * G > x.rg;
    x.few = x.tc ? x.rg : 0x7fffffff;
    // Sharing has a price, the launches, starts and joins of its kernels: about 33 us in all (45 with heads of 256; 20 us for
    // fp32 queries, which one kernel takes).  What the requests cost one by one, 10 us and 0.42 ns a tile of heads of 128 (more
    // for 16 rows and for fp32 queries), is known up to the width of the table and of the window: where that is less, they go
    // so, as they do where there are no two requests of a group.  Measured without the plan, one by one and shared: 2 x (700 +
    // 60) tokens, fp32, 8 KV heads of 128: 12.9 and 18.2 us; 38 requests of 6 groups, 5300 tokens, 2 of 256: 35 and 42 us; 8 KV
    // heads of 128, 16 x (8192 + 200): 41 and 34 us; 32 x (8192 + 512): 69 and 39 us; 64 x (32768 + 200) with a window of 1024:
    // 31 and 38 us; 64 x (16384 + 200) with one of 4096, 8 of 64: 47 and 36 us; 256 x (32768 + 128): 1690 and 183 us.
    const int64_t rows = G * std::min(p.max_q, p.n_tokens);
    const int64_t most = p.window > 0 ? std::min(p.width * p.page, p.window + p.sinks + p.max_q + 3 * KV_TILE) : p.width * p.page;
    const double tiles = (double)p.R * (double)p.hk * (double)((rows + x.rg - 1) / x.rg) * (double)(most / KV_TILE);
    const double us = 10.0 + tiles * 0.42e-3 * (double)d / 128.0 * (x.rg == 16 ? 1.4 : 1.0) * (p.qt == GGUF_F32 ? 1.9 : 1.0);
    // (one by one a request's units of 8 rows x tiles are counted in 32 bits; 16-bit queries have at most 64 rows in units)
    const int64_t unit_rows = p.qt == GGUF_F32 ? rows : std::min<int64_t>(rows, 64);
    const bool counted = (double)p.hk * (double)((unit_rows + 7) / 8) * (double)pf_most_tiles(p) <= 4.0e9;
    x.alone = counted && (NG == 0 || p.R < 2 || us < (!x.tc ? 20.0 : d == 256 ? 45.0 : 33.0));
    if (x.alone) {
        x.bytes = attn_ws_size(p, d);
        return x;
    }
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    const size_t rs = (size_t)(d + 4) * 4;
    x.part = up(2 * (size_t)p.n_tokens * p.h * rs);
    x.pieces = up(x.part + (size_t)x.ctas * ad_warps((int)d, p.qt == GGUF_F32, x.rg / 8) * x.rg * rs);
    x.bytes = x.tc ? x.pieces + (size_t)x.ctas * (d == 256 ? 128 : 256) * rs : x.pieces;
    return x;
}

size_t prefix_attn_ws_size(const Attn &p, int64_t NG, int64_t d) { return prefix_run(p, NG, d).bytes; }

cudaError_t launch_prefix_attn(const Attn &p, const void *plan, int64_t NG, int64_t d, void *ws, cudaStream_t s) {
    const PfRun x = prefix_run(p, NG, d);
    const int64_t es = p.qt == GGUF_F32 ? 4 : 2;
    if (x.alone) {
        Attn one = p;
        one.q_start = (const int32_t *)plan + pf_lengths_at(p.R, NG, p.n_tokens);
        one.kv_len = one.q_start + p.R + 1;
        return launch_attn(one, d, ws, s, (const int32_t *)plan, p.R + NG);
    }
    uint8_t *w = (uint8_t *)ws;
    AdShape a{};
    a.p = p;
    a.err = tg_error_word();
    auto shift_of = [](int32_t v) { return (v & (v - 1)) == 0 ? __builtin_ctz(v) : -1; };
    a.G = (int32_t)(p.h / p.hk);
    a.hk = (int32_t)p.hk;
    a.G_shift = shift_of(a.G);
    a.tpp = (int32_t)(p.page / KV_TILE);
    a.tpp_shift = shift_of(a.tpp);
    a.page_bytes = kv_page_bytes(d, p.hk, p.page);
    a.vec = (reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.out)) % 16 == 0 && p.ldq * es % 16 == 0 &&
            p.ldo * es % 16 == 0;
    a.part = (float *)(w + x.part);
    a.pieces = (float *)(w + x.pieces);
    a.pf = PfShape{(const int32_t *)plan, (int32_t)(p.R + NG), x.tc, x.ctas * ad_warps((int)d, p.qt == GGUF_F32, x.rg / 8), x.ctas,
                   pf_most_tiles(p), (float *)ws};
    a.min_rows = x.few;
    a.max_rows = 0x7fffffff;
    if (x.tc) {
        const cudaError_t e = d == 64 ? launch_prefix_prefill_64(a, x.ctas, s)
                            : d == 128 ? launch_prefix_prefill_128(a, x.ctas, s) : launch_prefix_prefill_256(a, x.ctas, s);
        if (e != cudaSuccess) return e;
    }
    a.min_rows = 0;
    a.max_rows = x.few;
    const cudaError_t e = d == 64 ? launch_prefix_decode_64(a, x.rg / 8, x.ctas, s)
                        : d == 128 ? launch_prefix_decode_128(a, x.rg / 8, x.ctas, s) : launch_prefix_decode_256(a, x.rg / 8, x.ctas, s);
    if (e != cudaSuccess) return e;
    a.max_rows = 0x7fffffff;   // the join looks at all entries
    int few = x.few, rg = x.rg;
    void *args[3] = {&a, &few, &rg};
    const bool many = p.n_tokens * p.h > 16 * device_info().sm_count;
    return launch_chained(d == 64 ? join_kernel<64>(p.qt, many) : d == 128 ? join_kernel<128>(p.qt, many) : join_kernel<256>(p.qt, many),
                          (p.n_tokens * p.h + PF_THREADS / 32 - 1) / (PF_THREADS / 32), PF_THREADS, s, args);
}

}  // namespace gg
