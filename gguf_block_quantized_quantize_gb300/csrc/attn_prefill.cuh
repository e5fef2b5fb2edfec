// Attention of many query rows over the paged Q4_0 cache (prompts and chunks of
// prompts) on the tcgen05 tensor cores, for bf16 and fp16 queries.
//
// Bound: the fp16 matrix rate (4 D operations per query head and visible
// token).  A CTA takes up to RT x 128 query rows of one KV head (row = token *
// group + head of the group, so grouped heads share every key) and walks over
// the tokens that they see in blocks of BT:
//   S = Q K^T   A = Q, B = K, both fp16 in shared memory (128-byte swizzle),
//               S in TMEM; two S buffers, so that one is computed while the
//               softmax works on the other
//   O += P V    A = P (fp16, in TMEM, over the columns of its S), B = V^T in
//               shared memory, O in TMEM
// The packed tiles of a block come by bulk copies; four warps turn them into
// fp16 operands (k, v = d * (c - 8), rounded to 2^-12 of them at most; for fp16
// queries k exactly, in two parts) once for all rows of the CTA.  bf16 queries
// are scaled per row by a power of two into fp16's range.  The softmax keeps a
// reference maximum per row and rescales O only when a score exceeds it by 2^5:
// probabilities are held as 2^(s - reference + 10), at most 2^15.  Statistics
// are fp32.
//
// Warps: 0-3 and 4-7 the softmax of a row tile each (TMEM lanes 32 * (warp %
// 4) on; a thread holds its row's scores of a block, so these warps take
// registers from the others), 8-11 unpack, 12 issues the MMAs (and owns the
// TMEM allocation), 13 loads.  Every wait is bounded (1 s); a timeout sets the
// error word and the CTA drains and exits.
//
// Measured: a prompt of 8192 tokens, 32 query heads, 8 KV heads of 128, bf16: 648
// us, 0.85 PFLOP/s (0.45 of the matrix rate); with heads of 256 1690 us (0.34);
// 2 x 4093 tokens with a window of 1000, heads of 64, fp16: 154 us (0.27 PFLOP/s).
// What bounds it now: no unit (tensor pipe 37 % active, issue slots 45 % used at
// heads of 128) but the chain scores, softmax, P, product of an S buffer, which
// the next scores into it wait for: 4800 cycles per block and two row tiles, and
// 4300 with heads of 64.  TMEM is full with heads of 128 only (two S buffers and O);
// with heads of 64 and of 256 128 of its columns are unused (384 on, and 128 to 255).
// Spills a thread: at most 76 bytes of stores and 64 of loads without CUT; with it
// 216 / 228 with heads of 128, 108 / 128 of 64, none of 256.
#pragma once

#include "attn_decode.cuh"

namespace gg {

constexpr int AP_UW = 4;                         // warps that unpack
constexpr int AP_THREADS = (12 + AP_UW) * 32;
constexpr int AP_MMA = 8 + AP_UW, AP_LOAD = 9 + AP_UW;

template <int D, int QT>
struct ApCfg {
    static constexpr int RT = D == 256 ? 1 : 2;        // row tiles of 128 (the O accumulators fill the TMEM)
    static constexpr int BT = D == 256 ? 64 : 128;     // tokens per block
    // fp16 results keep more bits than keys rounded to fp16 leave in the scores (error 4.8e-4 of the outputs' norm; an
    // output rounded once has 2.1e-4): for them keys are held in two parts, exactly, and scores are two products (3.0e-4;
    // 146 -> 153 us at 2048 tokens of heads of 64, 644 -> 766 us at 8192 of heads of 128).  In bf16 results it is lost.
    static constexpr int KP = QT == GGUF_F16 ? 2 : 1;
    static constexpr int KST = D > 64 && KP == 2 ? 1 : 2, VST = 2;   // as the shared memory allows
    static constexpr int GT = BT / KV_TILE;            // cache tiles of a block; a load is their keys, or their values
    static constexpr int RAWST = D == 64 ? 6 : 3;
    // registers of the softmax warps (a row's scores) and of the others (packed words read ahead): 256 for the two, as at
    // launch
    static constexpr int REGS = D == 256 ? 120 : 176, REGS_OTHER = 256 - REGS;
    static constexpr int PITCH = 9 * D + 16;           // half tiles apart by an odd number of 16-byte banks
    static constexpr int Q_BYTES = RT * 128 * D * 2;
    static constexpr int K_PART = BT * D * 2, K_BYTES = KP * K_PART, V_BYTES = BT * D * 2;
    static constexpr int RAW_BYTES = GT * PITCH;
    static constexpr int OFF_K = Q_BYTES, OFF_V = OFF_K + KST * K_BYTES, OFF_RAW = OFF_V + VST * V_BYTES;
    static constexpr int SMEM = OFF_RAW + RAWST * RAW_BYTES + 1024;   // 1024 for the base's alignment
    static constexpr int COL_S = BT, COL_O = 256;      // TMEM columns: S buffer x at x * BT, O of row tile t at 256 + t * D
    static_assert(SMEM <= 232448 - 6144, "static shared memory fits beside");
};

// a CTA's piece of work
struct ApItem {
    int r, head, row0, rows;      // request, KV head, first query row and rows (of token * G + head)
    int q0, pos0;                 // the request's first query token, position of row row0's token
    int tok0;                     // row0 / G
    int nt, n_sink, w_tile;       // the tiles that the rows see (see AdReq): the piece takes those from base to nt
    int base;
    int part;                     // its place among the partial results where the row block's tiles are cut, else -1
};

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// pairs of fp32 values in 64-bit registers, and two operations at once on them
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint64_t fma_2(uint64_t x, uint64_t m, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(m), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

template <int N>
__device__ __forceinline__ void set_registers() {   // from 128 at launch
    if constexpr (N > 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// true in one lane of the warp
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// row blocks (of `rows` query rows) x KV heads of one request
__device__ __forceinline__ int ap_items(const AdShape &a, const AdReq &q, int rows) {
    return (int)((q.q * (int64_t)a.G + rows - 1) / rows) * a.hk;
}

// whether `tile` is the first of its page that the request's queries see, and no row block before this one sees it
__device__ __forceinline__ bool ap_first_sight(const AdShape &a, const ApItem &w, int tile) {
    const AdReq q = ad_request(a, w.r);
    if (w.row0 > 0) {
        const int before = q.pos0 + (w.row0 - 1) / a.G;   // the position of the row before
        if (before >= 0 && tile <= before / KV_TILE) return false;
    }
    return ad_starts_page(a, q, tile < q.n_sink ? tile : tile - q.w_tile + q.n_sink);
}

template <int D, int QT, bool CUT>
__global__ void __launch_bounds__(AP_THREADS, 1) attn_prefill_kernel(const AdShape a) {
    using C = ApCfg<D, QT>;
    using L = KvTile<D>;
    constexpr int NB = L::NB, BW = L::BW, NC = L::NC, BT = C::BT, ROWS = C::RT * 128;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t raw_full[C::RAWST], raw_empty[C::RAWST], k_full[C::KST], k_empty[C::KST], v_full[C::VST],
        v_empty[C::VST], s_full[2], p_full[2], pv_done[2], q_full, drain;
    __shared__ int32_t raw_mask[C::RAWST], blk_mask[8];
    __shared__ float q_inv[ROWS];
    __shared__ uint32_t tmem_slot;
    __shared__ int32_t abort_word;
    __shared__ ApItem item;
    __shared__ int32_t part[2][AP_THREADS / 32], cut_rows, cut_pieces, cut_from;
    __shared__ int32_t chunk_end[AP_THREADS];   // at most (tokens x heads / 128) items: 31 bits
    volatile int32_t *abort_flag = &abort_word;
    const Attn &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.G;
    if (tid == 0) {
        for (int i = 0; i < C::RAWST; i++) { tc::mbar_init(&raw_full[i], 1); tc::mbar_init(&raw_empty[i], AP_UW); }
        for (int i = 0; i < C::KST; i++) { tc::mbar_init(&k_full[i], AP_UW); tc::mbar_init(&k_empty[i], 1); }
        for (int i = 0; i < C::VST; i++) { tc::mbar_init(&v_full[i], AP_UW); tc::mbar_init(&v_empty[i], 1); }
        for (int i = 0; i < 2; i++) { tc::mbar_init(&s_full[i], 1); tc::mbar_init(&p_full[i], 4); tc::mbar_init(&pv_done[i], 1); }
        tc::mbar_init(&q_full, 8);
        tc::mbar_init(&drain, 1);
        tc::fence_barrier_init();
        abort_word = 0;
    }
    if (warp == AP_MMA) {
        tc::tmem_alloc(&tmem_slot, 512);
        tc::tmem_relinquish();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Work of all requests: thread t counts requests [t * per, (t + 1) * per), in row blocks of ROWS rows, and of 128.
    // The larger ones unpack a key for twice the rows; the smaller ones are for calls that would leave SMs idle, as are
    // row blocks whose tokens are cut into pieces (CUT; of 4 blocks at least, joined by a second launch).
    const int R = (int)p.R, per = (R + AP_THREADS - 1) / AP_THREADS;
    {
        int item_rows = ROWS, splits = 1;
        int mine = 0, mine128 = 0;   // (tokens x heads / 128 is below 2^31)
        for (int r = tid * per; r < min(R, (tid + 1) * per); r++) {
            const AdReq q = ad_request(a, r);
            mine += ap_items(a, q, ROWS);
            mine128 += ap_items(a, q, 128);
        }
        int incl = mine, incl128 = mine128;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o), w = __shfl_up_sync(0xffffffffu, incl128, o);
            if (lane >= o) { incl += v; incl128 += w; }
        }
        if (lane == 31) { part[0][warp] = incl; part[1][warp] = incl128; }
        tc::tc_fence_before();
        __syncthreads();
        tc::tc_fence_after();
        int all = 0, all128 = 0;
        for (int w = 0; w < AP_THREADS / 32; w++) {
            if (w < warp) { incl += part[0][w]; incl128 += part[1][w]; }
            all += part[0][w];
            all128 += part[1][w];
        }
        if (all128 <= (int)gridDim.x) {   // (two rounds of the smaller ones would take longer than one of the larger)
            item_rows = 128;
            incl = incl128;
            mine = mine128;
            all = all128;
        }
        // the row blocks after the last full round are cut where that gives every CTA at most one piece
        const int rest = all % (int)gridDim.x;
        if (CUT && rest > 0) splits = max(1, min(a.max_splits, (int)gridDim.x / rest));
        const int from = splits > 1 ? all - rest : all;
        chunk_end[tid] = incl;
        if (tid == 0) { cut_rows = item_rows; if (CUT) { cut_pieces = splits; cut_from = from; } }
        if (CUT && blockIdx.x == 0) {   // for the join: the items before each request, and the cut
            int before = incl - mine;
            for (int r = tid * per; r < min(R, (tid + 1) * per); r++) {
                a.item_base[r] = before;
                before += ap_items(a, ad_request(a, r), item_rows);
            }
            if (tid == 0) { a.item_base[R] = item_rows; a.item_base[R + 1] = splits; a.item_base[R + 2] = from; }
        }
        __syncthreads();
    }
    const int64_t total = CUT ? cut_from + (int64_t)(chunk_end[AP_THREADS - 1] - cut_from) * cut_pieces : chunk_end[AP_THREADS - 1];
    const uint32_t tmem = tmem_slot;
    auto fail = [&](int code) {
        *abort_flag = 1;
        if (a.err != nullptr) atomicOr(a.err, code);
    };
    // one arrival for the warp, once all its lanes have come here (256 single ones take as many turns at the barrier)
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar);
    };
    auto token_of = [&](int i) { return (i < item.n_sink ? i : item.w_tile + i - item.n_sink) * KV_TILE; };

    // items in stripes of one per CTA, every other stripe backwards: a request's row blocks come longest first
    const int64_t stripes = (total + gridDim.x - 1) / gridDim.x;
    auto item_of = [&](int64_t stripe) { return stripe * gridDim.x + ((stripe & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x); };
    auto everyone = [] { asm volatile("bar.sync 0, %0;" ::"n"(AP_THREADS) : "memory"); };
    // what a role knows of the current item, and the running uses of the stages and of the S buffers before it
    struct Walk {
        int blocks_before = 0, loads_before = 0, uses[2] = {0, 0}, nrt = 0, nblk = 0, nitems = 0, items = -1;
    };
    // the item before is done with (its shared and tensor memory are free), and the next one is known
    auto begin = [&](Walk &wk, int64_t piece) {
        wk.blocks_before += wk.nblk;
        wk.loads_before += 2 * wk.nblk;
        wk.uses[0] += (wk.nitems + 1) / 2;
        wk.uses[1] += wk.nitems / 2;
        wk.items++;
        tc::tc_fence_before();
        everyone();
        tc::tc_fence_after();
        if (*abort_flag) return false;
        if (tid == 0) {
            const int item_rows = cut_rows, splits = CUT ? cut_pieces : 1;
            const int place = CUT ? (int)piece - cut_from : -1;   // among the pieces of the cut ones
            const int it = place >= 0 ? cut_from + place / splits : (int)piece, cut = place % splits;
            int lo = -1, hi = AP_THREADS - 1;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (chunk_end[mid] > it) hi = mid;
                else lo = mid;
            }
            int before = hi > 0 ? chunk_end[hi - 1] : 0;
            ApItem w;
            AdReq q;
            for (w.r = hi * per;; w.r++) {   // it is there: it < total
                q = ad_request(a, w.r);
                const int n = ap_items(a, q, item_rows);
                if (before + n > it) break;
                before += n;
            }
            const int rows = q.q * G, nblk = (rows + item_rows - 1) / item_rows;
            w.head = (it - before) % a.hk;
            w.row0 = (nblk - 1 - (it - before) / a.hk) * item_rows;
            w.rows = min(item_rows, rows - w.row0);
            w.q0 = q.rows0;
            w.tok0 = w.row0 / G;
            w.pos0 = q.pos0 + w.tok0;
            const int last = q.pos0 + (w.row0 + w.rows - 1) / G;
            w.nt = w.n_sink = w.w_tile = 0;
            if (last >= 0) {
                const int end = last / KV_TILE + 1;
                w.nt = end;
                if (p.window > 0) {
                    const int64_t w0 = (int64_t)w.pos0 - p.window + 1;
                    w.w_tile = w0 > 0 ? (int)(w0 / KV_TILE) : 0;
                    w.n_sink = (int)min((p.sinks + KV_TILE - 1) / KV_TILE, (int64_t)w.w_tile);
                    w.nt = w.n_sink + end - w.w_tile;
                }
            }
            // the blocks of the row block, shared out over the pieces
            if (CUT) {
                w.base = 0;
                w.part = place;
                if (place >= 0) {
                    const int64_t blocks = (w.nt + BT / KV_TILE - 1) / (BT / KV_TILE);
                    w.base = (int)(blocks * cut / splits) * (BT / KV_TILE);
                    w.nt = min(w.nt, (int)(blocks * (cut + 1) / splits) * (BT / KV_TILE));
                }
            }
            item = w;
        }
        everyone();
        wk.nrt = item.rows > 128 ? 2 : 1;
        wk.nblk = (item.nt - (CUT ? item.base : 0) + BT / KV_TILE - 1) / (BT / KV_TILE);
        wk.nitems = wk.nblk * wk.nrt;
        return true;
    };
    Walk wk;
    if (warp < 8) {
        set_registers<C::REGS>();
        for (int64_t st = 0; st < stripes; st++) {
            const int64_t it = item_of(st);
            if (it >= total) continue;
            if (!begin(wk, it)) break;
            // ---- queries: D / 8 lanes per row, 8 values each
            {
                constexpr int LPR = D / 8;
                for (int row = tid / LPR; row < ROWS; row += 256 / LPR) {
                    const int l = tid % LPR, rr = item.row0 + row;
                    uint32_t w[4] = {0, 0, 0, 0};
                    if (row < item.rows) {
                        const uint16_t *src = reinterpret_cast<const uint16_t *>(p.q) + (item.q0 + rr / G) * p.ldq +
                                              (int64_t)(item.head * G + rr % G) * D + 8 * l;
                        if (a.vec) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(src);
                            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; i++) w[i] = src[2 * i] | (uint32_t)src[2 * i + 1] << 16;
                        }
                    }
                    if constexpr (QT == GGUF_BF16) {
                        float v[8], mx = 0.0f;
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            v[i] = bf2f((uint16_t)(w[i / 2] >> (16 * (i & 1))));
                            mx = fmaxf(mx, fabsf(v[i]));
                        }
                        // a row's lanes lie in one warp and all of them are here (256 / LPR divides ROWS)
#pragma unroll
                        for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const float up = q_scale_up(mx);
#pragma unroll
                        for (int i = 0; i < 4; i++) w[i] = pack_h2(v[2 * i] * up, v[2 * i + 1] * up);
                        if (l == 0) q_inv[row] = 1.0f / up;
                    } else if (l == 0) q_inv[row] = 1.0f;
                    const int tile = row / 128, r7 = row % 128;
                    *reinterpret_cast<uint4 *>(smem + tile * (128 * D * 2) + (8 * l / 64) * 16384 + r7 * 128 +
                                               (((l & 7) ^ (r7 & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                tc::fence_proxy_async_smem();
                arrive(&q_full);
            }
            // ================= softmax
            const int t = warp >> 2;
            if (t < wk.nrt && t < C::RT) {
                const int quad = warp & 3;
                const int row = t * 128 + quad * 32 + lane;
                const uint32_t lanes = (uint32_t)(quad * 32) << 16;
                const uint32_t o_col = tmem + lanes + C::COL_O + t * D;
                const bool there = row < item.rows;
                const int pos = there ? item.pos0 + (item.row0 + row) / G - item.tok0 : -1;
                // positions of the warp's rows, from the first to the last that is there
                const int first = item.pos0 + (item.row0 + t * 128 + quad * 32) / G - item.tok0;
                const int lastr = min(item.rows - 1, t * 128 + quad * 32 + 31);
                const int last = item.pos0 + (item.row0 + lastr) / G - item.tok0;
                float ref = -INFINITY, lsum = 0.0f;
                bool ok = __all_sync(0xffffffffu, tc::mbar_wait(&q_full, (uint32_t)wk.items & 1u));
                if (!ok && lane == 0) fail(1);
                const float sl = p.scale * 1.44269504088896341f * q_inv[row];
                for (int j = 0; j < wk.nblk && ok; j++) {
                    const int n = j * wk.nrt + t, x = n & 1;
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&s_full[x], (uint32_t)(wk.uses[x] + n / 2) & 1u)) && !*abort_flag;
                    if (!ok) { if (lane == 0) fail(2); break; }
                    tc::tc_fence_after();
                    const uint32_t s_col = tmem + lanes + x * C::COL_S;
                    // whether every row of the warp sees the whole block
                    const int i0 = (CUT ? item.base : 0) + j * (BT / KV_TILE), i1 = min(item.nt, i0 + BT / KV_TILE);
                    const int mask = blk_mask[(wk.blocks_before + j) & 7];
                    const int t_first = i0 < item.n_sink ? 0 : token_of(i0), t_last = token_of(i1 - 1) + KV_TILE - 1;
                    const bool whole = mask == (1 << (BT / KV_TILE)) - 1 && t_last <= first &&
                                       (p.window <= 0 || t_first > last - p.window || t_last < p.sinks);
                    uint32_t rr[BT / 32][32];   // the row's scores
#pragma unroll
                    for (int c = 0; c < BT / 32; c++) tc::tmem_ld_32x32b_x32(s_col + 32 * c, rr[c]);
                    tc::tmem_ld_wait();
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < BT / KV_TILE; i++) {
                            const int tok = token_of(i0 + i);
                            // seen: tok + e <= pos, and tok + e > pos - window or tok + e < sinks
                            const int hi = (mask >> i) & 1 ? min(pos - tok, 15) : -1;
                            const int lo = p.window > 0 ? (int)min(max((int64_t)pos - p.window - tok, (int64_t)-1), (int64_t)15) : -1;
                            const int sk = (int)min(max(p.sinks - tok, (int64_t)0), (int64_t)KV_TILE);
                            const uint32_t back = lo < 0 ? 0u : (2u << lo) - 1;   // too far back
                            const uint32_t seen = hi < 0 ? 0u : ((2u << hi) - 1) & (~back | ((1u << sk) - 1));
#pragma unroll
                            for (int e = 0; e < KV_TILE; e++)
                                if (!(seen & (1u << e))) rr[i / 2][16 * (i & 1) + e] = 0xff800000u;   // -inf
                        }
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < BT / 32; c++)
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
#pragma unroll
                            for (int u = 0; u < 4; u++)
                                m4[u] = fmaxf(m4[u], fmaxf(__uint_as_float(rr[c][i + 2 * u]), __uint_as_float(rr[c][i + 2 * u + 1])));
                    float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    mx *= sl;
                    float alpha = 1.0f;
                    if (mx > ref + 5.0f) {
                        alpha = ex2(ref - mx);   // 0 from -inf
                        ref = mx;
                        lsum *= alpha;
                    }
                    if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
                        // O of the blocks before is complete once their last product is
                        const int np = n - wk.nrt, xp = np & 1;
                        ok = __all_sync(0xffffffffu, tc::mbar_wait(&pv_done[xp], (uint32_t)(wk.uses[xp] + np / 2) & 1u));
                        if (!ok) { if (lane == 0) fail(2); break; }
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 16; c++) {   // few at a time: the scores are in registers
                            uint32_t v[16];
                            tmem_ld_x16(o_col + 16 * c, v);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; i++) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                            tmem_st_x16(o_col + 16 * c, v);
                        }
                        tc::tmem_st_wait();
                    }
                    const float base = ref == -INFINITY ? 0.0f : AD_PBITS - ref;
                    const uint64_t sl2 = pair(sl, sl), base2 = pair(base, base);
                    uint64_t l2[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < BT / 32; c++) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; i++) {
                            float2 v = unpair(fma_2(pair(__uint_as_float(rr[c][2 * i]), __uint_as_float(rr[c][2 * i + 1])), sl2, base2));
                            v.x = ex2(v.x);
                            v.y = ex2(v.y);
                            l2[i & 3] = add_2(l2[i & 3], pair(v.x, v.y));
                            pk[i] = pack_h2(v.x, v.y);
                        }
                        tmem_st_x16(s_col + 16 * c, pk);   // over scores, which are in registers by now
                    }
                    const float2 ls = unpair(add_2(add_2(l2[0], l2[1]), add_2(l2[2], l2[3])));
                    lsum += ls.x + ls.y;
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    arrive(&p_full[x]);
                }
                // ---- the output rows
                if (ok && wk.nblk > 0) {
                    const int np = wk.nitems - wk.nrt + t, xp = np & 1;
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&pv_done[xp], (uint32_t)(wk.uses[xp] + np / 2) & 1u));
                    if (!ok && lane == 0) fail(8);
                    tc::tc_fence_after();
                }
                if (ok) {
                    const float inv = lsum == 0.0f ? 0.0f : 1.0f / lsum;
                    const int rr0 = item.row0 + row;
                    const int64_t at = (item.q0 + rr0 / G) * p.ldo + (int64_t)(item.head * G + rr0 % G) * D;
#pragma unroll 1
                    for (int c = 0; c < D / 32; c++) {
                        uint32_t rr[32];
                        if (wk.nblk > 0) {
                            tc::tmem_ld_32x32b_x32(o_col + 32 * c, rr);
                            tc::tmem_ld_wait();
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i++) rr[i] = 0;
                        }
                        if (CUT && there && item.part >= 0) {
                            float *to = a.pieces + ((int64_t)item.part * cut_rows + row) * (D + 2);
                            float2 *dst = reinterpret_cast<float2 *>(to + 2 + 32 * c);
#pragma unroll
                            for (int i = 0; i < 16; i++) dst[i] = make_float2(__uint_as_float(rr[2 * i]), __uint_as_float(rr[2 * i + 1]));
                            if (c == 0) *reinterpret_cast<float2 *>(to) = make_float2(ref, lsum);
                        } else if (there) {
                            uint16_t *out = reinterpret_cast<uint16_t *>(p.out) + at + 32 * c;
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; i++) {
                                const float f0 = lsum == 0.0f ? 0.0f : __uint_as_float(rr[2 * i]) * inv;
                                const float f1 = lsum == 0.0f ? 0.0f : __uint_as_float(rr[2 * i + 1]) * inv;
                                w[i] = QT == GGUF_BF16 ? f2bf_rn(f0) | (uint32_t)f2bf_rn(f1) << 16
                                                       : f2h_rn(f0) | (uint32_t)f2h_rn(f1) << 16;
                            }
                            if (a.vec) {
#pragma unroll
                                for (int i = 0; i < 4; i++)
                                    reinterpret_cast<uint4 *>(out)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                            } else {
#pragma unroll
                                for (int i = 0; i < 16; i++) { out[2 * i] = (uint16_t)w[i]; out[2 * i + 1] = (uint16_t)(w[i] >> 16); }
                            }
                        }
                    }
                    tc::tc_fence_before();
                }
            }
        }
    } else if (warp < AP_MMA) {
        set_registers<C::REGS_OTHER>();
        for (int64_t st = 0; st < stripes; st++) {
            const int64_t it = item_of(st);
            if (it >= total) continue;
            if (!begin(wk, it)) break;
            // ================= unpack: the keys of a block, then its values, 4 tiles a step.  The packed words of the next step are
            // read from shared memory before the current one is computed: the matrix unit's reads fill the shared memory's
            // bandwidth for long stretches, and a read may take many hundred cycles.
            // Keys: warp w8 takes tile w8 of a step; lane (g, q) holds values 8 q .. of the blocks of tokens g and g + 8; odd g
            // takes the blocks in another order, so that the stores of a warp hit different banks.
            // Values: lane (tile, p, gs) holds 8 tokens (one 16-byte chunk of a row of V^T) of 4 values of half of the
            // blocks; the tiles' pitch and the other eighth at odd p keep loads and stores off each other's banks.
            constexpr int XS = NB / 2;
            const int w8 = warp - 8;
            const int kg = lane >> 2, kq = lane & 3, odd = kg & 1;
            const int tl = lane & 3, pp = (lane >> 2) & 1, hb = w8 >> 1, vg = 2 * (lane >> 3) + (pp ^ (w8 & 1));
            const uint32_t k_off = (w8 * 16 + kg) * 128 + (((4 * odd + kq) ^ kg) * 16);   // of even blocks; odd ones: ^ 64
            const uint32_t v_cx = ((2 * tl + pp) ^ (4 * (vg & 1))) * 16, v_row = (32 * XS * hb + 4 * vg) * 128;
            const uint8_t *raws = smem + C::OFF_RAW;
            const int last = item.pos0 + (item.row0 + item.rows - 1) / G - item.tok0 - 8 * pp;
            const int n_sink = item.n_sink, w_tile = item.w_tile, i_base = CUT ? item.base : 0;
            bool ok = true;
            constexpr int STEPS = C::GT / 4;
            auto raw_wait = [&](int load) {
                const int gb = wk.loads_before + load;
                ok = ok && tc::mbar_wait(&raw_full[gb % C::RAWST], (uint32_t)(gb / C::RAWST) & 1u);
                return gb % C::RAWST;
            };
            struct Keys { uint32_t w[2][NB], d[2][NB]; bool live; };
            struct Values { uint32_t w[4][XS], d[4][XS]; int end; };   // end: last token of the 8 that counts
            auto load_keys = [&](int rs, int step, Keys &x) {
                const uint8_t *raw = raws + rs * C::RAW_BYTES + (4 * step + w8) * C::PITCH;
                x.live = (raw_mask[rs] >> (4 * step + w8)) & 1;
#pragma unroll
                for (int e = 0; e < 2; e++) {
#pragma unroll
                    for (int c = 0; c < NC; c++) {
                        lds_words<BW>(raw + 4 * ((e * NC + c) * 32 + lane) * BW, *reinterpret_cast<uint32_t(*)[BW]>(&x.w[e][c * BW]));
                        lds_words<BW>(raw + L::KS + 4 * ((4 * e + (kg >> 1)) * NB + c * BW), *reinterpret_cast<uint32_t(*)[BW]>(&x.d[e][c * BW]));
                    }
                }
            };
            auto put_keys = [&](uint8_t *sk, int step, const Keys &x) {
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    uint8_t *to = sk + (step * 64 + e * 8) * 128;
#pragma unroll
                    for (int i = 0; i < NB; i++) {   // block i ^ odd
                        const uint32_t w = odd ? x.w[e][i ^ 1] : x.w[e][i], s = odd ? x.d[e][i ^ 1] : x.d[e][i];
                        const __half2 d = u2h(x.live ? __byte_perm(s, 0, odd ? 0x3232 : 0x1010) : 0u);
                        const __half2 c[4] = {signed_f16<0>(w), signed_f16<1>(w), signed_f16<2>(w), signed_f16<3>(w)};
                        uint4 *at = reinterpret_cast<uint4 *>(to + (i >> 1) * (BT * 128) + (k_off ^ (i & 1 ? 64 : 0)));
                        __half2 k[4];
#pragma unroll
                        for (int x = 0; x < 4; x++) k[x] = __hmul2(c[x], d);
                        at[0] = make_uint4(h2u(k[0]), h2u(k[1]), h2u(k[2]), h2u(k[3]));
                        if constexpr (C::KP == 2) {   // what the rounding left, exactly
#pragma unroll
                            for (int x = 0; x < 4; x++) k[x] = __hfma2(c[x], d, __hneg2(k[x]));
                            at[C::K_PART / 16] = make_uint4(h2u(k[0]), h2u(k[1]), h2u(k[2]), h2u(k[3]));
                        }
                    }
                }
            };
            auto load_values = [&](int rs, int j, int step, Values &x) {
                const uint8_t *raw = raws + rs * C::RAW_BYTES + (4 * step + tl) * C::PITCH;
                const bool live = (raw_mask[rs] >> (4 * step + tl)) & 1;
                const int i = i_base + j * C::GT + 4 * step + tl;
                x.end = live ? last - (i < n_sink ? i : w_tile + i - n_sink) * KV_TILE : -1;
                const int b0 = hb * XS;
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const uint8_t *wp = raw + 4 * (((pp * NC + b0 / BW) * 32 + vg * 4 + q) * BW + b0 % BW);
                    const uint8_t *dp = raw + (L::VS - L::VC) + 4 * ((4 * pp + q) * NB + b0);
                    if constexpr (XS == 1) {
                        x.w[q][0] = *reinterpret_cast<const uint32_t *>(wp);
                        x.d[q][0] = *reinterpret_cast<const uint32_t *>(dp);
                    } else {
                        lds_words<XS>(wp, x.w[q]);
                        lds_words<XS>(dp, x.d[q]);
                    }
                }
            };
            auto put_values = [&](uint8_t *sv, int step, Values &x) {
                uint8_t *to = sv + step * (D * 128) + v_row;
                if (x.end < 7) {   // scales of tokens past the last query's position may be anything
                    const int end = x.end;
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const uint32_t keep = (2 * q <= end ? 0xffffu : 0u) | (2 * q + 1 <= end ? 0xffff0000u : 0u);
#pragma unroll
                        for (int i = 0; i < XS; i++) x.d[q][i] &= keep;
                    }
                }
#pragma unroll
                for (int i = 0; i < XS; i++) {
                    uint32_t v[4][4];
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const __half2 d = u2h(x.d[q][i]);
                        v[0][q] = h2u(__hmul2(signed_f16<0>(x.w[q][i]), d));
                        v[1][q] = h2u(__hmul2(signed_f16<1>(x.w[q][i]), d));
                        v[2][q] = h2u(__hmul2(signed_f16<2>(x.w[q][i]), d));
                        v[3][q] = h2u(__hmul2(signed_f16<3>(x.w[q][i]), d));
                    }
#pragma unroll
                    for (int nib = 0; nib < 4; nib++)
                        *reinterpret_cast<uint4 *>(to + (32 * i + nib) * 128 + (v_cx ^ (nib * 16))) =
                            make_uint4(v[nib][0], v[nib][1], v[nib][2], v[nib][3]);
                }
            };
            Keys ka, kc;
            Values va, vc;
            int rk = 0;
            if (wk.nblk > 0) {
                rk = raw_wait(0);
                if (ok) load_keys(rk, 0, ka);
            }
            for (int j = 0; j < wk.nblk && ok; j++) {
                const int kb = wk.blocks_before + j, ks = kb % C::KST, vs = kb % C::VST;
                uint8_t *sk = smem + C::OFF_K + ks * C::K_BYTES, *sv = smem + C::OFF_V + vs * C::V_BYTES;
                ok = tc::mbar_wait(&k_empty[ks], ((uint32_t)(kb / C::KST) & 1u) ^ 1u);
                if (!ok) break;
                const int mask = raw_mask[rk];
                if constexpr (STEPS == 2) {
                    load_keys(rk, 1, kc);
                    put_keys(sk, 0, ka);
                }
                const int rv = raw_wait(2 * j + 1);
                if (!ok) break;
                load_values(rv, j, 0, va);
                put_keys(sk, STEPS - 1, STEPS == 2 ? kc : ka);
                arrive(&raw_empty[rk]);
                if (w8 == 0 && lane == 0) blk_mask[kb & 7] = mask;
                tc::fence_proxy_async_smem();
                arrive(&k_full[ks]);
                if constexpr (STEPS == 2) load_values(rv, j, 1, vc);
                ok = tc::mbar_wait(&v_empty[vs], ((uint32_t)(kb / C::VST) & 1u) ^ 1u);
                if (!ok) break;
                put_values(sv, 0, va);
                if constexpr (STEPS == 2) put_values(sv, 1, vc);
                arrive(&raw_empty[rv]);
                tc::fence_proxy_async_smem();
                arrive(&v_full[vs]);
                if (*abort_flag) break;
                if (j + 1 < wk.nblk) {
                    rk = raw_wait(2 * j + 2);
                    if (ok) load_keys(rk, 0, ka);
                }
            }
            if (!ok && lane == 0) fail(4);
        }
    } else {
        set_registers<C::REGS_OTHER>();
        for (int64_t st = 0; st < stripes; st++) {
            const int64_t it = item_of(st);
            if (it >= total) continue;
            if (!begin(wk, it)) break;
            if (warp == AP_MMA) {
                // ================= MMA: the warp stays together and every operand comes from values that are known to
                // be the same in all lanes, so that they are computed in uniform registers, where the instruction
                // wants them (moving them there took 100 cycles an MMA); one elected lane issues
                auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
                const int nrt = same(wk.nrt), nitems = same(wk.nitems), before = same(wk.blocks_before);
                const int uses0 = same(wk.uses[0]), uses1 = same(wk.uses[1]);
                const uint32_t tm = (uint32_t)same((int)tmem);
                if (nitems > 0) {
                    constexpr uint32_t idesc_s = tc::idesc_f16_f32(128, BT), idesc_o = tc::idesc_f16_f32(128, D);
                    const uint32_t q_base = (uint32_t)same((int)tc::smem_u32(smem)), k_base = q_base + C::OFF_K, v_base = q_base + C::OFF_V;
                    auto wait = [](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity)); };
                    bool ok = wait(&q_full, (uint32_t)wk.items & 1u);
                    tc::tc_fence_after();
                    auto scores = [&](int j, int t, int x) {
                        const int kb = before + j, ks = kb % C::KST;
                        if (t == 0) ok = ok && wait(&k_full[ks], (uint32_t)(kb / C::KST) & 1u);
                        if (!ok) return;
                        tc::tc_fence_after();
                        // a step within a tile only adds to the address field of its descriptor
                        const uint64_t qd = tc::sw128_desc(q_base + t * (128 * D * 2)), kd = tc::sw128_desc(k_base + ks * C::K_BYTES);
                        const uint32_t d = tm + x * C::COL_S;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < D / 16; k++)
                                tc::mma_f16(d, qd + ((k / 4) * 16384 + (k % 4) * 32) / 16,
                                            kd + ((k / 4) * (BT * 128) + (k % 4) * 32) / 16, idesc_s, k > 0);
                            if constexpr (C::KP == 2)
#pragma unroll
                                for (int k = 0; k < D / 16; k++)
                                    tc::mma_f16(d, qd + ((k / 4) * 16384 + (k % 4) * 32) / 16,
                                                kd + (C::K_PART + (k / 4) * (BT * 128) + (k % 4) * 32) / 16, idesc_s, 1);
                            tc::mma_commit(&s_full[x]);
                            if (t == nrt - 1) tc::mma_commit(&k_empty[ks]);
                        }
                        __syncwarp();
                    };
                    if (ok) scores(0, 0, 0);
                    if (ok && nitems > 1) scores(nrt == 1 ? 1 : 0, nrt == 1 ? 0 : 1, 1);
                    // item n: row tile t of block j, S buffer x; item n + 2 two row tiles on
                    for (int n = 0, j = 0, t = 0; n < nitems && ok; n++) {
                        const int x = n & 1, kb = before + j, vs = kb % C::VST;
                        const uint32_t parity = (uint32_t)((x ? uses1 : uses0) + n / 2) & 1u;
                        ok = wait(&p_full[x], parity);
                        if (ok && t == 0) ok = wait(&v_full[vs], (uint32_t)(kb / C::VST) & 1u);
                        if (!ok || __any_sync(0xffffffffu, *abort_flag)) break;
                        tc::tc_fence_after();
                        const uint64_t vd = tc::sw128_desc(v_base + vs * C::V_BYTES);
                        const uint32_t d = tm + C::COL_O + t * D, pa = tm + x * C::COL_S, more = j > 0;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < BT / 16; k++)
                                tc::mma_f16_ts(d, pa + 8 * k, vd + ((k / 4) * (D * 128) + (k % 4) * 32) / 16, idesc_o, k > 0 ? 1 : more);
                            tc::mma_commit(&pv_done[x]);
                            if (t == nrt - 1) tc::mma_commit(&v_empty[vs]);
                        }
                        __syncwarp();
                        if (n + 2 < nitems) {
                            // the next scores overwrite this P
                            ok = wait(&pv_done[x], parity);
                            if (ok) scores(nrt == 1 ? j + 2 : j + 1, t, x);
                        }
                        if (++t == nrt) { t = 0; j++; }
                    }
                    if (!ok || __any_sync(0xffffffffu, *abort_flag)) {   // what was issued ends before the CTA does
                        if (lane == 0) fail(2);
                        if (elect_one()) tc::mma_commit(&drain);
                        __syncwarp();
                        tc::mbar_wait(&drain, 0);
                    }
                }
                __syncwarp();
            } else if (warp == AP_LOAD) {
                // ================= loads: the keys of a block, its values, the next one's keys, ..; lane i tile i
                bool ok = true;
                const int nloads = 2 * wk.nblk;
                int issued = 0;
                for (int e = 0; e < nloads && ok; e++) {
                    const int gb = wk.loads_before + e, rs = gb % C::RAWST;
                    const bool values = e & 1;
                    const int j = e / 2;
                    const int i = (CUT ? item.base : 0) + j * C::GT + (lane & (C::GT - 1));
                    int32_t pg = -1;
                    int tok = 0;
                    if (i < item.nt) {
                        tok = token_of(i);
                        const uint32_t pi = (uint32_t)tok / (uint32_t)p.page;
                        pg = pi < p.width ? p.table[item.r * p.ld + pi] : -1;
                        if (lane < C::GT && !values && item.head == 0 && (pg < 0 || pg >= p.n_pages) && p.status != nullptr &&
                            ap_first_sight(a, item, tok / KV_TILE))
                            atomicAdd(p.status, 1);
                    }
                    const bool live = lane < C::GT && pg >= 0 && pg < p.n_pages;
                    const uint32_t mask = __ballot_sync(0xffffffffu, live);
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&raw_empty[rs], ((uint32_t)(gb / C::RAWST) & 1u) ^ 1u)) && !*abort_flag;
                    if (!ok) { if (lane == 0) fail(32); break; }
                    if (lane == 0) {
                        raw_mask[rs] = (int32_t)mask;
                        tc::mbar_arrive_expect_tx(&raw_full[rs], (uint32_t)__popc(mask) * (L::BYTES / 2));
                    }
                    __syncwarp();
                    if (live) {
                        const uint32_t off = (uint32_t)tok % (uint32_t)p.page;
                        bulk_load(smem + C::OFF_RAW + rs * C::RAW_BYTES + lane * C::PITCH,
                                  p.cache + pg * a.page_bytes + (values ? L::VC : 0) +
                                      (item.head * (p.page / KV_TILE) + off / KV_TILE) * (int64_t)L::BYTES,
                                  L::BYTES / 2, &raw_full[rs]);
                    }
                    issued = e + 1;
                }
                if (!ok)   // copies that are under way land before the CTA exits
                    for (int e = max(0, issued - C::RAWST); e < issued; e++)
                        tc::mbar_wait(&raw_full[(wk.loads_before + e) % C::RAWST], (uint32_t)((wk.loads_before + e) / C::RAWST) & 1u);
            }
        }
    }
    tc::tc_fence_before();
    everyone();
    tc::tc_fence_after();
    if (warp == AP_MMA) tc::tmem_dealloc(tmem, 512);
}

// The pieces of row blocks whose tiles were cut: a warp per query row and head
// joins them in order (5 requests of up to 66 tokens, 32 heads of 256 after 3032:
// 141 us uncut, 106 us with it).
template <int D, int QT>
__global__ void __launch_bounds__(256) attn_prefill_join_kernel(const AdShape a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Attn &p = a.p;
    const int64_t w = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5, t = w / p.h;
    const int head = (int)(w - t * p.h), lane = threadIdx.x & 31;
    if (t >= p.n_tokens || t < p.q_start[0]) return;
    int r = 0;   // the last request that starts at or before t
    for (int lo = 0, hi = (int)p.R; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (p.q_start[mid] <= t) lo = mid;
        else hi = mid;
        r = lo;
    }
    const int item_rows = a.item_base[p.R], splits = a.item_base[p.R + 1], first_cut = a.item_base[p.R + 2];
    const AdReq q = ad_request(a, r);
    if (splits == 1 || t - q.rows0 >= q.q) return;   // nothing was cut; not of the prefill kernel's, or past the rows that are computed
    const int kh = head / a.G, row = (int)(t - q.rows0) * a.G + head - kh * a.G;
    const int rb = row / item_rows, nrb = (q.q * a.G + item_rows - 1) / item_rows;
    const int64_t item = a.item_base[r] + (int64_t)(nrb - 1 - rb) * a.hk + kh - first_cut;
    if (item < 0) return;   // not cut
    const float *from = a.pieces + (item * splits * item_rows + row - rb * item_rows) * (D + 2);
    const int64_t step = (int64_t)item_rows * (D + 2);
    float mx = -INFINITY, l = 0.0f;
    for (int i = 0; i < splits; i++) mx = fmaxf(mx, from[i * step]);
    const float base = mx == -INFINITY ? 0.0f : mx;
    constexpr int PL = D / 64;   // pairs per lane
    float2 v[PL];
#pragma unroll
    for (int x = 0; x < PL; x++) v[x] = make_float2(0.0f, 0.0f);
    for (int i = 0; i < splits; i++) {
        const float f = ex2(from[i * step] - base);
        l = fmaf(f, from[i * step + 1], l);
#pragma unroll
        for (int x = 0; x < PL; x++) {
            const float2 o = *reinterpret_cast<const float2 *>(from + i * step + 2 + 2 * lane + 64 * x);
            v[x].x = fmaf(f, o.x, v[x].x);
            v[x].y = fmaf(f, o.y, v[x].y);
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *out = reinterpret_cast<uint16_t *>(p.out) + t * p.ldo + (int64_t)head * D + 2 * lane;
#pragma unroll
    for (int x = 0; x < PL; x++) {
        const float f0 = l == 0.0f ? 0.0f : v[x].x * inv, f1 = l == 0.0f ? 0.0f : v[x].y * inv;
        out[64 * x] = QT == GGUF_BF16 ? f2bf_rn(f0) : f2h_rn(f0);
        out[64 * x + 1] = QT == GGUF_BF16 ? f2bf_rn(f1) : f2h_rn(f1);
    }
}

template <int D, int QT, bool CUT>
static cudaError_t attn_prefill_launch(const AdShape &a, int ctas, cudaStream_t s) {
    cudaError_t err = cudaSuccess;
    if (kernel_occupancy((const void *)attn_prefill_kernel<D, QT, CUT>, AP_THREADS, ApCfg<D, QT>::SMEM, &err) == 0) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(AP_THREADS);
    cfg.dynamicSmemBytes = ApCfg<D, QT>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_prefill_kernel<D, QT, CUT>, a); e != cudaSuccess || !CUT) return e;
    cfg.gridDim = dim3((unsigned)((a.p.n_tokens * a.p.h + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn_prefill_join_kernel<D, QT>, a);
}

// Two builds of the kernel: what cutting adds costs its spare registers (8192 tokens: 664 us with it, 644 without).
template <int D, int QT>
static cudaError_t attn_prefill_run(const AdShape &a, int ctas, cudaStream_t s) {
    return a.max_splits > 1 ? attn_prefill_launch<D, QT, true>(a, ctas, s) : attn_prefill_launch<D, QT, false>(a, ctas, s);
}

}  // namespace gg
