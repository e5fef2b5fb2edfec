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
// fp16 operands (k, v = d * (c - 8), rounded to 2^-12 of them at most) once for
// all rows of the CTA.  bf16 queries are scaled per row by a power of two into
// fp16's range.  The softmax keeps a reference maximum per row and rescales O
// only when a score exceeds it by 2^5: probabilities are held as
// 2^(s - reference + 10), at most 2^15.  Statistics are fp32.
//
// Warps: 0-3 and 4-7 the softmax of a row tile each (TMEM lanes 32 * (warp %
// 4) on), 8-11 unpack, 12 issues the MMAs (and owns the TMEM allocation), 13
// loads.  Every wait is bounded (1 s); a timeout sets the error word and the
// CTA drains and exits.
#pragma once

#include "attn_decode.cuh"

namespace gg {

constexpr int AP_THREADS = 14 * 32;

template <int D>
struct ApCfg {
    static constexpr int RT = D == 256 ? 1 : 2;        // row tiles of 128 (the O accumulators fill the TMEM)
    static constexpr int BT = D == 256 ? 64 : 128;     // tokens per block
    static constexpr int KST = 2, VST = D == 256 ? 1 : 2;
    static constexpr int GT = 4;                       // cache tiles (of 16 tokens) per load
    static constexpr int RAWST = D == 64 ? 4 : 3;
    static constexpr int PITCH = 18 * D + 16;          // raw tiles apart by an odd number of 16-byte banks
    static constexpr int Q_BYTES = RT * 128 * D * 2;
    static constexpr int K_BYTES = BT * D * 2, V_BYTES = BT * D * 2;
    static constexpr int RAW_BYTES = GT * PITCH;
    static constexpr int OFF_K = Q_BYTES, OFF_V = OFF_K + KST * K_BYTES, OFF_RAW = OFF_V + VST * V_BYTES;
    static constexpr int SMEM = OFF_RAW + RAWST * RAW_BYTES + 1024;   // 1024 for the base's alignment
    static constexpr int COL_S = BT, COL_O = 256;      // TMEM columns: S buffer x at x * BT, O of row tile t at 256 + t * D
    static_assert(SMEM <= 232448 - 5120, "static shared memory fits beside");
};

// a CTA's piece of work
struct ApItem {
    int r, head, row0, rows;      // request, KV head, first query row and rows (of token * G + head)
    int q0, pos0;                 // the request's first query token, position of row row0's token
    int tok0;                     // row0 / G
    int nt, n_sink, w_tile;       // the tiles that the rows see (see AdReq)
};

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// row blocks (of ROWS query rows) x KV heads of one request
template <int ROWS>
__device__ __forceinline__ int64_t ap_items(const AdShape &a, const AdReq &q) {
    const int G = (int)(a.p.h / a.p.hk);
    return ((int64_t)q.q * G + ROWS - 1) / ROWS * a.p.hk;
}

template <int D, int QT>
__global__ void __launch_bounds__(AP_THREADS, 1) attn_prefill_kernel(const AdShape a) {
    using C = ApCfg<D>;
    using L = KvTile<D>;
    constexpr int NB = L::NB, BW = L::BW, NC = L::NC, BT = C::BT, ROWS = C::RT * 128;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t raw_full[C::RAWST], raw_empty[C::RAWST], k_full[C::KST], k_empty[C::KST], v_full[C::VST],
        v_empty[C::VST], s_full[2], p_full[2], pv_done[2], drain;
    __shared__ int32_t raw_mask[C::RAWST], blk_mask[8];
    __shared__ float q_inv[ROWS];
    __shared__ uint32_t tmem_slot;
    __shared__ int32_t abort_word;
    __shared__ ApItem item;
    __shared__ int64_t part[AP_THREADS / 32], chunk_end[AP_THREADS];
    volatile int32_t *abort_flag = &abort_word;
    const Attn &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = (int)(p.h / p.hk);
    if (tid == 0) {
        for (int i = 0; i < C::RAWST; i++) { tc::mbar_init(&raw_full[i], 1); tc::mbar_init(&raw_empty[i], 128); }
        for (int i = 0; i < C::KST; i++) { tc::mbar_init(&k_full[i], 128); tc::mbar_init(&k_empty[i], 1); }
        for (int i = 0; i < C::VST; i++) { tc::mbar_init(&v_full[i], 128); tc::mbar_init(&v_empty[i], 1); }
        for (int i = 0; i < 2; i++) { tc::mbar_init(&s_full[i], 1); tc::mbar_init(&p_full[i], 128); tc::mbar_init(&pv_done[i], 1); }
        tc::mbar_init(&drain, 1);
        tc::fence_barrier_init();
        abort_word = 0;
    }
    if (warp == 12) {
        tc::tmem_alloc(&tmem_slot, 512);
        tc::tmem_relinquish();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // work of all requests: thread t counts requests [t * per, (t + 1) * per)
    const int R = (int)p.R, per = (R + AP_THREADS - 1) / AP_THREADS;
    {
        int64_t mine = 0;
        for (int r = tid * per; r < min(R, (tid + 1) * per); r++) mine += ap_items<ROWS>(a, ad_request(a, r));
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) part[warp] = incl;
        tc::tc_fence_before();
        __syncthreads();
        tc::tc_fence_after();
        for (int w = 0; w < warp; w++) incl += part[w];
        chunk_end[tid] = incl;
        __syncthreads();
    }
    const int64_t total = chunk_end[AP_THREADS - 1];
    const uint32_t tmem = tmem_slot;
    auto fail = [&](int code) {
        *abort_flag = 1;
        if (a.err != nullptr) atomicOr(a.err, code);
    };
    auto token_of = [&](int i) { return (i < item.n_sink ? i : item.w_tile + i - item.n_sink) * KV_TILE; };

    // running uses of the stages and of the S buffers before the current item
    int blocks_before = 0, groups_before = 0, uses[2] = {0, 0};
    // items in stripes of one per CTA, every other stripe backwards: a request's row blocks come longest first
    for (int64_t stripe = 0; stripe * gridDim.x < total; stripe++) {
        const int64_t it = stripe * gridDim.x + ((stripe & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        if (it >= total) continue;
        if (tid == 0) {
            int lo = -1, hi = AP_THREADS - 1;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (chunk_end[mid] > it) hi = mid;
                else lo = mid;
            }
            int64_t before = hi > 0 ? chunk_end[hi - 1] : 0;
            ApItem w;
            AdReq q;
            for (w.r = hi * per;; w.r++) {   // it is there: it < total
                q = ad_request(a, w.r);
                const int64_t n = ap_items<ROWS>(a, q);
                if (before + n > it) break;
                before += n;
            }
            const int rows = q.q * G, nblk = (rows + ROWS - 1) / ROWS;
            w.head = (int)((it - before) % p.hk);
            w.row0 = (nblk - 1 - (int)((it - before) / p.hk)) * ROWS;
            w.rows = min(ROWS, rows - w.row0);
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
            item = w;
        }
        __syncthreads();
        // ---- queries: D / 8 lanes per row, 8 values each
        {
            constexpr int LPR = D / 8;
            for (int row = tid / LPR; row < ROWS; row += AP_THREADS / LPR) {
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
                    // a row's lanes lie in one warp and all of them are here (AP_THREADS and ROWS are multiples of 32 / LPR rows)
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
        }
        __syncthreads();
        const int nrt = item.rows > 128 ? 2 : 1;
        const int nblk = (item.nt + BT / KV_TILE - 1) / (BT / KV_TILE);
        const int nitems = nblk * nrt;
        constexpr int GPB = BT / 64;   // loads per block

        if (warp < 8) {
            // ================= softmax
            const int t = warp >> 2;
            if (t < nrt && t < C::RT) {
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
                const float sl = p.scale * 1.44269504088896341f * q_inv[row];
                float ref = -INFINITY, lsum = 0.0f;
                bool ok = true;
                for (int j = 0; j < nblk && ok; j++) {
                    const int n = j * nrt + t, x = n & 1;
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&s_full[x], (uint32_t)(uses[x] + n / 2) & 1u)) && !*abort_flag;
                    if (!ok) { if (lane == 0) fail(2); break; }
                    tc::tc_fence_after();
                    const uint32_t s_col = tmem + lanes + x * C::COL_S;
                    // whether every row of the warp sees the whole block
                    const int i0 = j * (BT / KV_TILE), i1 = min(item.nt, i0 + BT / KV_TILE);
                    const int mask = blk_mask[(blocks_before + j) & 7];
                    const int t_first = i0 < item.n_sink ? 0 : token_of(i0), t_last = token_of(i1 - 1) + KV_TILE - 1;
                    const bool whole = mask == (1 << (BT / KV_TILE)) - 1 && t_last <= first &&
                                       (p.window <= 0 || t_first > last - p.window || t_last < p.sinks);
                    auto hide = [&](float (&s)[32], int c) {   // columns 32 c .. + 31: two cache tiles
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int i = i0 + 2 * c + h;
                            const int tok = token_of(i);
                            const bool there2 = (mask >> (2 * c + h)) & 1;
                            // seen: tok + e <= pos, and tok + e > pos - window or tok + e < sinks
                            const int hi = there2 ? pos - tok : -1;
                            const int lo = p.window > 0 ? (int)max((int64_t)pos - p.window - tok, (int64_t)-1) : -1;
                            const int sk = (int)min(max(p.sinks - tok, (int64_t)0), (int64_t)KV_TILE);
#pragma unroll
                            for (int e = 0; e < 16; e++)
                                if (!(e <= hi && (e > lo || e < sk))) s[16 * h + e] = -INFINITY;
                        }
                    };
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < BT / 32; c++) {
                        uint32_t rr[32];
                        tc::tmem_ld_32x32b_x32(s_col + 32 * c, rr);
                        tc::tmem_ld_wait();
                        float s[32];
#pragma unroll
                        for (int i = 0; i < 32; i++) s[i] = __uint_as_float(rr[i]);
                        if (!whole) hide(s, c);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) mx = fmaxf(mx, fmaxf(s[i], s[i + 1]));
                    }
                    mx *= sl;
                    float alpha = 1.0f;
                    if (mx > ref + 5.0f) {
                        alpha = ex2(ref - mx);   // 0 from -inf
                        ref = mx;
                        lsum *= alpha;
                    }
                    if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
                        // O of the blocks before is complete once their last product is
                        const int np = n - nrt, xp = np & 1;
                        ok = __all_sync(0xffffffffu, tc::mbar_wait(&pv_done[xp], (uint32_t)(uses[xp] + np / 2) & 1u));
                        if (!ok) { if (lane == 0) fail(2); break; }
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 32; c++) {
                            uint32_t rr[32];
                            tc::tmem_ld_32x32b_x32(o_col + 32 * c, rr);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; i++) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha);
                            tmem_st_x32(o_col + 32 * c, rr);
                        }
                        tc::tmem_st_wait();
                    }
                    const float base = ref == -INFINITY ? 0.0f : AD_PBITS - ref;
#pragma unroll 1
                    for (int c = 0; c < BT / 32; c++) {
                        uint32_t rr[32];
                        tc::tmem_ld_32x32b_x32(s_col + 32 * c, rr);
                        tc::tmem_ld_wait();
                        float s[32];
#pragma unroll
                        for (int i = 0; i < 32; i++) s[i] = __uint_as_float(rr[i]);
                        if (!whole) hide(s, c);
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; i++) {
                            const float p0 = ex2(fmaf(s[2 * i], sl, base)), p1 = ex2(fmaf(s[2 * i + 1], sl, base));
                            lsum += p0 + p1;
                            pk[i] = pack_h2(p0, p1);
                        }
                        tmem_st_x16(s_col + 16 * c, pk);   // columns that were read before
                    }
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&p_full[x]);
                }
                // ---- the output rows
                if (ok && nblk > 0) {
                    const int np = nitems - nrt + t, xp = np & 1;
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&pv_done[xp], (uint32_t)(uses[xp] + np / 2) & 1u));
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
                        if (nblk > 0) {
                            tc::tmem_ld_32x32b_x32(o_col + 32 * c, rr);
                            tc::tmem_ld_wait();
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i++) rr[i] = 0;
                        }
                        if (there) {
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
        } else if (warp < 12) {
            // ================= unpack: warp w8 of four
            const int w8 = warp - 8;
            bool ok = true;
            for (int j = 0; j < nblk && ok; j++) {
                const int kb = blocks_before + j, ks = kb % C::KST, vs = kb % C::VST;
                uint8_t *sk = smem + C::OFF_K + ks * C::K_BYTES, *sv = smem + C::OFF_V + vs * C::V_BYTES;
                ok = tc::mbar_wait(&k_empty[ks], ((uint32_t)(kb / C::KST) & 1u) ^ 1u);
                int mask_all = 0;
                for (int gi = 0; gi < GPB && ok; gi++) {
                    const int gb = groups_before + j * GPB + gi, rs = gb % C::RAWST;
                    ok = tc::mbar_wait(&raw_full[rs], (uint32_t)(gb / C::RAWST) & 1u);
                    if (!ok) break;
                    const uint8_t *raw = smem + C::OFF_RAW + rs * C::RAW_BYTES + w8 * C::PITCH;
                    const int mask = raw_mask[rs];
                    mask_all |= mask << (4 * gi);
                    const bool live = (mask >> w8) & 1;
                    // keys: warp w8 takes tile w8, 8 tokens at a time; lane (g, q) holds values 8 q .. of its blocks
                    const int g = lane >> 2, q4 = lane & 3;
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int row = gi * 64 + w8 * 16 + e * 8 + g;   // token within the block
#pragma unroll
                        for (int c = 0; c < NC; c++) {
                            uint32_t w[BW], ds[BW];
                            if (live) {
                                lds_words<BW>(raw + 4 * ((e * NC + c) * 32 + lane) * BW, w);
                                lds_words<BW>(raw + L::KS + 4 * ((4 * e + (g >> 1)) * NB + c * BW), ds);
                            } else {
#pragma unroll
                                for (int i = 0; i < BW; i++) w[i] = ds[i] = 0;
                            }
                            if (g & 1) {   // odd rows take the blocks in another order: their stores hit other banks
#pragma unroll
                                for (int i = 0; i < BW; i += 2) {
                                    const uint32_t u = w[i], d = ds[i];
                                    w[i] = w[i + 1]; w[i + 1] = u;
                                    ds[i] = ds[i + 1]; ds[i + 1] = d;
                                }
                            }
#pragma unroll
                            for (int i = 0; i < BW; i++) {
                                const int b = c * BW + (i ^ (g & 1));
                                const __half2 d = u2h(__byte_perm(ds[i], 0, (g & 1) ? 0x3232 : 0x1010));
                                uint4 o;
                                o.x = h2u(__hmul2(signed_f16<0>(w[i]), d));
                                o.y = h2u(__hmul2(signed_f16<1>(w[i]), d));
                                o.z = h2u(__hmul2(signed_f16<2>(w[i]), d));
                                o.w = h2u(__hmul2(signed_f16<3>(w[i]), d));
                                const int chunk = 4 * b + q4;   // of 8 values
                                *reinterpret_cast<uint4 *>(sk + (chunk >> 3) * (BT * 128) + row * 128 +
                                                           (((chunk & 7) ^ (row & 7)) * 16)) = o;
                            }
                        }
                    }
                }
                if (ok) {
                    if (w8 == 0 && lane == 0) blk_mask[kb & 7] = mask_all;
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&k_full[ks]);
                    ok = tc::mbar_wait(&v_empty[vs], ((uint32_t)(kb / C::VST) & 1u) ^ 1u);
                }
                for (int gi = 0; gi < GPB && ok; gi++) {
                    const int gb = groups_before + j * GPB + gi, rs = gb % C::RAWST;
                    const uint8_t *raw0 = smem + C::OFF_RAW + rs * C::RAW_BYTES;
                    const int mask = raw_mask[rs];
                    // values: lane (tile, p, gs): 8 tokens (one 16-byte chunk of a row of V^T) of 4 values of half of
                    // the blocks; the tiles' pitch and the other eighth at odd p keep loads and stores off each
                    // other's banks
                    constexpr int XS = NB / 2;
                    const int tl = lane & 3, pp = (lane >> 2) & 1, gs = lane >> 3, hb = w8 >> 1;
                    const int g = 2 * gs + (pp ^ (w8 & 1));
                    const bool live = (mask >> tl) & 1;
                    const uint8_t *raw = raw0 + tl * C::PITCH;
                    uint32_t w[4][XS], dv[4][XS];
#pragma unroll
                    for (int q = 0; q < 4; q++)
#pragma unroll
                        for (int i = 0; i < XS; i++) {
                            const int b = hb * XS + i;
                            w[q][i] = live ? *reinterpret_cast<const uint32_t *>(raw + L::VC + 4 * (((pp * NC + b / BW) * 32 + g * 4 + q) * BW + b % BW)) : 0;
                            dv[q][i] = live ? *reinterpret_cast<const uint32_t *>(raw + L::VS + 4 * ((4 * pp + q) * NB + b)) : 0;
                        }
                    const int i0 = j * (BT / KV_TILE) + 4 * gi + tl;
                    // scales of tokens past the last query's position may be anything
                    const int end = item.pos0 + (item.row0 + item.rows - 1) / G - item.tok0 - token_of(i0) - 8 * pp;
                    if (end < 7) {
#pragma unroll
                        for (int q = 0; q < 4; q++) {
                            const uint32_t keep = (2 * q <= end ? 0xffffu : 0u) | (2 * q + 1 <= end ? 0xffff0000u : 0u);
#pragma unroll
                            for (int i = 0; i < XS; i++) dv[q][i] &= keep;
                        }
                    }
                    const int chunk = tl * 2 + pp;
#pragma unroll
                    for (int i = 0; i < XS; i++) {
                        const int b = hb * XS + i;
                        auto put = [&](int nib, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
                            const int row = 32 * b + 4 * g + nib;
                            *reinterpret_cast<uint4 *>(sv + gi * (D * 128) + row * 128 + ((chunk ^ (row & 7)) * 16)) =
                                make_uint4(x0, x1, x2, x3);
                        };
                        uint32_t x[4][4];
#pragma unroll
                        for (int q = 0; q < 4; q++) {
                            const __half2 d = u2h(dv[q][i]);
                            x[0][q] = h2u(__hmul2(signed_f16<0>(w[q][i]), d));
                            x[1][q] = h2u(__hmul2(signed_f16<1>(w[q][i]), d));
                            x[2][q] = h2u(__hmul2(signed_f16<2>(w[q][i]), d));
                            x[3][q] = h2u(__hmul2(signed_f16<3>(w[q][i]), d));
                        }
#pragma unroll
                        for (int nib = 0; nib < 4; nib++) put(nib, x[nib][0], x[nib][1], x[nib][2], x[nib][3]);
                    }
                    tc::mbar_arrive(&raw_empty[rs]);
                }
                if (ok) {
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(&v_full[vs]);
                }
                if (!ok) { if (lane == 0) fail(4); }
                if (*abort_flag) break;
            }
        } else if (warp == 12) {
            // ================= MMA
            if (lane == 0 && nblk > 0) {
                constexpr uint32_t idesc_s = tc::idesc_f16_f32(128, BT), idesc_o = tc::idesc_f16_f32(128, D);
                const uint32_t q_base = tc::smem_u32(smem), k_base = q_base + C::OFF_K, v_base = q_base + C::OFF_V;
                bool ok = true;
                auto scores = [&](int n) {
                    const int j = n / nrt, t = n % nrt, x = n & 1, kb = blocks_before + j, ks = kb % C::KST;
                    if (t == 0) ok = ok && tc::mbar_wait(&k_full[ks], (uint32_t)(kb / C::KST) & 1u);
                    if (!ok) return;
                    tc::tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / 16; k++)
                        tc::mma_f16(tmem + x * C::COL_S,
                                    tc::sw128_desc(q_base + t * (128 * D * 2) + (k / 4) * 16384 + (k % 4) * 32),
                                    tc::sw128_desc(k_base + ks * C::K_BYTES + (k / 4) * (BT * 128) + (k % 4) * 32), idesc_s, k > 0);
                    tc::mma_commit(&s_full[x]);
                    if (t == nrt - 1) tc::mma_commit(&k_empty[ks]);
                };
                scores(0);
                if (nitems > 1) scores(1);
                for (int n = 0; n < nitems && ok; n++) {
                    const int j = n / nrt, t = n % nrt, x = n & 1, kb = blocks_before + j, vs = kb % C::VST;
                    ok = tc::mbar_wait(&p_full[x], (uint32_t)(uses[x] + n / 2) & 1u);
                    if (ok && t == 0) ok = tc::mbar_wait(&v_full[vs], (uint32_t)(kb / C::VST) & 1u);
                    if (!ok || *abort_flag) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int k = 0; k < BT / 16; k++)
                        tc::mma_f16_ts(tmem + C::COL_O + t * D, tmem + x * C::COL_S + 8 * k,
                                       tc::sw128_desc(v_base + vs * C::V_BYTES + (k / 4) * (D * 128) + (k % 4) * 32), idesc_o,
                                       j > 0 || k > 0);
                    tc::mma_commit(&pv_done[x]);
                    if (t == nrt - 1) tc::mma_commit(&v_empty[vs]);
                    if (n + 2 < nitems) {
                        // the next scores overwrite this P
                        ok = tc::mbar_wait(&pv_done[x], (uint32_t)(uses[x] + n / 2) & 1u);
                        if (ok) scores(n + 2);
                    }
                }
                if (!ok || *abort_flag) {   // what was issued ends before the CTA does
                    fail(2);
                    tc::mma_commit(&drain);
                    tc::mbar_wait(&drain, 0);
                }
            }
        } else {
            // ================= loads: GT tiles at a time, lane i tile i
            bool ok = true;
            const int ngroups = nblk * GPB;
            int issued = 0;
            for (int gi = 0; gi < ngroups && ok; gi++) {
                const int gb = groups_before + gi, rs = gb % C::RAWST;
                const int i = gi * C::GT + (lane & 3);
                int32_t pg = -1;
                int tok = 0;
                if (i < item.nt) {
                    tok = token_of(i);
                    const uint32_t pi = (uint32_t)tok / (uint32_t)p.page;
                    pg = pi < p.width ? p.table[item.r * p.ld + pi] : -1;
                    if (lane < 4 && (pg < 0 || pg >= p.n_pages) && p.status != nullptr) atomicAdd(p.status, 1);
                }
                const bool live = lane < 4 && pg >= 0 && pg < p.n_pages;
                const uint32_t mask = __ballot_sync(0xffffffffu, live);
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&raw_empty[rs], ((uint32_t)(gb / C::RAWST) & 1u) ^ 1u)) && !*abort_flag;
                if (!ok) { if (lane == 0) fail(32); break; }
                if (lane == 0) {
                    raw_mask[rs] = (int32_t)mask;
                    tc::mbar_arrive_expect_tx(&raw_full[rs], (uint32_t)__popc(mask) * L::BYTES);
                }
                __syncwarp();
                if (live) {
                    const uint32_t off = (uint32_t)tok % (uint32_t)p.page;
                    bulk_load(smem + C::OFF_RAW + rs * C::RAW_BYTES + lane * C::PITCH,
                              p.cache + pg * kv_page_bytes(D, p.hk, p.page) +
                                  (item.head * (p.page / KV_TILE) + off / KV_TILE) * (int64_t)L::BYTES,
                              L::BYTES, &raw_full[rs]);
                }
                issued = gi + 1;
            }
            if (!ok)   // copies that are under way land before the CTA exits
                for (int gi = max(0, issued - C::RAWST); gi < issued; gi++)
                    tc::mbar_wait(&raw_full[(groups_before + gi) % C::RAWST], (uint32_t)((groups_before + gi) / C::RAWST) & 1u);
        }
        blocks_before += nblk;
        groups_before += nblk * GPB;
        uses[0] += (nitems + 1) / 2;
        uses[1] += nitems / 2;
        tc::tc_fence_before();
        __syncthreads();   // the item's shared and tensor memory are free
        tc::tc_fence_after();
        if (*abort_flag) break;
    }
    __syncthreads();
    if (warp == 12) tc::tmem_dealloc(tmem, 512);
}

template <int D, int QT>
static cudaError_t attn_prefill_run(const AdShape &a, int ctas, cudaStream_t s) {
    cudaError_t err = cudaSuccess;
    if (kernel_occupancy((const void *)attn_prefill_kernel<D, QT>, AP_THREADS, ApCfg<D>::SMEM, &err) == 0) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(AP_THREADS);
    cfg.dynamicSmemBytes = ApCfg<D>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_prefill_kernel<D, QT>, a);
}

}  // namespace gg
