// gguf_paged_attention: causal attention of queries over the paged Q4_0 cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - max),
// over the tokens j that query i (at position pos_i) sees: j <= pos_i and,
// with a window w > 0, j > pos_i - w or j < sinks.  A query that sees nothing
// gets zeros.
//
// One CTA per query row and head; the visible tokens go by in chunks of one
// key per thread.
#include "common.cuh"
#include "internal.h"
#include "kv.cuh"

namespace gg {

constexpr int AT_THREADS = 128;

__device__ __forceinline__ float ld_float(const void *p, int t, int64_t i) {
    if (t == GGUF_F32) return reinterpret_cast<const float *>(p)[i];
    const uint16_t h = reinterpret_cast<const uint16_t *>(p)[i];
    return t == GGUF_BF16 ? bf2f(h) : h2f(h);
}

template <int D>
__global__ void __launch_bounds__(AT_THREADS) attn_simple_kernel(const Attn p) {
    __shared__ float q[D], sp[AT_THREADS], red[AT_THREADS / 32];
    __shared__ int64_t tiles[AT_THREADS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    const int head = blockIdx.y, hk = head / (int)(p.h / p.hk);
    int r = 0;
    for (int lo = 0, hi = (int)p.R; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (p.q_start[mid] <= t) lo = mid;
        else hi = mid;
        r = lo;
    }
    if (t < p.q_start[0] || t >= p.q_start[p.R]) return;
    const int64_t kv = p.kv_len[r], pos = kv - (p.q_start[r + 1] - t);
    for (int i = tid; i < D; i += AT_THREADS) q[i] = ld_float(p.q, p.qt, t * p.ldq + (int64_t)head * D + i);
    float m = -INFINITY, lsum = 0.0f, acc[D / AT_THREADS + 1] = {};
    const int64_t w0 = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
    for (int64_t j0 = 0; j0 <= pos; j0 += AT_THREADS) {
        if (j0 >= p.sinks && j0 + AT_THREADS <= w0) continue;
        const int64_t j = j0 + tid;
        bool see = j <= pos && (j >= w0 || j < p.sinks);
        __syncthreads();
        const int64_t pi = j / p.page;
        const int64_t pg = see && pi < p.width ? p.table[r * p.ld + pi] : -1;
        if (see && (pg < 0 || pg >= p.n_pages)) {
            see = false;
            if (p.status != nullptr) atomicAdd(p.status, 1);
        }
        tiles[tid] = see ? pg * kv_page_bytes(D, p.hk, p.page) +
                               (hk * (p.page / KV_TILE) + (j - pi * p.page) / KV_TILE) * kv_tile_bytes(D) : -1;
        float s = -INFINITY;
        if (see) {
            const uint8_t *tile = p.cache + tiles[tid];
            const int tok = (int)(j % KV_TILE);
            s = 0.0f;
            for (int b = 0; b < D / 32; b++) {
                float a = 0.0f;
                for (int x = 0; x < 4; x++) {
                    const uint32_t w = ld_u32(tile + KvTile<D>::k_word(tok, b, x));
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        a += q[32 * b + 8 * x + i] * (float)((int)((w >> (4 * (i >> 1) + 16 * (i & 1))) & 15) - 8);
                }
                s += a * h2f(ld_u16(tile + KvTile<D>::KS + KvTile<D>::scale(tok, b)));
            }
            s *= p.scale;
        }
        float mx = s;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) red[warp] = mx;
        __syncthreads();
        for (int i = 0; i < AT_THREADS / 32; i++) mx = fmaxf(mx, red[i]);
        const float mn = fmaxf(m, mx);
        const float alpha = mn == -INFINITY ? 1.0f : expf(m - mn);
        sp[tid] = see ? expf(s - mn) : 0.0f;
        __syncthreads();
        m = mn;
        lsum *= alpha;
#pragma unroll
        for (int i = 0; i < D / AT_THREADS + 1; i++) acc[i] *= alpha;
        for (int x = 0; x < AT_THREADS; x++) {
            if (tiles[x] < 0) continue;
            lsum += sp[x];
            const int tok = (int)((j0 + x) % KV_TILE);
            const uint8_t *tile = p.cache + tiles[x];
#pragma unroll
            for (int i = 0; i < D / AT_THREADS + 1; i++) {
                const int e = tid + i * AT_THREADS;
                if (e >= D) break;
                const uint32_t w = ld_u16(tile + KvTile<D>::v_half(tok, e / 32, e % 32 / 4));
                acc[i] += sp[x] * h2f(ld_u16(tile + KvTile<D>::VS + KvTile<D>::scale(tok, e / 32))) *
                          (float)((int)((w >> (4 * (e % 4))) & 15) - 8);
            }
        }
    }
    for (int i = 0; i < D / AT_THREADS + 1; i++) {
        const int e = tid + i * AT_THREADS;
        if (e < D) store_out(p.out, p.qt, t * p.ldo + (int64_t)head * D + e, lsum > 0.0f ? acc[i] / lsum : 0.0f);
    }
}

size_t attn_ws_size(const Attn &, int64_t) { return 0; }

cudaError_t launch_attn(const Attn &p, int64_t d, void *ws, cudaStream_t s) {
    const dim3 grid((unsigned)p.n_tokens, (unsigned)p.h);
    if (d == 64) attn_simple_kernel<64><<<grid, AT_THREADS, 0, s>>>(p);
    else if (d == 128) attn_simple_kernel<128><<<grid, AT_THREADS, 0, s>>>(p);
    else attn_simple_kernel<256><<<grid, AT_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gg
