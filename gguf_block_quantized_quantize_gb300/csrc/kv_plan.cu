// gguf_kv_plan: the pages, slots and positions of one step, from the lengths
// of its requests.
//
// With c_r tokens cached and n_r new ones, request r holds had_r = ceil(c_r / P)
// pages and needs has_r = ceil((c_r + n_r) / P).  The prefix sums of n_r and of
// has_r - had_r number the new tokens and the new pages in request order; page
// number j is the j-th free one.  Every token then follows from its own number
// by a search in the prefix sums, so one launch does everything: each CTA makes
// both prefix sums in its shared memory (8 bytes read per request, from L2) and
// takes its share of the tokens and of the new pages.  A token of a new page
// takes its page from the free list itself, never from a table entry that
// another CTA may be writing.
//
// Bound: latency (launch, one scan, two dependent loads); the bytes are 12 per
// token.
#include "common.cuh"
#include "internal.h"

namespace gg {

constexpr int KP_THREADS = 512;

// the last i in [0, n) with a[i] <= v (a non-decreasing, a[0] <= v)
__device__ __forceinline__ int last_not_above(const int32_t *a, int n, int32_t v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(KP_THREADS) kv_plan_kernel(const KvPlan p) {
    extern __shared__ int32_t sm[];
    int32_t *start = sm, *before = sm + p.R + 1;
    __shared__ int64_t part[2][KP_THREADS / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = (int)p.R, P = (int)p.page;
    const int per = (R + KP_THREADS - 1) / KP_THREADS;
    const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
    // 64-bit sums, so that lengths of any size leave the prefix sums monotone
    int64_t nt = 0, np = 0;
    for (int r = r0; r < r1; r++) {
        const int64_t c = max(p.ctx[r], 0), n = max(p.add[r], 0);
        nt += n;
        np += min((c + n + P - 1) / P, p.width) - min((c + P - 1) / P, p.width);
    }
    int64_t st = nt, sp = np;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, st, o), b = __shfl_up_sync(0xffffffffu, sp, o);
        if (lane >= o) { st += a; sp += b; }
    }
    if (lane == 31) { part[0][warp] = st; part[1][warp] = sp; }
    __syncthreads();
    st -= nt;
    sp -= np;
    for (int w = 0; w < warp; w++) { st += part[0][w]; sp += part[1][w]; }
    constexpr int64_t CAP = 0x7fffffff;
    for (int r = r0; r < r1; r++) {
        const int64_t c = max(p.ctx[r], 0), n = max(p.add[r], 0);
        start[r] = (int32_t)min(st, CAP);
        before[r] = (int32_t)min(sp, CAP);
        if (blockIdx.x == 0) {
            p.q_start[r] = start[r];
            p.kv_len[r] = (int32_t)min(c + n, CAP);
        }
        st += n;
        sp += min((c + n + P - 1) / P, p.width) - min((c + P - 1) / P, p.width);
    }
    if (r1 == R && (r0 < R || tid == 0)) {   // the thread with the last request, or thread 0 without requests
        start[R] = (int32_t)min(st, CAP);
        before[R] = (int32_t)min(sp, CAP);
    }
    __syncthreads();
    const int32_t tokens = start[R], pages = before[R];
    if (blockIdx.x == 0 && tid == 0) {
        p.q_start[R] = tokens;
        p.used[0] = (int32_t)min((int64_t)pages, p.n_free);
        if (p.status != nullptr && tokens > p.n_tokens)
            atomicAdd(p.status, (int32_t)min((int64_t)tokens - p.n_tokens, CAP));
    }
    const int64_t step = (int64_t)gridDim.x * KP_THREADS, first = (int64_t)blockIdx.x * KP_THREADS + tid;
    for (int64_t j = first; j < pages; j += step) {
        const int r = last_not_above(before, R, (int32_t)j);
        const int64_t had = min(((int64_t)max(p.ctx[r], 0) + P - 1) / P, p.width);
        p.table[r * p.ld + had + (j - before[r])] = j < p.n_free ? p.free_pages[j] : -1;
    }
    int lost = 0;
    for (int64_t t = first; t < p.n_tokens; t += step) {
        int32_t pos = -1;
        int64_t slot = -1;
        if (t < tokens) {
            const int r = last_not_above(start, R, (int32_t)t);
            const int64_t c = max(p.ctx[r], 0);
            const int64_t at = c + (t - start[r]);
            const uint32_t pi = (uint32_t)min(at, CAP) / (uint32_t)P;
            const int64_t had = min((int64_t)((uint32_t)(c + P - 1) / (uint32_t)P), p.width);
            pos = (int32_t)min(at, CAP);
            int32_t pg = -1;
            if (pi < had) pg = p.table[r * p.ld + pi];
            else if (pi < p.width) {
                const int64_t j = before[r] + ((int64_t)pi - had);
                if (j < p.n_free) pg = p.free_pages[j];
            }
            if (pg >= 0) slot = (int64_t)pg * P + (at - (int64_t)pi * P);
            else lost++;
        }
        p.pos[t] = pos;
        p.slots[t] = slot;
    }
    if (lost && p.status != nullptr) atomicAdd(p.status, lost);
}

cudaError_t launch_kv_plan(const KvPlan &p, cudaStream_t s) {
    const size_t smem = (size_t)(2 * (p.R + 1)) * sizeof(int32_t);
    cudaError_t err = cudaSuccess;
    if (smem > 48 * 1024 && kernel_occupancy((const void *)kv_plan_kernel, KP_THREADS, smem, &err) == 0) return err;
    // one token per thread up to a GPU's worth of CTAs
    int64_t grid = (p.n_tokens + KP_THREADS - 1) / KP_THREADS;
    const int64_t cap = 2 * (int64_t)device_info().sm_count;
    grid = grid < 1 ? 1 : grid > cap ? cap : grid;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(KP_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_plan_kernel, p);
}

}  // namespace gg
