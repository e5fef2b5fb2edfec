// gguf_kv_plan: the pages, slots and positions of one step, from the lengths
// of its requests.
//
// With c_r tokens cached and n_r new ones, request r holds had_r = ceil(c_r / P)
// pages and needs has_r = ceil((c_r + n_r) / P).  The prefix sums of n_r and of
// has_r - had_r number the new tokens and the new pages in request order; page
// number j is the j-th free one.  Every token then follows from its own number
// by a search in the prefix sums, so one launch does everything: each CTA makes
// both prefix sums in its shared memory (8 bytes read per request, from L2) and
// takes its share of the tokens or of the new pages.  A token of a new page
// takes its page from the free list itself, never from a table entry that
// another CTA may be writing.
//
// Bound: latency (launch, one scan, two dependent loads); the bytes are 12 per
// token.  Measured, call after call: 8 decoding requests 2.9 us, 2048 requests
// of 131072 new tokens 10.2 us (1.6 MB; in a captured graph 2.7 and 9.2 us): there
// the 11 dependent reads of every token's search show.
#include <algorithm>

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

// ceil(x / P) for x < 2^32, by a shift where P is a power of two
struct Pages {
    uint32_t P;
    int shift;
    __device__ __forceinline__ uint32_t of(uint32_t x) const { return shift >= 0 ? x >> shift : x / P; }
    __device__ __forceinline__ uint32_t up(uint32_t x) const { return of(x) + (x != of(x) * P ? 1u : 0u); }
};

__global__ void __launch_bounds__(KP_THREADS) kv_plan_kernel(const KvPlan p, int token_ctas) {
    extern __shared__ int32_t sm[];
    int32_t *start = sm, *before = sm + p.R + 1, *cached = sm + 2 * (p.R + 1);
    __shared__ int64_t part[2][KP_THREADS / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = (int)p.R, width = (int)p.width;
    const uint32_t P = (uint32_t)p.page;
    const Pages pages_of{P, (P & (P - 1)) == 0 ? __ffs(P) - 1 : -1};
    const int per = (R + KP_THREADS - 1) / KP_THREADS;
    const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
    auto held = [&](uint32_t tokens) { return (int)min(pages_of.up(tokens), (uint32_t)width); };   // pages of a row
    // 64-bit sums, so that lengths of any size leave the prefix sums monotone
    int64_t nt = 0, np = 0;
    for (int r = r0; r < r1; r += 4) {   // four at a time: their loads are under way together
        int32_t c4[4], n4[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            c4[i] = r + i < r1 ? p.ctx[r + i] : 0;
            n4[i] = r + i < r1 ? p.add[r + i] : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (r + i >= r1) break;
            const uint32_t c = (uint32_t)max(c4[i], 0), n = (uint32_t)max(n4[i], 0);
            const int fresh = held(c + n) - held(c);
            cached[r + i] = (int32_t)c;
            start[r + i] = (int32_t)n;            // until the sums are known
            before[r + i] = fresh;
            nt += n;
            np += fresh;
        }
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
#pragma unroll
    for (int w = 0; w < KP_THREADS / 32; w++)
        if (w < warp) { st += part[0][w]; sp += part[1][w]; }
    constexpr int64_t CAP = 0x7fffffff;
    for (int r = r0; r < r1; r++) {
        const int32_t n = start[r], fresh = before[r];
        start[r] = (int32_t)min(st, CAP);
        before[r] = (int32_t)min(sp, CAP);
        if (blockIdx.x == 0) {
            p.q_start[r] = start[r];
            p.kv_len[r] = (int32_t)min((uint32_t)cached[r] + (uint32_t)n, (uint32_t)CAP);
        }
        st += n;
        sp += fresh;
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
    // the first token_ctas CTAs take the tokens, the others the new pages
    if ((int)blockIdx.x >= token_ctas) {
        for (int64_t j = (int64_t)(blockIdx.x - token_ctas) * KP_THREADS + tid; j < pages; j += (int64_t)(gridDim.x - token_ctas) * KP_THREADS) {
            const int r = last_not_above(before, R, (int32_t)j);
            p.table[r * p.ld + held((uint32_t)cached[r]) + (j - before[r])] = j < p.n_free ? p.free_pages[j] : -1;
        }
        return;
    }
    const int64_t step = (int64_t)token_ctas * KP_THREADS, first = (int64_t)blockIdx.x * KP_THREADS + tid;
    int lost = 0;
    for (int64_t t = first; t < p.n_tokens; t += step) {
        int32_t pos = -1;
        int64_t slot = -1;
        if (t < tokens) {
            const int r = last_not_above(start, R, (int32_t)t);
            const uint32_t c = (uint32_t)cached[r], at = c + (uint32_t)((int32_t)t - start[r]);
            const uint32_t pi = pages_of.of(at);
            const int had = held(c);
            pos = (int32_t)min(at, (uint32_t)CAP);
            int32_t pg = -1;
            if (pi < (uint32_t)had) pg = p.table[r * p.ld + pi];
            else if (pi < (uint32_t)width) {
                const int64_t j = before[r] + (int64_t)(pi - (uint32_t)had);
                if (j < p.n_free) pg = p.free_pages[j];
            }
            if (pg >= 0) slot = (int64_t)pg * P + (at - pi * P);
            else lost++;
        }
        p.pos[t] = pos;
        p.slots[t] = slot;
    }
    if (lost && p.status != nullptr) atomicAdd(p.status, lost);
}

cudaError_t launch_kv_plan(const KvPlan &p, cudaStream_t s) {
    const size_t smem = (size_t)(3 * (p.R + 1)) * sizeof(int32_t);
    cudaError_t err = cudaSuccess;
    if (smem > 48 * 1024 && kernel_occupancy((const void *)kv_plan_kernel, KP_THREADS, smem, &err) == 0) return err;
    // one token or new page per thread, up to a GPU's worth of CTAs; a step has at most a page per request more than its
    // tokens fill
    const int64_t cap = 2 * (int64_t)device_info().sm_count;
    auto ctas = [&](int64_t n, int64_t most) { return std::max<int64_t>(1, std::min(most, (n + KP_THREADS - 1) / KP_THREADS)); };
    const int64_t tokens = ctas(p.n_tokens, cap), grid = tokens + ctas(p.n_tokens / p.page + p.R, cap / 8);
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
    return cudaLaunchKernelEx(&cfg, kv_plan_kernel, p, (int)tokens);
}

}  // namespace gg
