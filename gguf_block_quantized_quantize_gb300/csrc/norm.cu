// gguf_block_norm: what stands between the product that ends a block and the
// product that begins the next one.
//
//   y  = act(g) * N_post(x)          N: RMS   v / sqrt(mean v^2 + eps) * w + b
//   h' = rs * h + bs * y                LAYER (v - mean) / sqrt(mean (v - mean)^2 + eps) * w + b
//   z  = N_pre(h')                   as floats, and / or as q8_1 blocks
//
// One pass: a row lies in the registers of 32 to 512 threads from its loads to
// its stores, so x, h and g are read once and h', z and the blocks written once;
// nothing in between goes to memory, and every step of it is fp32 (h' is rounded
// for its store, but the next norm takes the sum before that rounding, z's blocks
// are quantized from fp32).  A sum over the row is a tree within each warp, then the
// warps' sums in order: the same bits on every run and in every thread.  LAYER takes
// the mean first and the squares of the differences from it after, from registers.
//
// Aligned rows: a thread holds 8 consecutive values of each of its C chunks,
// four threads a q8_1 block.  Other rows: values a row width of threads apart,
// single loads that lie side by side, a warp a q8_1 block.
//
// Bound: HBM for many rows (x and h in, h', z and 36 bytes per 32 values out),
// latency for few.  Measured in a captured graph, post and pre RMS norms, bf16,
// float and q8_1 outputs: 8192 rows of 4096 67 us (4.6 TB/s; the bytes take 45;
// without q8_1 52 us, 5.2 TB/s), of 8192 131 us, of 16384 321 us; 2048 of 2048
// 13.4 us; fp32, 4096 of 4096 54 us (5.3 TB/s); 1 row of 4096 2.9 us; 777 rows of
// 1111 fp32 values (single loads, LAYER, a gate row) 8.7 us.  Between the two: the issue of about
// 48 instructions a value with its 16-bit output pair (56 % of the slots), and the
// barriers of the two sums with 32 warps an SM, which the registers of two chunks a
// thread allow.  Sums warp by warp (16 loads each), four barriers a row and a
// rounding at a time took 101 us.
//
// Rows wider than 16384 values take eight chunks a thread, more than the registers hold:
// 344 to 448 bytes of spill loads a thread, 1000 to 1032 with single loads.  bf16 as above,
// 8192 rows of 24576 991 us, of 32768 1087 us (2.3 TB/s), 1 row of 32768 15 us; fp32, 4096
// of 32768 541 us (4.3 TB/s).  Rows that start anywhere, bf16: 8192 of 16383 591 us, of
// 32767 1472 us.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace gg {

int *tg_error_word();   // the library's device error word (mmq.cu)

constexpr int BN_THREADS = 512;

__device__ __forceinline__ float bn_from16(int t, uint32_t h) { return t == GGUF_BF16 ? bf2f((uint16_t)h) : h2f((uint16_t)h); }
// two values rounded to 16 bits, the first in the low half
__device__ __forceinline__ uint32_t bn_pair16(int t, float a, float b) {
    uint32_t w;
    if (t == GGUF_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}

// n values of a chunk (8, or fewer in the last one) from element `at`, which is 16-byte aligned
__device__ __forceinline__ void bn_ld8(const void *x, int t, int64_t at, int n, float (&v)[8]) {
    if (n == 8) {
        if (t == GGUF_F32) {
            const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(x) + at);
            const float4 a = p[0], b = p[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(x) + at);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[2 * i] = bn_from16(t, w[i] & 0xffff);
                v[2 * i + 1] = bn_from16(t, w[i] >> 16);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            v[i] = i >= n ? 0.0f : t == GGUF_F32 ? reinterpret_cast<const float *>(x)[at + i] : bn_from16(t, reinterpret_cast<const uint16_t *>(x)[at + i]);
    }
}
__device__ __forceinline__ void bn_st8(void *x, int t, int64_t at, int n, const float (&v)[8]) {
    if (n == 8) {
        if (t == GGUF_F32) {
            float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(x) + at);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; i++) w[i] = bn_pair16(t, v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(x) + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) store_out(x, t, at + i, v[i]);
    }
}

// the thread's part of a row
template <int C, bool VEC>
struct RowPart {
    int tid, threads, k;
    __device__ __forceinline__ int chunk(int c) const { return (c * threads + tid) * 8; }              // VEC: first value
    __device__ __forceinline__ int left(int c) const { return min(max(k - chunk(c), 0), 8); }          // VEC: its values
    __device__ __forceinline__ int one(int c, int i) const { return (c * 8 + i) * threads + tid; }     // else: value i
    __device__ __forceinline__ bool has(int c, int i) const { return (VEC ? chunk(c) + i : one(c, i)) < k; }
    __device__ __forceinline__ void load(const void *x, int t, int64_t row, float (&v)[C][8]) const {
#pragma unroll
        for (int c = 0; c < C; c++) {
            if constexpr (VEC) bn_ld8(x, t, row + chunk(c), left(c), v[c]);
            else {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int e = one(c, i);
                    v[c][i] = e >= k ? 0.0f : t == GGUF_F32 ? reinterpret_cast<const float *>(x)[row + e]
                                                            : bn_from16(t, reinterpret_cast<const uint16_t *>(x)[row + e]);
                }
            }
        }
    }
    __device__ __forceinline__ void store(void *x, int t, int64_t row, const float (&v)[C][8]) const {
#pragma unroll
        for (int c = 0; c < C; c++) {
            if constexpr (VEC) bn_st8(x, t, row + chunk(c), left(c), v[c]);
            else {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (one(c, i) < k) store_out(x, t, row + one(c, i), v[c][i]);
            }
        }
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// (every warp sums up the warps' parts in the same tree: the same bits everywhere.)  behind(): past the row's barrier
struct Nothing {
    __device__ __forceinline__ void operator()() const {}
};
template <class F>
__device__ __forceinline__ float row_sum(float v, float *part, int warps, F behind) {
    v = warp_sum(v);
    if (warps == 1) return v;   // a row per warp
    constexpr int MOST = BN_THREADS / 32;   // 16: both halves of a warp sum them up
    const int lane = threadIdx.x & 31, w = lane % MOST;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    behind();
    v = w < warps ? part[w] : 0.0f;
#pragma unroll
    for (int o = MOST / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// v <- N(v); part: two arrays of partial sums that nothing else uses
template <int C, bool VEC, class F>
__device__ __forceinline__ void normed(const RowPart<C, VEC> &r, int kind, const float *w, const float *b, float eps, float inv_k,
                                       float (&v)[C][8], float (*part)[BN_THREADS / 32], int warps, F behind) {
    if (kind == GGUF_NORM_NONE) return;
    if (kind == GGUF_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) s += v[c][i];   // (zeros past the row)
        const float mean = row_sum(s, part[0], warps, behind) * inv_k;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[c][i] = r.has(c, i) ? v[c][i] - mean : 0.0f;
    }
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int i = 0; i < 8; i++) s = fmaf(v[c][i], v[c][i], s);
    const float sum = kind == GGUF_NORM_LAYER ? row_sum(s, part[1], warps, Nothing()) : row_sum(s, part[1], warps, behind);
    const float inv = __frsqrt_rn(fmaf(sum, inv_k, eps));
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int i = 0; i < 8; i++) v[c][i] *= inv;
    float wv[C][8];
    if (w != nullptr) {
        r.load(w, GGUF_F32, 0, wv);
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[c][i] *= wv[c][i];
    }
    if (b != nullptr) {
        r.load(b, GGUF_F32, 0, wv);
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[c][i] += wv[c][i];
    }
}

// roundf(v / d) of N values (ties away from zero; 0 with d == 0), as the low bytes of q.  v * (1 / d) is within 2^-21 of
// the quotient relatively and the quotient below 128, so within 2^-14, which decides the rounding unless it lies that near to
// a half, or d is so small that 1 / d or the products might not be ordinary numbers: then the division itself does.
// Adding 1.5 * 2^23 leaves the rounded quotient in the low bits.
template <int N>
__device__ __forceinline__ void q8_codes(const float (&v)[N], float d, uint32_t (&q)[N]) {
    const float inv = __frcp_rn(d);
    bool near = !(d > 0x1p-100f);
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float r = __fmaf_rn(v[i], inv, kI2fBias), off = __fmaf_rn(v[i], inv, -__fsub_rn(r, kI2fBias));
        near |= !(fabsf(off) < 0.5f - 0x1p-13f);
        q[i] = __float_as_uint(r);
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < N; i++) q[i] = d != 0.0f ? (uint32_t)min(max((int)roundf(__fdiv_rn(v[i], d)), -127), 127) : 0u;
    }
}

// a row, from its x, h and gate to its outputs; release(): behind a barrier that all threads reach when they have read them
template <int XT, int HT, int C, bool VEC, bool EARLY, class F>
__device__ __forceinline__ void norm_row(const BlockNorm &p, const RowPart<C, VEC> &r, int64_t t, const void *x, const void *h,
                                         const void *gate, float (*part)[BN_THREADS / 32], F release) {
    const int warps = blockDim.x >> 5;
    const float inv_k = 1.0f / (float)(int)p.k;
    float v[C][8], o[C][8];
    if (EARLY && p.h != nullptr) r.load(h, HT, 0, o);
    if (p.x != nullptr) {
        r.load(x, XT, 0, v);
        normed(r, p.post, p.post_w, p.post_b, p.post_eps, inv_k, v, part, warps, Nothing());
        if (p.gate != nullptr) {
            float g[C][8];
            r.load(gate, p.gt, 0, g);
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    float a = g[c][i];
                    if (p.act == GGUF_GATE_TANH) a = tanhf(a);
                    else if (p.act != GGUF_GATE_NONE) a = __fdiv_rn(p.act == GGUF_GATE_SILU ? a : 1.0f, 1.0f + expf(-a));
                    v[c][i] *= a;
                }
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[c][i] = 0.0f;
    }
    if (p.h != nullptr) {
        if (!EARLY) r.load(h, HT, 0, o);
        if (p.resid != 1.0f) {
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int i = 0; i < 8; i++) o[c][i] *= p.resid;
        }
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[c][i] = fmaf(v[c][i], p.branch, o[c][i]);
    } else {
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[c][i] *= p.branch;
    }
    const bool on = p.z != nullptr || p.zq != nullptr;
    if (!std::is_same_v<F, Nothing> && (!on || p.pre == GGUF_NORM_NONE)) {   // no barrier follows
        __syncthreads();
        release();
    }
    if (p.h_out != nullptr) r.store(p.h_out, HT, t * p.ldho, v);
    if (!on) return;
    normed(r, p.pre, p.pre_w, p.pre_b, p.pre_eps, inv_k, v, part + 2, warps, release);
    if (p.z != nullptr) r.store(p.z, p.zt, t * p.ldz, v);
    if (p.zq == nullptr) return;
    uint8_t *row = p.zq + t * (p.k / QK8 * Q8_1_BYTES);
#pragma unroll
    for (int c = 0; c < C; c++) {
        if constexpr (VEC) {
            const int at = r.chunk(c), j = threadIdx.x & 3;
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++) amax = fmaxf(amax, fabsf(v[c][i]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const float d = __fdiv_rn(amax, 127.0f);
            uint32_t q[8], word[2];
            q8_codes<8>(v[c], d, q);
#pragma unroll
            for (int i = 0; i < 2; i++)
                word[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040), __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
            int sum = dp4a_ss((int)word[1], 0x01010101, dp4a_ss((int)word[0], 0x01010101, 0));
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (at < r.k) {   // (k is a multiple of 32: whole blocks)
                uint32_t *to = reinterpret_cast<uint32_t *>(row + at / QK8 * Q8_1_BYTES);
                to[1 + 2 * j] = word[0];
                to[2 + 2 * j] = word[1];
                if (j == 0) to[0] = f2h_rn(d) | (uint32_t)f2h_rn(__fmul_rn(d, (float)sum)) << 16;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int at = r.one(c, i);
                float amax = fabsf(v[c][i]);
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
                const float d = __fdiv_rn(amax, 127.0f), one[1] = {v[c][i]};
                uint32_t q[1];
                q8_codes<1>(one, d, q);
                const int sum = __reduce_add_sync(0xffffffffu, (int)(int8_t)q[0]);
                if (at >= r.k) continue;
                uint8_t *to = row + at / QK8 * Q8_1_BYTES;
                to[4 + at % QK8] = (uint8_t)q[0];
                if (at % QK8 == 0) *reinterpret_cast<uint32_t *>(to) = f2h_rn(d) | (uint32_t)f2h_rn(__fmul_rn(d, (float)sum)) << 16;
            }
        }
    }
}

__device__ __forceinline__ const uint8_t *row_at(const void *x, int t, int64_t i) { return reinterpret_cast<const uint8_t *>(x) + i * (t == GGUF_F32 ? 4 : 2); }

template <int XT, int HT, int C, bool VEC>
__global__ void __launch_bounds__(BN_THREADS) block_norm_kernel(const BlockNorm p) {
    __shared__ float part[4][BN_THREADS / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.n_tokens) return;   // whole warps, and rows of several warps have no other in their CTA
    const RowPart<C, VEC> r{(int)threadIdx.x, (int)blockDim.x, (int)p.k};
    // h is asked for before the norm of x, where there are registers for it
    norm_row<XT, HT, C, VEC, (C < 8)>(p, r, t, row_at(p.x, XT, t * p.ldx), row_at(p.h, HT, t * p.ldh), row_at(p.gate, p.gt, t * p.ldg),
                                      part, Nothing());
}

// Many rows: a CTA takes every gridDim-th row, and bulk copies bring the rows ahead into a ring in shared memory while it
// computes; without them the loads, sums and stores of the 2 to 4 rows that an SM holds wait for one another.
// Rows of x, h and gate (that of one row for all tokens apart) start and end on 16 bytes.
constexpr int BN_STAGES = 4;
struct BnRing {
    int stages;
    uint32_t bytes_x, bytes_h, bytes_g;   // of a row; 0: not there
    int *err;
};
template <int XT, int HT, int C>
__global__ void __launch_bounds__(BN_THREADS, C <= 2 ? 2 : 1) block_norm_ring_kernel(const BlockNorm p, const BnRing ring) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float part[2][4][BN_THREADS / 32];   // of every other row: a thread may still read those of the row before
    __shared__ uint64_t full[BN_STAGES];
    __shared__ int32_t dead_word;   // a wait was given up
    volatile int32_t *dead = &dead_word;
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < ring.stages; i++) tc::mbar_init(&full[i], 1);
        dead_word = 0;
    }
    tc::fence_barrier_init();
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const RowPart<C, true> r{tid, (int)blockDim.x, (int)p.k};
    const uint32_t bytes = ring.bytes_x + ring.bytes_h + ring.bytes_g;
    auto ask = [&](int64_t t, int stage) {   // thread 0
        if (t >= p.n_tokens) return;
        uint8_t *to = smem + (size_t)stage * bytes;
        tc::mbar_arrive_expect_tx(&full[stage], bytes);
        if (ring.bytes_x) tc::bulk_load(to, row_at(p.x, XT, t * p.ldx), ring.bytes_x, &full[stage]);
        if (ring.bytes_h) tc::bulk_load(to + ring.bytes_x, row_at(p.h, HT, t * p.ldh), ring.bytes_h, &full[stage]);
        if (ring.bytes_g) tc::bulk_load(to + ring.bytes_x + ring.bytes_h, row_at(p.gate, p.gt, t * p.ldg), ring.bytes_g, &full[stage]);
    };
    if (tid == 0)
        for (int i = 0; i < ring.stages; i++) ask(blockIdx.x + (int64_t)i * gridDim.x, i);
    int stage = 0, odd = 0;
    uint32_t phase = 0;
    for (int64_t t = blockIdx.x; t < p.n_tokens; t += gridDim.x) {
        if (!tc::mbar_wait(&full[stage], phase)) *dead = 1;   // (the row goes on to its barrier with what is there)
        const uint8_t *x = smem + (size_t)stage * bytes, *h = x + ring.bytes_x;
        const void *gate = ring.bytes_g ? h + ring.bytes_h : row_at(p.gate, p.gt, 0);
        norm_row<XT, HT, C, true, false>(p, r, t, x, h, gate, part[odd], [&] {
            if (tid == 0 && !*dead) ask(t + (int64_t)ring.stages * gridDim.x, stage);
        });
        if (*dead) {   // (written before a barrier of this row: seen by all) what is under way lands before the CTA exits
            if (tid == 0) {
                if (ring.err != nullptr) atomicOr(ring.err, 1);
                for (int i = 0; i < ring.stages; i++)
                    if (t + (int64_t)i * gridDim.x < p.n_tokens) tc::mbar_wait(&full[(stage + i) % ring.stages], stage + i < ring.stages ? phase : phase ^ 1);
            }
            return;
        }
        odd ^= 1;
        if (++stage == ring.stages) { stage = 0; phase ^= 1; }
    }
}

template <int XT, int HT, bool VEC>
static const void *norm_kernel(int c) {
    return c == 1 ? (const void *)block_norm_kernel<XT, HT, 1, VEC> : c == 2 ? (const void *)block_norm_kernel<XT, HT, 2, VEC>
         : c == 4 ? (const void *)block_norm_kernel<XT, HT, 4, VEC> : (const void *)block_norm_kernel<XT, HT, 8, VEC>;
}
template <bool VEC>
static const void *norm_kernel(int xt, int ht, int c) {
    if (xt == GGUF_F32) return norm_kernel<GGUF_F32, GGUF_F32, VEC>(c);
    if (xt == GGUF_BF16)
        return ht == GGUF_F32 ? norm_kernel<GGUF_BF16, GGUF_F32, VEC>(c) : norm_kernel<GGUF_BF16, GGUF_BF16, VEC>(c);
    return ht == GGUF_F32 ? norm_kernel<GGUF_F16, GGUF_F32, VEC>(c) : norm_kernel<GGUF_F16, GGUF_F16, VEC>(c);
}

template <int XT, int HT>
static const void *ring_kernel(int c) {
    return c == 1 ? (const void *)block_norm_ring_kernel<XT, HT, 1> : c == 2 ? (const void *)block_norm_ring_kernel<XT, HT, 2>
                                                                             : (const void *)block_norm_ring_kernel<XT, HT, 4>;
}
static const void *ring_kernel(int xt, int ht, int c) {
    if (xt == GGUF_F32) return ring_kernel<GGUF_F32, GGUF_F32>(c);
    if (xt == GGUF_BF16) return ht == GGUF_F32 ? ring_kernel<GGUF_BF16, GGUF_F32>(c) : ring_kernel<GGUF_BF16, GGUF_BF16>(c);
    return ht == GGUF_F32 ? ring_kernel<GGUF_F16, GGUF_F32>(c) : ring_kernel<GGUF_F16, GGUF_F16>(c);
}

cudaError_t launch_block_norm(const BlockNorm &p, int xt, int ht, bool vec, cudaStream_t s) {
    const int64_t eighths = (p.k + 7) / 8;
    int c = 1;
    while (eighths > (int64_t)BN_THREADS * c) c *= 2;
    const int threads = (int)std::max<int64_t>(32, ((eighths + c - 1) / c + 31) / 32 * 32);
    const int rows = threads == 32 ? 4 : 1;   // a row per warp needs no others of its CTA
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.n_tokens + rows - 1) / rows));
    cfg.blockDim = dim3(threads, rows);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    BlockNorm a = p;
    auto size = [](int t) { return t == GGUF_F32 ? 4u : 2u; };
    BnRing ring{0, p.x ? (uint32_t)p.k * size(xt) : 0, p.h ? (uint32_t)p.k * size(ht) : 0,
                p.gate && p.ldg ? (uint32_t)p.k * size(p.gt) : 0, nullptr};
    const uint32_t bytes = ring.bytes_x + ring.bytes_h + ring.bytes_g;
    const int64_t sms = device_info().sm_count;
    if (vec && p.k > 256 && p.k <= 16384 && p.n_tokens > 8 * sms && ring.bytes_x % 16 == 0 && ring.bytes_h % 16 == 0 &&
        ring.bytes_g % 16 == 0 && 2 * bytes <= 200 * 1024) {
        // two chunks a thread where that leaves four warps: what a row costs beside its values is shared by more of them
        while (c < (p.k >= 2048 ? 2 : 1)) c *= 2;
        const int tpr = (int)(((eighths + c - 1) / c + 31) / 32 * 32);
        const int ctas = c <= 2 ? std::max(2, std::min(1024 / tpr, 8)) : 1;   // what registers leave room for
        ring.stages = std::max(2, std::min<int>(BN_STAGES, (int)(200 * 1024 / ctas / bytes)));
        ring.err = tg_error_word();
        const void *kern = ring_kernel(xt, ht, c);
        cudaError_t err = cudaSuccess;
        const int per_sm = kernel_occupancy(kern, tpr, (size_t)ring.stages * bytes, &err);
        if (per_sm == 0) return err;
        cfg.blockDim = dim3(tpr);
        cfg.gridDim = dim3((unsigned)std::min<int64_t>(p.n_tokens, per_sm * sms));
        cfg.dynamicSmemBytes = (size_t)ring.stages * bytes;
        void *args[2] = {&a, &ring};
        return cudaLaunchKernelExC(&cfg, kern, args);
    }
    void *args[1] = {&a};
    return cudaLaunchKernelExC(&cfg, vec ? norm_kernel<true>(xt, ht, c) : norm_kernel<false>(xt, ht, c), args);
}

}  // namespace gg
