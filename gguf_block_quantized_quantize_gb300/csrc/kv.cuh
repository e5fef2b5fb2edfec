// Layout of the paged Q4_0 key / value cache, shared by the kernels that write
// it (kv_rope.cu) and read it (attn*.cu).
//
// A page holds page_size tokens of every KV head, head by head, as tiles of 16
// tokens of one head; a tile is 18 * D bytes for heads of D values, the size
// of its Q4_0 blocks (18 bytes per 32 values), in the order in which the
// warp-level 16x8x16 matrix instructions take their fragments:
//   [0, 8D)    key codes    32-bit word (((t/8)*NC + b/BW)*32 + (t%8)*4 + x/8)*BW + b%BW
//                           holds values x/8*8 .. +7 of block b of token t;
//                           value x in the 4 bits from (x%8)/2*4 + (x%2)*16
//   [8D, 9D)   key scales   fp16 ((t/2)*NB + b)*2 + t%2
//   [9D, 17D)  value codes  word (((t/8)*NC + b/BW)*32 + (x/4)*4 + (t%8)/2)*BW + b%BW
//                           holds values x/4*4 .. +3 of block b of tokens t & ~1 (low
//                           half) and t | 1 (high half); value x from bit (x%4)*4
//   [17D, 18D) value scales as the key scales
// with NB = D / 32 blocks per token, in chunks of BW = min(NB, 4) whose words
// a lane reads as one vector, NC = NB / BW.  Two codes that one
// 32-bit "and" leaves at the bottom of the two halves of a register are a pair
// of neighbouring values of one key, or one value of two neighbouring tokens:
// the pairs that the matrix instructions contract over.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace gg {

constexpr int KV_TILE = 16;   // tokens per tile
__host__ __device__ constexpr int64_t kv_tile_bytes(int64_t d) { return 18 * d; }
__host__ __device__ constexpr int64_t kv_page_bytes(int64_t d, int64_t hk, int64_t page) {
    return hk * (page / KV_TILE) * kv_tile_bytes(d);
}

template <int D>
struct KvTile {
    static constexpr int NB = D / 32, BW = NB < 4 ? NB : 4, NC = NB / BW;
    static constexpr int KS = 8 * D, VC = 9 * D, VS = 17 * D, BYTES = 18 * D;
    // byte offset of the word with values 8 * x8 .. + 7 of block b of token t's key
    static __device__ __forceinline__ int k_word(int t, int b, int x8) {
        return 4 * ((((t >> 3) * NC + b / BW) * 32 + (t & 7) * 4 + x8) * BW + b % BW);
    }
    // byte offset of the 16 bits with values 4 * x4 .. + 3 of block b of token t's value
    static __device__ __forceinline__ int v_half(int t, int b, int x4) {
        return VC + 4 * ((((t >> 3) * NC + b / BW) * 32 + x4 * 4 + ((t & 7) >> 1)) * BW + b % BW) + 2 * (t & 1);
    }
    // byte offset of token t's scale of block b, from KS or VS
    static __device__ __forceinline__ int scale(int t, int b) { return 2 * (((t >> 1) * NB + b) * 2 + (t & 1)); }
};

template <int T>
__device__ __forceinline__ float from16(uint32_t h) { return T == GGUF_BF16 ? bf2f((uint16_t)h) : h2f((uint16_t)h); }

}  // namespace gg
