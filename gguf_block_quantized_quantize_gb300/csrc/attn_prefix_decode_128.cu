// attention over shared prefixes, heads of 128 values: entries of few query rows
#include "attn_decode.cuh"
#include "attn_prefix.h"

namespace gg {

cudaError_t launch_prefix_decode_128(const AdShape &a, int nt, int ctas, cudaStream_t s) {
    if (a.p.qt == GGUF_F32) return attn_prefix_decode_run<128, GGUF_F32, 1>(a, ctas, s);
    if (a.p.qt == GGUF_F16) return nt == 2 ? attn_prefix_decode_run<128, GGUF_F16, 2>(a, ctas, s) : attn_prefix_decode_run<128, GGUF_F16, 1>(a, ctas, s);
    return nt == 2 ? attn_prefix_decode_run<128, GGUF_BF16, 2>(a, ctas, s) : attn_prefix_decode_run<128, GGUF_BF16, 1>(a, ctas, s);
}

}  // namespace gg
