// attention over shared prefixes, heads of 256 values: entries of few query rows
#include "attn_decode.cuh"
#include "attn_prefix.h"

namespace gg {

cudaError_t launch_prefix_decode_256(const AdShape &a, int nt, int ctas, cudaStream_t s) {
    (void)nt;   // units of 8 rows
    if (a.p.qt == GGUF_F32) return attn_prefix_decode_run<256, GGUF_F32, 1>(a, ctas, s);
    if (a.p.qt == GGUF_F16) return attn_prefix_decode_run<256, GGUF_F16, 1>(a, ctas, s);
    return attn_prefix_decode_run<256, GGUF_BF16, 1>(a, ctas, s);
}

}  // namespace gg
