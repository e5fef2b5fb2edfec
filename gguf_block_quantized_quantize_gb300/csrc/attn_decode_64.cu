// attention of few query rows, heads of 64 values
#include "attn_decode.cuh"

namespace gg {

cudaError_t launch_attn_decode_64(const AdShape &a, int nt, int ctas, cudaStream_t s) {
    if (a.p.qt == GGUF_F32) return attn_decode_run<64, GGUF_F32, 1>(a, ctas, s);
    if (a.p.qt == GGUF_F16)
        return nt == 2 ? attn_decode_run<64, GGUF_F16, 2>(a, ctas, s) : attn_decode_run<64, GGUF_F16, 1>(a, ctas, s);
    return nt == 2 ? attn_decode_run<64, GGUF_BF16, 2>(a, ctas, s) : attn_decode_run<64, GGUF_BF16, 1>(a, ctas, s);
}

}  // namespace gg
