// attention of few query rows, heads of 256 values
#include "attn_decode.cuh"

namespace gg {

cudaError_t launch_attn_decode_256(const AdShape &a, int nt, int ctas, cudaStream_t s) {
    (void)nt;   // two row tiles would not fit in the registers
    if (a.p.qt == GGUF_F32) return attn_decode_run<256, GGUF_F32, 1>(a, ctas, s);
    if (a.p.qt == GGUF_F16) return attn_decode_run<256, GGUF_F16, 1>(a, ctas, s);
    return attn_decode_run<256, GGUF_BF16, 1>(a, ctas, s);
}

}  // namespace gg
