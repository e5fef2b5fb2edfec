// attention of many query rows, heads of 256 values
#include "attn_prefill.cuh"

namespace gg {

cudaError_t launch_attn_prefill_256(const AdShape &a, int ctas, cudaStream_t s) {
    return a.p.qt == GGUF_F16 ? attn_prefill_run<256, GGUF_F16>(a, ctas, s) : attn_prefill_run<256, GGUF_BF16>(a, ctas, s);
}

}  // namespace gg
