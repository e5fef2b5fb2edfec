// attention over shared prefixes, heads of 64 values: entries of many query rows
#include "attn_prefill.cuh"
#include "attn_prefix.h"

namespace gg {

cudaError_t launch_prefix_prefill_64(const AdShape &a, int ctas, cudaStream_t s) {
    static_assert(ApCfg<64, GGUF_BF16>::RT * 128 == (64 == 256 ? 128 : 256) && ApCfg<64, GGUF_BF16>::GT == (64 == 256 ? 4 : 8), "as the join has them");
    return a.p.qt == GGUF_F16 ? attn_prefill_launch<64, GGUF_F16, AP_PRE, false>(a, ctas, s) : attn_prefill_launch<64, GGUF_BF16, AP_PRE, false>(a, ctas, s);
}

}  // namespace gg
