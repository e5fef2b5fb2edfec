// The launches of gguf_prefix_attention by head size (attn_prefix_*.cu).
#pragma once

#include <cuda_runtime.h>

namespace gg {

struct AdShape;

cudaError_t launch_prefix_decode_64(const AdShape &a, int nt, int ctas, cudaStream_t s);
cudaError_t launch_prefix_decode_128(const AdShape &a, int nt, int ctas, cudaStream_t s);
cudaError_t launch_prefix_decode_256(const AdShape &a, int nt, int ctas, cudaStream_t s);
cudaError_t launch_prefix_prefill_64(const AdShape &a, int ctas, cudaStream_t s);
cudaError_t launch_prefix_prefill_128(const AdShape &a, int ctas, cudaStream_t s);
cudaError_t launch_prefix_prefill_256(const AdShape &a, int ctas, cudaStream_t s);

}  // namespace gg
