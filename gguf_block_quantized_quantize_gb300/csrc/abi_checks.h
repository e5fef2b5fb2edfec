// Argument checks that the C-ABI files share.
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include "internal.h"

namespace gg {

inline gguf_status refuse(gguf_status st, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return report(st, buf);
}
inline gguf_status launched(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return GGUF_OK;
    return refuse(GGUF_ERR_CUDA, "%s: CUDA error %d (%s)", what, (int)e, cudaGetErrorString(e));
}
inline bool float_type(int t) { return t == GGUF_F32 || t == GGUF_F16 || t == GGUF_BF16; }
inline int64_t float_size(int t) { return t == GGUF_F32 ? 4 : 2; }
inline bool at(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// every row of an array of rows starts on 16 bytes (or there is none)
inline bool rows16(const void *p, int64_t ld, int64_t es) { return p == nullptr || (at(p, 16) && (ld * es) % 16 == 0); }

}  // namespace gg
