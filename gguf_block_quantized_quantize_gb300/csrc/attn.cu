// gguf_paged_attention: which kernels run, and their workspace.
#include "attn_decode.cuh"

namespace gg {

int *tg_error_word();   // the library's device error word (mmq.cu)

cudaError_t launch_attn_decode_64(const AdShape &a, int nt, int ctas, cudaStream_t s);
cudaError_t launch_attn_decode_128(const AdShape &a, int nt, int ctas, cudaStream_t s);
cudaError_t launch_attn_decode_256(const AdShape &a, int nt, int ctas, cudaStream_t s);

cudaError_t launch_attn_prefill_64(const AdShape &a, int ctas, cudaStream_t s);
cudaError_t launch_attn_prefill_128(const AdShape &a, int ctas, cudaStream_t s);
cudaError_t launch_attn_prefill_256(const AdShape &a, int ctas, cudaStream_t s);

// one CTA per SM (the rings take the shared memory of one)
constexpr int MAX_CTAS = 1024;
static int decode_ctas() { return device_info().sm_count < MAX_CTAS ? device_info().sm_count : MAX_CTAS; }

// two partial results of up to 16 rows (8 rows of 256 values) per CTA, and its meta data
size_t attn_ws_size(const Attn &p, int64_t d) {
    (void)p;
    return (size_t)decode_ctas() * (2 * (d == 256 ? 8 : 16) * (d + 2) * 4 + sizeof(AdMeta));
}

cudaError_t launch_attn(const Attn &p, int64_t d, void *ws, cudaStream_t s) {
    const int ctas = decode_ctas();
    const int64_t es = p.qt == GGUF_F32 ? 4 : 2;
    AdShape a{};
    a.p = p;
    a.max_rows = 0x7fffffff;
    a.part = (float *)ws;
    a.err = tg_error_word();
    auto shift_of = [](int32_t x) { return (x & (x - 1)) == 0 ? __builtin_ctz(x) : -1; };
    a.G = (int32_t)(p.h / p.hk);
    a.hk = (int32_t)p.hk;
    a.G_shift = shift_of(a.G);
    a.tpp = (int32_t)(p.page / KV_TILE);
    a.tpp_shift = shift_of(a.tpp);
    a.page_bytes = kv_page_bytes(d, p.hk, p.page);
    a.meta = (AdMeta *)((uint8_t *)ws + (size_t)ctas * 2 * (d == 256 ? 8 : 16) * (d + 2) * 4);
    a.vec = (reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.out)) % 16 == 0 && p.ldq * es % 16 == 0 &&
            p.ldo * es % 16 == 0;
    // Requests with few query rows per KV head go to the decode kernel, the others to the prefill kernel (which takes
    // 16-bit queries); the device decides request by request.  An SM spends about 1500 cycles on 128 tokens for 8 rows
    // in the decode kernel (2100 for 16), 2800 and 5000 for up to 128 and 256 rows in the prefill kernel, so 16 rows are
    // the limit where there is work for every SM.  The prefill kernel does not cut a row block's tokens among CTAs:
    // with fewer row blocks than SMs the limit grows by what stands idle (5 requests of 3 tokens after 600, 8 heads of
    // 256 per KV head: 48 us there, 17 us here).
    const int64_t G = p.h / p.hk, most = G * p.max_q, sms = device_info().sm_count;
    const int64_t blocks = p.R * p.hk * ((most + 255) / 256);
    const int64_t few = std::min<int64_t>(std::max<int64_t>(16, 16 * sms / std::max<int64_t>(blocks, 1)), 64);
    const bool prefill = p.qt != GGUF_F32 && most > few;
    if (prefill) a.max_rows = (int32_t)few;
    // 16 rows at once where a unit has more than 8, so that its cache bytes are read and unpacked once
    const int nt = (prefill ? few : most) > 8 && (G > 8 || !prefill) && p.qt != GGUF_F32 ? 2 : 1;
    // half the rows per CTA where that fills the GPU better
    a.item_rows = d == 256 || blocks < sms ? 128 : 256;
    cudaError_t e = cudaSuccess;
    if (!prefill || G <= few)   // some request may have as few rows
        e = d == 64 ? launch_attn_decode_64(a, nt, ctas, s)
          : d == 128 ? launch_attn_decode_128(a, nt, ctas, s) : launch_attn_decode_256(a, nt, ctas, s);
    if (e != cudaSuccess || !prefill) return e;
    a.min_rows = a.max_rows;
    a.max_rows = 0x7fffffff;
    return d == 64 ? launch_attn_prefill_64(a, ctas, s)
         : d == 128 ? launch_attn_prefill_128(a, ctas, s) : launch_attn_prefill_256(a, ctas, s);
}

}  // namespace gg
