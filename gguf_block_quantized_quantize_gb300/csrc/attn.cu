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

// What a call runs, from its host arguments alone.
struct AttnPlan {
    int ctas;          // of both kernels
    bool decode, prefill;
    int32_t few;       // requests with at most this many query rows per KV head go to the decode kernel
    int nt;            // its row tiles
    int32_t max_splits;
    size_t meta, base, pieces, bytes;   // offsets in the workspace behind the decode kernel's partial results, and its size
};

static AttnPlan attn_plan(const Attn &p, int64_t d) {
    AttnPlan x{};
    x.ctas = decode_ctas();
    const int64_t G = p.h / p.hk, most = G * std::min(p.max_q, p.n_tokens), sms = device_info().sm_count;
    // Requests with few query rows per KV head go to the decode kernel, the others to the prefill kernel (which takes
    // 16-bit queries); the device decides request by request.  An SM spends about 1500 cycles on 128 tokens for 8 rows
    // in the decode kernel (2100 for 16), 2800 and 5000 for up to 128 and 256 rows in the prefill kernel, so 16 rows are
    // the limit where there is work for every SM.  With fewer row blocks than SMs the limit grows by what would stand
    // idle (5 requests of 3 tokens after 600, 8 heads of 256 per KV head: 48 us there, 17 us here).
    const int64_t blocks = p.R * p.hk * ((most + 255) / 256);
    x.few = (int32_t)std::min<int64_t>(std::max<int64_t>(16, 16 * sms / std::max<int64_t>(blocks, 1)), 64);
    x.prefill = p.qt != GGUF_F32 && most > x.few;
    x.decode = !x.prefill || G <= x.few;   // some request may have as few rows
    // 16 rows at once where a unit has more than 8, so that its cache bytes are read and unpacked once
    x.nt = (x.prefill ? x.few : most) > 8 && (G > 8 || !x.prefill) && p.qt != GGUF_F32 ? 2 : 1;
    // The device cuts the tokens of row blocks into pieces, of 4 blocks at least, where SMs would stand idle: of all of
    // them where there are fewer than SMs (5 requests of up to 66 tokens, 32 heads of 256 after 3032 tokens: 141 us uncut,
    // 106 us so), of those after the last full round where few rounds end in a short one and what was cached before
    // makes them long (4 chunks of 512 tokens after 3500, 24 heads of 128: 190 us uncut, 169 us so).  Elsewhere it
    // only costs (8192 tokens: 664 us with what cutting costs the kernel, 644 us without).  The count of row blocks here is
    // an estimate: the device rounds up per request and KV head, so many short requests make more of them, and `span`
    // comes from the table's width, not from the lengths (a prompt of 77 tokens, 32 heads of 128: 17.9 us with a table of
    // its own width, 30.6 us with one of 32768 tokens; of 2048 tokens 69.9 and 70.6 us).
    const int64_t span = p.window > 0 ? std::min(p.width * p.page, p.window + p.sinks + p.max_q) : p.width * p.page;
    const int64_t rows = d == 256 ? 128 : 256, heads_rows = (p.n_tokens - std::min(p.R, p.n_tokens)) * p.h;
    const int64_t rounds = heads_rows / rows / sms, rest = heads_rows / rows % sms;
    const bool idle = heads_rows / 128 <= sms / 2 || (rounds >= 1 && rounds < 4 && rest <= sms / 2 && span >= 4 * p.max_q);
    x.max_splits = x.prefill && idle ? (int32_t)std::max<int64_t>(1, std::min<int64_t>(span / (d == 256 ? 256 : 512), 16)) : 1;
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    // two partial results of up to 16 rows (8 rows of 256 values) per CTA, and its meta data
    x.meta = up((size_t)x.ctas * 2 * (d == 256 ? 8 : 16) * (d + 2) * 4);
    x.base = up(x.meta + (size_t)x.ctas * sizeof(AdMeta));
    x.pieces = x.max_splits > 1 ? up(x.base + (size_t)(p.R + 3) * 4) : x.base;   // a piece per SM at most
    x.bytes = x.max_splits > 1 ? x.pieces + (size_t)x.ctas * rows * (d + 2) * 4 : x.base;
    return x;
}

size_t attn_ws_size(const Attn &p, int64_t d) { return attn_plan(p, d).bytes; }

cudaError_t launch_attn(const Attn &p, int64_t d, void *ws, cudaStream_t s, const int32_t *plan, int64_t entries) {
    const AttnPlan x = attn_plan(p, d);
    const int64_t es = p.qt == GGUF_F32 ? 4 : 2;
    AdShape a{};
    a.p = p;
    a.max_rows = x.prefill ? x.few : 0x7fffffff;
    a.part = (float *)ws;
    a.meta = (AdMeta *)((uint8_t *)ws + x.meta);
    a.err = tg_error_word();
    a.pf.plan = plan;
    a.pf.n_entries = (int32_t)entries;
    a.pf.tiles = pf_most_tiles(p);
    auto shift_of = [](int32_t v) { return (v & (v - 1)) == 0 ? __builtin_ctz(v) : -1; };
    a.G = (int32_t)(p.h / p.hk);
    a.hk = (int32_t)p.hk;
    a.G_shift = shift_of(a.G);
    a.tpp = (int32_t)(p.page / KV_TILE);
    a.tpp_shift = shift_of(a.tpp);
    a.page_bytes = kv_page_bytes(d, p.hk, p.page);
    a.vec = (reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.out)) % 16 == 0 && p.ldq * es % 16 == 0 &&
            p.ldo * es % 16 == 0;
    a.max_splits = x.max_splits;
    a.item_base = (int32_t *)((uint8_t *)ws + x.base);
    a.pieces = (float *)((uint8_t *)ws + x.pieces);
    cudaError_t e = cudaSuccess;
    if (x.decode)
        e = d == 64 ? launch_attn_decode_64(a, x.nt, x.ctas, s)
          : d == 128 ? launch_attn_decode_128(a, x.nt, x.ctas, s) : launch_attn_decode_256(a, x.nt, x.ctas, s);
    if (e != cudaSuccess || !x.prefill) return e;
    a.pf.chained = x.decode;
    a.min_rows = a.max_rows;
    a.max_rows = 0x7fffffff;
    return d == 64 ? launch_attn_prefill_64(a, x.ctas, s)
         : d == 128 ? launch_attn_prefill_128(a, x.ctas, s) : launch_attn_prefill_256(a, x.ctas, s);
}

}  // namespace gg
