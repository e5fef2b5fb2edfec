// Native marshalling of the paged-cache calls (module _bind of the package):
// torch tensors -> pointers and strides of the C ABI, with the same argument
// rules as the ctypes binding of the other calls.  These calls stand between
// the products of every layer of a decode step, where the host's share of a
// small call is larger than the GPU's: a call costs about 0.7 us here beside
// the launch, and 5 to 10 us through ctypes.
//
// The functions take positional arguments and return the status of the C
// function that they call (whose address bind() got), or raise ValueError for a
// tensor that does not fit.  They allocate nothing, but prefix_plan and
// prefix_attention: those make what they are not given (plan, output, workspace) in
// the same call, and return the plan or the output instead of the status 0.
#include <Python.h>

#include <ATen/Functions.h>

#include <torch/csrc/autograd/python_variable.h>

#include "gguf_gb300.h"

namespace {

typedef gguf_status (*plan_fn)(const int32_t *, const int32_t *, int64_t, const int32_t *, int64_t, int32_t *, int64_t,
                               int64_t, int64_t, int64_t, int32_t *, int32_t *, int32_t *, int64_t *, int32_t *, int32_t *,
                               gguf_stream_t);
typedef gguf_status (*rope_fn)(const gguf_qk_rope_args *, gguf_stream_t);
typedef gguf_status (*rows_fn)(const void *, int64_t, int64_t, int64_t, int64_t, const int64_t *, int64_t, void *, void *, int,
                               gguf_stream_t);
typedef size_t (*attn_ws_fn)(const gguf_attn_args *);
typedef gguf_status (*attn_fn)(const gguf_attn_args *, void *, size_t, gguf_stream_t);
typedef int64_t (*page_fn)(int64_t, int64_t, int64_t);
typedef gguf_status (*mrope_fn)(const gguf_qk_rope_args *, const gguf_rope_axes *, gguf_stream_t);
typedef gguf_status (*pplan_fn)(const int32_t *, const int32_t *, int64_t, const int32_t *, const int32_t *, int64_t, int64_t,
                                int64_t, void *, size_t, gguf_stream_t);
typedef size_t (*pattn_ws_fn)(const gguf_attn_args *, int64_t);
typedef gguf_status (*pattn_fn)(const gguf_attn_args *, const void *, size_t, int64_t, void *, size_t, gguf_stream_t);
typedef gguf_status (*norm_fn)(const gguf_block_norm_args *, gguf_stream_t);

struct {
    plan_fn plan;
    rope_fn rope;
    rows_fn rows;
    attn_ws_fn attn_ws;
    attn_fn attn;
    page_fn page_bytes;
    mrope_fn mrope;
    norm_fn norm;
    pplan_fn pplan;
    pattn_ws_fn pattn_ws;
    pattn_fn pattn;
    page_fn pplan_bytes;
} api;

struct Bad {};   // a Python exception is set

[[noreturn]] void refuse(const char *what, const char *name, const char *want) {
    PyErr_Format(PyExc_ValueError, "%s: %s must be %s", what, name, want);
    throw Bad();
}
// The device of the call's tensors: ANY (the calls of the cache itself: what the current device can read), or ONE, that of
// the first
constexpr int ANY = -2, ONE = -1;
thread_local int device_of_call = ANY;
const at::Tensor &tensor(PyObject *o, const char *what, const char *name) {
    if (!THPVariable_Check(o)) refuse(what, name, "a tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) {
        PyErr_SetString(PyExc_ValueError, "gguf: tensors must live on a CUDA device");
        throw Bad();
    }
    if (device_of_call == ONE) device_of_call = t.get_device();
    if (device_of_call != ANY && t.get_device() != device_of_call) refuse(what, name, "on the device of the call's other tensors");
    return t;
}
int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Bad();
    return v;
}
double real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Bad();
    return v;
}
// a contiguous array of at least n elements
template <class T>
T *array(PyObject *o, int64_t n, const char *what, const char *name) {
    constexpr bool wide = sizeof(T) == 8;
    const at::Tensor &t = tensor(o, what, name);
    if (t.scalar_type() != (wide ? at::kLong : at::kInt) || t.numel() < n || !t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s: %s must be a contiguous %s tensor of at least %lld", what, name,
                     wide ? "int64" : "int32", (long long)n);
        throw Bad();
    }
    return static_cast<T *>(t.data_ptr());
}
template <class T>
T *array_or_none(PyObject *o, int64_t n, const char *what, const char *name) {
    return o == Py_None ? nullptr : array<T>(o, n, what, name);
}
struct Table {
    int32_t *p;
    int64_t ld, width;
};
Table table(PyObject *o, int64_t rows, const char *what) {
    const at::Tensor &t = tensor(o, what, "block_table");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) < rows || (t.size(1) > 1 && t.stride(1) != 1))
        refuse(what, "block_table", "int32 [requests, width] with contiguous rows");
    return {static_cast<int32_t *>(t.data_ptr()), t.size(0) > 1 ? t.stride(0) : t.size(1), t.size(1)};
}
// [tokens, heads, head_dim] with the heads of a token side by side; the tokens may be strided
struct Rows {
    void *p;
    int64_t ld;
};
Rows rows(const at::Tensor &t, int64_t n, int64_t heads, int64_t d, at::ScalarType type, const char *what, const char *name) {
    if (t.scalar_type() != type || t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != d ||
        (d > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != d)) {
        PyErr_Format(PyExc_ValueError, "%s: %s must be [%lld, %lld, %lld] of q's dtype with the heads of a token side by side",
                     what, name, (long long)n, (long long)heads, (long long)d);
        throw Bad();
    }
    return {t.data_ptr(), n > 1 ? t.stride(0) : heads * d};
}
int float_type(at::ScalarType t, const char *what) {
    if (t == at::kBFloat16) return GGUF_BF16;
    if (t == at::kHalf) return GGUF_F16;
    if (t == at::kFloat) return GGUF_F32;
    refuse(what, "the tensors", "fp32, bf16 or fp16");
}
struct Pages {
    void *p;
    int64_t n;
};
Pages pages(PyObject *o, int64_t d, int64_t hk, int64_t page, const char *what) {
    const at::Tensor &t = tensor(o, what, "cache");
    const int64_t bytes = api.page_bytes(d, hk, page);   // -1: the library refuses the sizes itself
    if (t.dim() != 2 || (bytes > 0 && (t.scalar_type() != at::kByte || t.size(1) != bytes || !t.is_contiguous()))) {
        PyErr_Format(PyExc_ValueError, "%s: cache must be a contiguous uint8 tensor [pages, %lld]", what, (long long)bytes);
        throw Bad();
    }
    return {t.data_ptr(), t.size(0)};
}
const float *weights(PyObject *o, int64_t d, const char *what, const char *name) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, what, name);
    if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != d || t.stride(0) != 1) {
        PyErr_Format(PyExc_ValueError, "%s: %s must be %lld contiguous fp32 values", what, name, (long long)d);
        throw Bad();
    }
    return static_cast<const float *>(t.data_ptr());
}
gguf_stream_t stream(PyObject *o) { return reinterpret_cast<gguf_stream_t>(static_cast<intptr_t>(integer(o))); }
void count(Py_ssize_t n, Py_ssize_t want, const char *what) {
    if (n == want) return;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", what, want, n);
    throw Bad();
}
template <class F>
PyObject *guarded(F f, int devices = ANY) {
    device_of_call = devices;
    try {
        return f();
    } catch (const Bad &) {
    } catch (const c10::OutOfMemoryError &e) {   // what torch.empty raises
        PyObject *torch = PyImport_ImportModule("torch"), *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// ctx, new, free, table, page, n_tokens, q_start, kv_len, positions, slots, used, status, stream
PyObject *kv_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const char *what = "gguf_kv_plan";
        count(n, 13, what);
        const int64_t r = tensor(a[1], what, "new_len").numel(), tokens = integer(a[5]);
        const Table t = table(a[3], r, what);
        return PyLong_FromLong(api.plan(
            array<int32_t>(a[0], r, what, "ctx_len"), array<int32_t>(a[1], r, what, "new_len"), r,
            array<int32_t>(a[2], 0, what, "free_pages"), tensor(a[2], what, "free_pages").numel(), t.p, t.ld, t.width,
            integer(a[4]), tokens, array<int32_t>(a[6], r + 1, what, "q_start"), array<int32_t>(a[7], r, what, "kv_len"),
            array<int32_t>(a[8], tokens, what, "positions"), array<int64_t>(a[9], tokens, what, "slots"),
            array<int32_t>(a[10], 1, what, "pages_used"), array_or_none<int32_t>(a[11], 1, what, "dev_status"), stream(a[12])));
    });
}

// q, k, v, q_norm, k_norm, eps, positions, cos_sin, rope_type, cache, slots, page, q_out, k_out, status, stream
// (positions apart)
gguf_qk_rope_args rope_args(PyObject *const *a, const char *what) {
    const at::Tensor &q = tensor(a[0], what, "q");
    if (q.dim() != 3) refuse(what, "q", "[tokens, heads, head_dim]");
    const int64_t t = q.size(0), h = q.size(1), d = q.size(2);
    const at::ScalarType type = q.scalar_type();
    gguf_qk_rope_args x{};
    x.xt = float_type(type, what);
    x.n_tokens = t;
    x.n_heads = h;
    x.head_dim = d;
    Rows r = rows(q, t, h, d, type, what, "q");
    x.q = r.p;
    x.ldq = r.ld;
    r = rows(tensor(a[12], what, "q_out"), t, h, d, type, what, "q_out");
    x.q_out = r.p;
    x.ldqo = r.ld;
    if (a[1] != Py_None) {
        const at::Tensor &k = tensor(a[1], what, "k");
        x.n_kv_heads = k.dim() == 3 ? k.size(1) : 0;
        r = rows(k, t, x.n_kv_heads, d, type, what, "k");
        x.k = r.p;
        x.ldk = r.ld;
    }
    if (a[13] != Py_None) {
        r = rows(tensor(a[13], what, "k_out"), t, x.n_kv_heads, d, type, what, "k_out");
        x.k_out = r.p;
        x.ldko = r.ld;
    }
    x.page_size = integer(a[11]);
    if (a[9] != Py_None) {
        if (a[1] == Py_None || a[2] == Py_None || a[10] == Py_None) refuse(what, "k, v and slots", "given to store");
        r = rows(tensor(a[2], what, "v"), t, x.n_kv_heads, d, type, what, "v");
        x.v = r.p;
        x.ldv = r.ld;
        const Pages c = pages(a[9], d, x.n_kv_heads, x.page_size, what);
        x.cache = c.p;
        x.n_pages = c.n;
        x.slots = array<int64_t>(a[10], t, what, "slots");
    }
    x.q_norm = weights(a[3], d, what, "q_norm");
    x.k_norm = weights(a[4], d, what, "k_norm");
    x.eps = static_cast<float>(real(a[5]));
    if (a[7] != Py_None) {
        const at::Tensor &c = tensor(a[7], what, "cos_sin");
        if (c.scalar_type() != at::kFloat || c.dim() != 2 || !c.is_contiguous())
            refuse(what, "cos_sin", "a contiguous fp32 tensor [positions, rot]");
        x.cos_sin = static_cast<const float *>(c.data_ptr());
        x.n_positions = c.size(0);
        x.rot = c.size(1);
    }
    x.rope_type = static_cast<int>(integer(a[8]));
    x.dev_status = array_or_none<int32_t>(a[14], 1, what, "dev_status");
    return x;
}

PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const char *what = "gguf_qk_norm_rope";
        count(n, 16, what);
        gguf_qk_rope_args x = rope_args(a, what);
        x.positions = array<int32_t>(a[6], x.n_tokens, what, "positions");
        return PyLong_FromLong(api.rope(&x, stream(a[15])));
    });
}

// the same, then sections (a tuple) and interleaved
PyObject *qk_norm_mrope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const char *what = "gguf_qk_norm_mrope";
        count(n, 18, what);
        gguf_qk_rope_args x = rope_args(a, what);
        gguf_rope_axes axes{};
        if (!PyTuple_Check(a[16])) refuse(what, "sections", "a tuple of the pairs of each axis");
        axes.n_axes = PyTuple_GET_SIZE(a[16]);
        for (int64_t i = 0; i < axes.n_axes && i < GGUF_MAX_AXES; i++) {
            const int64_t pairs = integer(PyTuple_GET_ITEM(a[16], i));
            if (pairs < 0 || pairs > 65535) refuse(what, "sections", "the pairs of each axis");
            axes.sections[i] = static_cast<int32_t>(pairs);
        }
        const at::Tensor &pos = tensor(a[6], what, "positions");
        if (pos.scalar_type() != at::kInt || pos.dim() != 2 || pos.size(0) != axes.n_axes || pos.size(1) != x.n_tokens ||
            (x.n_tokens > 1 && pos.stride(1) != 1))
            refuse(what, "positions", "int32 [axes, tokens] with contiguous rows");
        x.positions = static_cast<const int32_t *>(pos.data_ptr());
        axes.ld_positions = axes.n_axes > 1 ? pos.stride(0) : x.n_tokens;
        axes.interleaved = static_cast<int>(integer(a[17]));
        return PyLong_FromLong(api.mrope(&x, &axes, stream(a[15])));
    }, ONE);
}

// [tokens, k] with contiguous rows, or none
struct Flat {
    void *p;
    int type;
    int64_t ld;
};
Flat flat(PyObject *o, int64_t t, int64_t k, const char *what, const char *name) {
    if (o == Py_None) return {nullptr, GGUF_F32, k};
    const at::Tensor &x = tensor(o, what, name);
    if (x.dim() != 2 || x.size(0) != t || x.size(1) != k || (k > 1 && x.stride(1) != 1)) {
        PyErr_Format(PyExc_ValueError, "%s: %s must be [%lld, %lld] with contiguous rows", what, name, (long long)t, (long long)k);
        throw Bad();
    }
    return {x.data_ptr(), float_type(x.scalar_type(), what), t > 1 ? x.stride(0) : k};
}

// x, h, gate, gate_act, branch_scale, residual_scale, post kind, weight, bias, eps, pre kind, weight, bias, eps, h_out, z,
// z_q8_1, stream
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const char *what = "gguf_block_norm";
        count(n, 18, what);
        const at::Tensor &any = tensor(a[0] != Py_None ? a[0] : a[1], what, a[0] != Py_None ? "x" : "residual");
        if (any.dim() != 2) refuse(what, "x and residual", "[tokens, k]");
        const int64_t t = any.size(0), k = any.size(1);
        gguf_block_norm_args x{};
        x.n_tokens = t;
        x.k = k;
        const Flat fx = flat(a[0], t, k, what, "x"), fh = flat(a[1], t, k, what, "residual");
        const Flat fo = flat(a[14], t, k, what, "residual_out"), fz = flat(a[15], t, k, what, "out");
        x.ht = a[1] != Py_None ? fh.type : a[14] != Py_None ? fo.type : fx.type;
        x.xt = a[0] != Py_None ? fx.type : x.ht;
        if (a[14] != Py_None && fo.type != x.ht) refuse(what, "residual_out", "of the residual's dtype");
        x.x = fx.p;
        x.ldx = fx.ld;
        x.h = fh.p;
        x.ldh = fh.ld;
        x.h_out = fo.p;
        x.ldho = fo.ld;
        x.z = fz.p;
        x.zt = fz.type;
        x.ldz = fz.ld;
        x.gt = x.xt;
        if (a[2] != Py_None) {
            const at::Tensor &g = tensor(a[2], what, "gate");
            if (g.dim() == 1 || (g.dim() == 2 && g.size(0) == 1 && t != 1)) {   // one row for all tokens
                if (g.size(-1) != k || (k > 1 && g.stride(-1) != 1)) refuse(what, "gate", "[tokens, k] or [k] with contiguous rows");
                x.gate = g.data_ptr();
                x.gt = float_type(g.scalar_type(), what);
                x.ldg = 0;
            } else {
                const Flat fg = flat(a[2], t, k, what, "gate");
                x.gate = fg.p;
                x.gt = fg.type;
                x.ldg = fg.ld;
            }
        }
        x.gate_act = static_cast<int>(integer(a[3]));
        x.branch_scale = static_cast<float>(real(a[4]));
        x.residual_scale = static_cast<float>(real(a[5]));
        x.post_kind = static_cast<int>(integer(a[6]));
        x.post_w = weights(a[7], k, what, "post_weight");
        x.post_b = weights(a[8], k, what, "post_bias");
        x.post_eps = static_cast<float>(real(a[9]));
        x.pre_kind = static_cast<int>(integer(a[10]));
        x.pre_w = weights(a[11], k, what, "pre_weight");
        x.pre_b = weights(a[12], k, what, "pre_bias");
        x.pre_eps = static_cast<float>(real(a[13]));
        if (a[16] != Py_None) {
            const at::Tensor &q = tensor(a[16], what, "out_q8_1");
            if (q.scalar_type() != at::kByte || q.dim() != 2 || q.size(0) != t || !q.is_contiguous() || q.size(1) != k / 32 * 36)
                refuse(what, "out_q8_1", "contiguous uint8 [tokens, k / 32 * 36]");
            x.z_q8_1 = q.data_ptr();
        }
        return PyLong_FromLong(api.norm(&x, stream(a[17])));
    }, ONE);
}

// cache, slots, n_kv_heads, head_dim, page, k, v, stream
PyObject *kv_get_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const char *what = "gguf_kv_get_rows";
        count(n, 8, what);
        const int64_t hk = integer(a[2]), d = integer(a[3]), page = integer(a[4]);
        const int64_t m = tensor(a[1], what, "slots").numel();
        const Pages c = pages(a[0], d, hk, page, what);
        const at::Tensor &k = tensor(a[5], what, "out"), &v = tensor(a[6], what, "out");
        if (k.scalar_type() != v.scalar_type() || !k.is_contiguous() || !v.is_contiguous() || k.numel() < m * hk * d ||
            v.numel() < m * hk * d)
            refuse(what, "out", "two contiguous tensors [n, kv_heads, d] of one dtype");
        return PyLong_FromLong(api.rows(c.p, c.n, page, hk, d, array<int64_t>(a[1], m, what, "slots"), m, k.data_ptr(),
                                        v.data_ptr(), float_type(k.scalar_type(), what), stream(a[7])));
    });
}

// of q, cache, n_kv_heads, page, max_q_len, scale, window, sinks, out, status
gguf_attn_args attn_args(PyObject *q_, PyObject *cache, PyObject *const *a, const char *what) {
    const at::Tensor &q = tensor(q_, what, "q");
    if (q.dim() != 3) refuse(what, "q", "[tokens, heads, head_dim]");
    gguf_attn_args x{};
    const at::ScalarType type = q.scalar_type();
    x.qt = float_type(type, what);
    x.n_tokens = q.size(0);
    x.n_heads = q.size(1);
    x.head_dim = q.size(2);
    x.n_kv_heads = integer(a[0]);
    x.page_size = integer(a[1]);
    x.max_q_len = integer(a[2]);
    x.scale = static_cast<float>(real(a[3]));
    x.window = integer(a[4]);
    x.sinks = integer(a[5]);
    Rows r = rows(q, x.n_tokens, x.n_heads, x.head_dim, type, what, "q");
    x.q = r.p;
    x.ldq = r.ld;
    r = rows(tensor(a[6], what, "out"), x.n_tokens, x.n_heads, x.head_dim, type, what, "out");
    x.out = r.p;
    x.ldo = r.ld;
    const Pages c = pages(cache, x.head_dim, x.n_kv_heads, x.page_size, what);
    x.cache = c.p;
    x.n_pages = c.n;
    x.dev_status = array_or_none<int32_t>(a[8], 1, what, "dev_status");
    return x;
}
struct Bytes {
    void *p;
    size_t n;
};
Bytes bytes_or_none(PyObject *o, const char *what, const char *name) {
    if (o == Py_None) return {nullptr, 0};
    const at::Tensor &w = tensor(o, what, name);
    if (!w.is_contiguous()) refuse(what, name, "contiguous");
    return {w.data_ptr(), static_cast<size_t>(w.numel() * w.element_size())};
}

// q, cache, table, q_start, kv_len, n_kv_heads, page, max_q_len, scale, window, sinks, out, ws, status, stream; with ws an
// int instead of a tensor, the bytes of workspace are returned and nothing runs
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const char *what = "gguf_paged_attention";
        count(n, 15, what);
        gguf_attn_args x = attn_args(a[0], a[1], a + 5, what);
        x.n_requests = tensor(a[4], what, "kv_len").numel();
        const Table t = table(a[2], x.n_requests, what);
        x.block_table = t.p;
        x.ld_table = t.ld;
        x.width = t.width;
        x.q_start = array<int32_t>(a[3], x.n_requests + 1, what, "q_start");
        x.kv_len = array<int32_t>(a[4], x.n_requests, what, "kv_len");
        if (PyLong_Check(a[12])) return PyLong_FromSize_t(api.attn_ws(&x));
        const Bytes w = bytes_or_none(a[12], what, "ws");
        return PyLong_FromLong(api.attn(&x, w.p, w.n, stream(a[14])));
    });
}

PyObject *status_or(gguf_status st, PyObject *made) {   // takes `made` over
    if (st == GGUF_OK) return made;
    Py_DECREF(made);
    return PyLong_FromLong(st);
}
at::Tensor bytes_like(const at::Tensor &t, int64_t n) { return at::empty({n}, t.options().dtype(at::kByte)); }

// q_start, kv_len, group_start, prefix_len, page, n_tokens, plan (None: it is made), stream
PyObject *prefix_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const char *what = "gguf_prefix_plan";
        count(n, 8, what);
        const at::Tensor &kv_len = tensor(a[1], what, "kv_len");
        const int64_t r = kv_len.numel(), groups = tensor(a[3], what, "prefix_len").numel(), tokens = integer(a[5]);
        at::Tensor made;
        Bytes plan = bytes_or_none(a[6], what, "plan");
        if (a[6] == Py_None) {
            made = bytes_like(kv_len, std::max<int64_t>(api.pplan_bytes(r, groups, tokens), 0));   // (the library refuses the sizes itself)
            plan = {made.data_ptr(), static_cast<size_t>(made.numel())};
        }
        const gguf_status st = api.pplan(array<int32_t>(a[0], r + 1, what, "q_start"), array<int32_t>(a[1], r, what, "kv_len"), r,
                                         array<int32_t>(a[2], groups + 1, what, "group_start"),
                                         array<int32_t>(a[3], groups, what, "prefix_len"), groups, integer(a[4]), tokens, plan.p, plan.n,
                                         stream(a[7]));
        if (a[6] != Py_None) Py_INCREF(a[6]);
        return status_or(st, a[6] != Py_None ? a[6] : THPVariable_Wrap(made));
    }, ONE);
}

// q, cache, table, plan, n_groups, n_kv_heads, page, max_q_len, scale, window, sinks, out, ws (None: they are made), status, stream
PyObject *prefix_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const char *what = "gguf_prefix_attention";
        count(n, 15, what);
        PyObject *args[9] = {a[5], a[6], a[7], a[8], a[9], a[10], a[11], nullptr, a[13]};
        struct Held {
            PyObject *p;
            ~Held() { Py_XDECREF(p); }
        } out{nullptr};
        if (a[11] == Py_None) {
            const at::Tensor &q = tensor(a[0], what, "q");
            out.p = THPVariable_Wrap(at::empty(q.sizes(), q.options()));
        } else {
            out.p = a[11];
            Py_INCREF(out.p);
        }
        args[6] = out.p;
        gguf_attn_args x = attn_args(a[0], a[1], args, what);
        const Table t = table(a[2], 0, what);
        x.n_requests = tensor(a[2], what, "block_table").size(0);
        x.block_table = t.p;
        x.ld_table = t.ld;
        x.width = t.width;
        const int64_t groups = integer(a[4]);
        const Bytes plan = bytes_or_none(a[3], what, "plan");
        Bytes w = bytes_or_none(a[12], what, "ws");
        at::Tensor made;
        if (a[12] == Py_None) {
            if (const size_t need = api.pattn_ws(&x, groups)) {
                made = bytes_like(THPVariable_Unpack(a[0]), static_cast<int64_t>(need));
                w = {made.data_ptr(), need};
            }
        }
        const gguf_status st = api.pattn(&x, plan.p, plan.n, groups, w.p, w.n, stream(a[14]));
        if (st != GGUF_OK) return PyLong_FromLong(st);
        Py_INCREF(out.p);
        return out.p;
    }, ONE);
}

// the addresses of gguf_kv_plan, gguf_qk_norm_rope, gguf_kv_get_rows, gguf_paged_attention_ws_size, gguf_paged_attention,
// gguf_kv_page_bytes, gguf_qk_norm_mrope, gguf_block_norm, gguf_prefix_plan, gguf_prefix_attention_ws_size,
// gguf_prefix_attention and gguf_prefix_plan_bytes
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 12, "bind");
        void *p[12];
        for (int i = 0; i < 12; i++) p[i] = reinterpret_cast<void *>(static_cast<intptr_t>(integer(a[i])));
        api = {reinterpret_cast<plan_fn>(p[0]), reinterpret_cast<rope_fn>(p[1]), reinterpret_cast<rows_fn>(p[2]),
               reinterpret_cast<attn_ws_fn>(p[3]), reinterpret_cast<attn_fn>(p[4]), reinterpret_cast<page_fn>(p[5]),
               reinterpret_cast<mrope_fn>(p[6]), reinterpret_cast<norm_fn>(p[7]), reinterpret_cast<pplan_fn>(p[8]),
               reinterpret_cast<pattn_ws_fn>(p[9]), reinterpret_cast<pattn_fn>(p[10]), reinterpret_cast<page_fn>(p[11])};
        Py_RETURN_NONE;
    });
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(kv_plan), FAST(qk_norm_rope), FAST(kv_get_rows), FAST(paged_attention),
                         FAST(qk_norm_mrope), FAST(block_norm), FAST(prefix_plan), FAST(prefix_attention),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
