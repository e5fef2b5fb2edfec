// Native marshalling of the paged-cache calls (module _bind of the package):
// torch tensors -> pointers and strides of the C ABI, with the same argument
// rules as the ctypes binding of the other calls.  These calls stand between
// the products of every layer of a decode step, where the host's share of a
// small call is larger than the GPU's: a call costs about 0.7 us here beside
// the launch, and 5 to 10 us through ctypes.
//
// The functions take positional arguments, allocate nothing, and return the
// status of the C function that they call (whose address bind() got), or raise
// ValueError for a tensor that does not fit.
#include <Python.h>

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

struct {
    plan_fn plan;
    rope_fn rope;
    rows_fn rows;
    attn_ws_fn attn_ws;
    attn_fn attn;
    page_fn page_bytes;
} api;

struct Bad {};   // a Python exception is set

[[noreturn]] void refuse(const char *what, const char *name, const char *want) {
    PyErr_Format(PyExc_ValueError, "%s: %s must be %s", what, name, want);
    throw Bad();
}
const at::Tensor &tensor(PyObject *o, const char *what, const char *name) {
    if (!THPVariable_Check(o)) refuse(what, name, "a tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) {
        PyErr_SetString(PyExc_ValueError, "gguf: tensors must live on a CUDA device");
        throw Bad();
    }
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
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const Bad &) {
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
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const char *what = "gguf_qk_norm_rope";
        count(n, 16, what);
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
        x.positions = array<int32_t>(a[6], t, what, "positions");
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
        return PyLong_FromLong(api.rope(&x, stream(a[15])));
    });
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

// q, cache, table, q_start, kv_len, n_kv_heads, page, max_q_len, scale, window, sinks, out, ws, status, stream; with ws an
// int instead of a tensor, the bytes of workspace are returned and nothing runs
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        const char *what = "gguf_paged_attention";
        count(n, 15, what);
        const at::Tensor &q = tensor(a[0], what, "q");
        if (q.dim() != 3) refuse(what, "q", "[tokens, heads, head_dim]");
        gguf_attn_args x{};
        const at::ScalarType type = q.scalar_type();
        x.qt = float_type(type, what);
        x.n_tokens = q.size(0);
        x.n_heads = q.size(1);
        x.head_dim = q.size(2);
        x.n_kv_heads = integer(a[5]);
        x.page_size = integer(a[6]);
        x.max_q_len = integer(a[7]);
        x.scale = static_cast<float>(real(a[8]));
        x.window = integer(a[9]);
        x.sinks = integer(a[10]);
        Rows r = rows(q, x.n_tokens, x.n_heads, x.head_dim, type, what, "q");
        x.q = r.p;
        x.ldq = r.ld;
        r = rows(tensor(a[11], what, "out"), x.n_tokens, x.n_heads, x.head_dim, type, what, "out");
        x.out = r.p;
        x.ldo = r.ld;
        const Pages c = pages(a[1], x.head_dim, x.n_kv_heads, x.page_size, what);
        x.cache = c.p;
        x.n_pages = c.n;
        x.n_requests = tensor(a[4], what, "kv_len").numel();
        const Table t = table(a[2], x.n_requests, what);
        x.block_table = t.p;
        x.ld_table = t.ld;
        x.width = t.width;
        x.q_start = array<int32_t>(a[3], x.n_requests + 1, what, "q_start");
        x.kv_len = array<int32_t>(a[4], x.n_requests, what, "kv_len");
        x.dev_status = array_or_none<int32_t>(a[13], 1, what, "dev_status");
        if (PyLong_Check(a[12])) return PyLong_FromSize_t(api.attn_ws(&x));
        void *ws = nullptr;
        size_t bytes = 0;
        if (a[12] != Py_None) {
            const at::Tensor &w = tensor(a[12], what, "ws");
            if (!w.is_contiguous()) refuse(what, "ws", "contiguous");
            ws = w.data_ptr();
            bytes = w.numel() * w.element_size();
        }
        return PyLong_FromLong(api.attn(&x, ws, bytes, stream(a[14])));
    });
}

// the addresses of gguf_kv_plan, gguf_qk_norm_rope, gguf_kv_get_rows, gguf_paged_attention_ws_size, gguf_paged_attention
// and gguf_kv_page_bytes
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 6, "bind");
        void *p[6];
        for (int i = 0; i < 6; i++) p[i] = reinterpret_cast<void *>(static_cast<intptr_t>(integer(a[i])));
        api = {reinterpret_cast<plan_fn>(p[0]), reinterpret_cast<rope_fn>(p[1]), reinterpret_cast<rows_fn>(p[2]),
               reinterpret_cast<attn_ws_fn>(p[3]), reinterpret_cast<attn_fn>(p[4]), reinterpret_cast<page_fn>(p[5])};
        Py_RETURN_NONE;
    });
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(kv_plan), FAST(qk_norm_rope), FAST(kv_get_rows), FAST(paged_attention),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
