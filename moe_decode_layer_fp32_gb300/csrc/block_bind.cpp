// Python entry points of the decode-block calls (include/moe_block.h): they
// read pointers, types, sizes and strides from the tensors, check that they fit one
// another, and call the C ABI on the current stream.  A decode step makes such a call
// every few microseconds; the same marshalling through ctypes took 7 to 12 us a
// call on the GB300's host, and takes 2.7 to 3.1 here, most of it the launch.
//
// The functions' addresses come from the loaded library (bind()), and a call's error
// code goes to the Python function given there, which raises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe_block.h"

namespace {

decltype(&moe_rmsnorm) g_rmsnorm = nullptr;
decltype(&moe_kv_append) g_append = nullptr;
decltype(&moe_attn_decode) g_attn = nullptr;
decltype(&moe_lora_project) g_lora = nullptr;
PyObject* g_on_error = nullptr;      // (name, code) -> raises
PyTypeObject* g_cache_type = nullptr;
PyObject* g_address = nullptr;       // "address"

// A ValueError has been set.
struct Refused {};

[[noreturn]] void refuse(const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(PyExc_ValueError, fmt, ap);
    va_end(ap);
    throw Refused();
}

// What a call reads and writes has to be on the current device, on whose stream it runs.
thread_local int t_device;           // -1: not asked yet in this call
void check_device(int device, const char* name) {
    if (t_device < 0) t_device = c10::cuda::current_device();
    if (device != t_device) refuse("%s: on device %d, but the current one is %d", name, device, t_device);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse("%s: expected a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse("%s: expected a CUDA tensor", name);
    check_device(t.get_device(), name);
    return t;
}

// A size as the C ABI takes it.
int size32(int64_t n, const char* name) {
    if (n > INT_MAX) refuse("%s: a size of %lld does not fit 32 bits", name, (long long)n);
    return (int)n;
}

int code_of(const at::Tensor& t, const char* name) {
    switch (t.scalar_type()) {
        case at::kFloat: return MOE_DTYPE_F32;
        case at::kBFloat16: return MOE_DTYPE_BF16;
        case at::kFloat8_e4m3fn: return MOE_DTYPE_FP8_E4M3;
        default: refuse("%s: unsupported dtype", name);
    }
}

struct Rows {
    void* p;
    int code;
    int64_t ld;
};
// A matrix [rows, cols] with contiguous rows (a single row's stride means nothing).
Rows rows(PyObject* o, const char* name, int64_t r, int64_t c) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2 || t.size(0) != r || t.size(1) != c)
        refuse("%s: expected shape [%lld, %lld]", name, (long long)r, (long long)c);
    if (t.stride(1) != 1 && c != 1) refuse("%s: expected contiguous rows", name);
    return {t.data_ptr(), code_of(t, name), r > 1 ? t.stride(0) : c};
}

struct Heads {
    void* p;
    int code;
    int64_t outer, inner;
};
// [T, heads, D] with contiguous rows (the stride of a single token or head means nothing).
Heads heads(PyObject* o, const char* name, int64_t T, int64_t h, int64_t D) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 3 || t.size(0) != T || t.size(1) != h || t.size(2) != D)
        refuse("%s: expected shape [%lld, %lld, %lld]", name, (long long)T, (long long)h, (long long)D);
    if (t.stride(2) != 1 && D != 1) refuse("%s: expected contiguous rows", name);
    return {t.data_ptr(), code_of(t, name), T > 1 ? t.stride(0) : h * D, h > 1 ? t.stride(1) : D};
}

// A contiguous tensor of this type and shape; None is nullptr.
void* exactly(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    if (o == nullptr || o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) {
        const std::string want = c10::str(type, " ", shape);
        refuse("%s: expected a contiguous tensor %s", name, want.c_str());
    }
    return t.data_ptr();
}

struct Table {
    const int32_t* p;
    int64_t ld;
    int R, pages;
};
Table table(PyObject* o) {
    const at::Tensor& t = tensor(o, "block_table");
    if (t.dim() != 2 || t.scalar_type() != at::kInt || (t.size(1) > 1 && t.stride(1) != 1))
        refuse("block_table: expected int32 [requests, pages] with contiguous rows");
    return {static_cast<const int32_t*>(t.data_ptr()), t.size(0) > 1 ? t.stride(0) : t.size(1),
            size32(t.size(0), "block_table"), size32(t.size(1), "block_table")};
}

struct Workspace {
    void* p;
    size_t bytes;
};
Workspace workspace(PyObject* o) {
    const at::Tensor& t = tensor(o, "ws");
    if (!t.is_contiguous()) refuse("ws: expected a contiguous tensor");
    return {t.data_ptr(), t.nbytes()};
}

struct CacheHandle {                 // KvCacheHandle of binding.py
    moe_kv_cache cache;
    int device;
};
const moe_kv_cache* cache_of(PyObject* o) {
    if (!PyObject_TypeCheck(o, g_cache_type)) refuse("cache: expected a KvCache");
    PyObject* a = PyObject_GetAttr(o, g_address);
    if (!a) throw Refused();
    auto* c = static_cast<const CacheHandle*>(PyLong_AsVoidPtr(a));
    Py_DECREF(a);
    if (!c) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "cache: no address");
        throw Refused();
    }
    check_device(c->device, "cache");
    return &c->cache;
}

double number(PyObject* o, double otherwise) {
    if (!o) return otherwise;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}
int integer(PyObject* o, int otherwise) {
    if (!o) return otherwise;
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    if (v > INT_MAX || v < INT_MIN) refuse("an argument does not fit 32 bits");
    return (int)v;
}
bool given(PyObject* o) { return o != nullptr && o != Py_None; }

void* stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

// Positional and keyword arguments into slots; the first `needed` must be there.
template <int N>
struct Signature {
    const char* fn;
    const char* names[N];
    int needed;
    PyObject* interned[N] = {};
    void parse(PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames, PyObject* (&out)[N]) {
        if (!interned[0])
            for (int i = 0; i < N; ++i) interned[i] = PyUnicode_InternFromString(names[i]);
        if (nargs > N) wrong("takes at most %d arguments", N);
        for (int i = 0; i < N; ++i) out[i] = i < nargs ? args[i] : nullptr;
        const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t k = 0; k < nk; ++k) {
            PyObject* key = PyTuple_GET_ITEM(kwnames, k);
            int at = -1;
            for (int i = 0; i < N && at < 0; ++i)
                if (key == interned[i]) at = i;
            for (int i = 0; i < N && at < 0; ++i)
                if (PyUnicode_Compare(key, interned[i]) == 0) at = i;
            if (at < 0) wrong("got an unexpected keyword argument");
            if (out[at]) wrong("got two values for '%s'", names[at]);
            out[at] = args[nargs + k];
        }
        for (int i = 0; i < needed; ++i)
            if (!out[i]) wrong("needs '%s'", names[i]);
    }
    template <class... A>
    [[noreturn]] void wrong(const char* fmt, A... a) {
        PyObject* m = PyUnicode_FromFormat(fmt, a...);
        if (m) {
            PyErr_Format(PyExc_TypeError, "%s() %U", fn, m);
            Py_DECREF(m);
        }
        throw Refused();
    }
};

PyObject* done(const char* name, int rc) {
    if (rc == MOE_OK) Py_RETURN_NONE;
    PyObject* r = PyObject_CallFunction(g_on_error, "si", name, rc);
    Py_XDECREF(r);
    if (r) PyErr_Format(PyExc_RuntimeError, "%s failed: %d", name, rc);
    return nullptr;
}

// Runs f; what it throws becomes a Python exception.
template <class F>
PyObject* guarded(F f) {
    t_device = -1;
    try {
        return f();
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* py_rmsnorm(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    static Signature<7> sig = {"moe_rmsnorm", {"x", "weight", "eps", "y", "residual", "residual_out", "y_scale"}, 4};
    return guarded([&] {
        PyObject* a[7];
        sig.parse(args, nargs, kwnames, a);
        const at::Tensor& xt = tensor(a[0], "x");
        if (xt.dim() != 2) refuse("x: expected [T, d]");
        const int T = size32(xt.size(0), "x"), d = size32(xt.size(1), "x");
        const Rows x = rows(a[0], "x", T, d), y = rows(a[3], "y", T, d);
        Rows r = {nullptr, 0, 0}, ro = {nullptr, 0, 0};
        if (given(a[4])) r = rows(a[4], "residual", T, d);
        if (given(a[5])) ro = rows(a[5], "residual_out", T, d);
        if (r.p && ro.p && r.code != ro.code) refuse("residual and residual_out must have one dtype");
        void* w = nullptr;
        int w_code = 0;
        if (given(a[1])) {
            const at::Tensor& t = tensor(a[1], "weight");
            w_code = code_of(t, "weight");
            w = exactly(a[1], "weight", t.scalar_type(), {d});
        }
        void* s = nullptr;
        int group = 0;
        if (given(a[6])) {
            if (tensor(a[6], "y_scale").dim() == 2) {
                group = 128;
                s = exactly(a[6], "y_scale", at::kFloat, {T, d / 128});
            } else {
                s = exactly(a[6], "y_scale", at::kFloat, {T});
            }
        }
        return done("moe_rmsnorm", g_rmsnorm(x.p, x.code, x.ld, r.p, r.p ? r.code : ro.code, r.ld, ro.p, ro.ld, w, w_code,
                                             (float)number(a[2], 0.0), T, d, y.p, y.code, y.ld,
                                             static_cast<float*>(s), group, stream()));
    });
}

PyObject* py_append(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    static Signature<10> sig = {"moe_kv_append",
                                {"k", "v", "cache", "block_table", "positions", "req", "cos_sin", "q", "q_out", "status"}, 5};
    return guarded([&] {
        PyObject* a[10];
        sig.parse(args, nargs, kwnames, a);
        const moe_kv_cache* c = cache_of(a[2]);
        const at::Tensor& kt = tensor(a[0], "k");
        if (kt.dim() != 3) refuse("k: expected [T, heads, D]");
        const int T = size32(kt.size(0), "k"), D = c->head_dim;
        const Heads k = heads(a[0], "k", T, c->heads, D), v = heads(a[1], "v", T, c->heads, D);
        if (k.code != v.code) refuse("k and v must have one dtype");
        Heads q = {nullptr, 0, 0, 0}, o = {nullptr, 0, 0, 0};
        int hq = 0;
        if (given(a[7]) != given(a[8])) refuse("q and q_out go together");
        if (given(a[7])) {
            const at::Tensor& qt = tensor(a[7], "q");
            if (qt.dim() != 3) refuse("q: expected [T, q_heads, D]");
            hq = size32(qt.size(1), "q");
            q = heads(a[7], "q", T, hq, D);
            o = heads(a[8], "q_out", T, hq, D);
            if (q.code != k.code || o.code != k.code) refuse("q, q_out and k must have one dtype");
        }
        const float* cs = nullptr;
        int max_pos = 0, rot = 0;
        if (given(a[6])) {
            const at::Tensor& t = tensor(a[6], "cos_sin");
            if (t.dim() != 2) refuse("cos_sin: expected [positions, rot]");
            max_pos = size32(t.size(0), "cos_sin");
            rot = size32(t.size(1), "cos_sin");
            cs = static_cast<const float*>(exactly(a[6], "cos_sin", at::kFloat, {max_pos, rot}));
        }
        const Table t = table(a[3]);
        auto* pos = static_cast<const int32_t*>(exactly(a[4], "positions", at::kInt, {T}));
        auto* req = static_cast<const int32_t*>(exactly(a[5], "req", at::kInt, {T}));
        auto* st = static_cast<int32_t*>(exactly(a[9], "status", at::kInt, {1}));
        return done("moe_kv_append",
                    g_append(k.p, k.outer, k.inner, v.p, v.outer, v.inner, k.code, T, c, t.p, t.ld, t.R, t.pages, pos, req,
                             cs, rot, max_pos, q.p, q.outer, q.inner, o.p, o.outer, o.inner, hq, st, stream()));
    });
}

PyObject* py_attn(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    static Signature<10> sig = {
        "moe_attn_decode", {"q", "cache", "block_table", "seq_lens", "scale", "out", "ws", "window", "softcap", "lse"}, 7};
    return guarded([&] {
        PyObject* a[10];
        sig.parse(args, nargs, kwnames, a);
        const moe_kv_cache* c = cache_of(a[1]);
        const at::Tensor& qt = tensor(a[0], "q");
        if (qt.dim() != 3) refuse("q: expected [B, q_heads, D]");
        const int B = size32(qt.size(0), "q"), hq = size32(qt.size(1), "q"), D = c->head_dim;
        const Heads q = heads(a[0], "q", B, hq, D), o = heads(a[5], "out", B, hq, D);
        const Table t = table(a[2]);
        if (t.R != B) refuse("block_table must have a row per request");
        auto* lens = static_cast<const int32_t*>(exactly(a[3], "seq_lens", at::kInt, {B}));
        auto* lse = static_cast<float*>(exactly(a[9], "lse", at::kFloat, {B, hq}));
        const Workspace ws = workspace(a[6]);
        return done("moe_attn_decode",
                    g_attn(q.p, q.code, q.outer, q.inner, B, hq, c, t.p, t.ld, t.pages, lens, (float)number(a[4], 0.0),
                           integer(a[7], 0), (float)number(a[8], 0.0), o.p, o.code, o.outer, o.inner, lse, ws.p, ws.bytes,
                           stream()));
    });
}

PyObject* py_lora(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    static Signature<8> sig = {"moe_lora_project", {"x", "w", "y", "ws", "lora", "adapter", "x_scale", "w_scale"}, 4};
    return guarded([&] {
        PyObject* a[8];
        sig.parse(args, nargs, kwnames, a);
        const at::Tensor &xt = tensor(a[0], "x"), &wt = tensor(a[1], "w");
        if (xt.dim() != 2 || wt.dim() != 2) refuse("x must be [T, d] and w [N, d]");
        const int T = size32(xt.size(0), "x"), d = size32(xt.size(1), "x"), N = size32(wt.size(0), "w");
        const Rows x = rows(a[0], "x", T, d), w = rows(a[1], "w", N, d), y = rows(a[2], "y", T, N);
        void *la = nullptr, *lb = nullptr, *ls = nullptr, *ad = nullptr;
        int n = 0, r = 0;
        if (given(a[4])) {
            if (!PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != 3) refuse("lora: expected a tuple (A, B, scale)");
            PyObject* A = PyTuple_GET_ITEM(a[4], 0);
            const at::Tensor& at_ = tensor(A, "lora A");
            if (at_.dim() != 3) refuse("lora A: expected [adapters, r, d]");
            n = size32(at_.size(0), "lora A");
            r = size32(at_.size(1), "lora A");
            la = exactly(A, "lora A", at::kBFloat16, {n, r, d});
            lb = exactly(PyTuple_GET_ITEM(a[4], 1), "lora B", at::kBFloat16, {n, N, r});
            ls = exactly(PyTuple_GET_ITEM(a[4], 2), "lora scale", at::kFloat, {n});
            ad = exactly(a[5], "adapter", at::kInt, {T});
        } else if (given(a[5])) {
            refuse("adapter without lora");
        }
        auto* xs = static_cast<const float*>(exactly(a[6], "x_scale", at::kFloat, {T}));
        auto* wsc = static_cast<const float*>(exactly(a[7], "w_scale", at::kFloat, {N}));
        const Workspace ws = workspace(a[3]);
        return done("moe_lora_project",
                    g_lora(x.p, x.code, x.ld, xs, T, d, w.p, w.code, w.ld, wsc, N, la, lb,
                           static_cast<const float*>(ls), n, r, static_cast<const int32_t*>(ad), y.p, y.code, y.ld,
                           ws.p, ws.bytes, stream()));
    });
}

// bind(rmsnorm, kv_append, attn_decode, lora_project, on_error, cache type): addresses of the library's
// functions, what raises for an error code, and the class of caches.
PyObject* py_bind(PyObject*, PyObject* args) {
    unsigned long long f[4];
    PyObject *on_error, *cache_type;
    if (!PyArg_ParseTuple(args, "KKKKOO!", &f[0], &f[1], &f[2], &f[3], &on_error, &PyType_Type, &cache_type)) return nullptr;
    g_rmsnorm = reinterpret_cast<decltype(g_rmsnorm)>(f[0]);
    g_append = reinterpret_cast<decltype(g_append)>(f[1]);
    g_attn = reinterpret_cast<decltype(g_attn)>(f[2]);
    g_lora = reinterpret_cast<decltype(g_lora)>(f[3]);
    Py_INCREF(on_error);
    Py_XSETREF(g_on_error, on_error);
    Py_INCREF(cache_type);
    Py_XSETREF(g_cache_type, reinterpret_cast<PyTypeObject*>(cache_type));
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS
PyMethodDef kMethods[] = {
    {"moe_rmsnorm", FAST(py_rmsnorm), "moe_rmsnorm of include/moe_block.h"},
    {"moe_kv_append", FAST(py_append), "moe_kv_append of include/moe_block.h"},
    {"moe_attn_decode", FAST(py_attn), "moe_attn_decode of include/moe_block.h"},
    {"moe_lora_project", FAST(py_lora), "moe_lora_project of include/moe_block.h"},
    {"bind", py_bind, METH_VARARGS, "addresses of the library's functions, and what they need of Python"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_block_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_bind() {
    g_address = PyUnicode_InternFromString("address");
    return PyModule_Create(&kModule);
}
