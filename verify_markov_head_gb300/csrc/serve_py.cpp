// serve_py.cpp -- the serving operators as functions of a Python module: the
// tensors' types, shapes and layout are checked and the C function is called
// (include/dspark.h), whose status is returned.  A small call is over on the
// GPU before Python has looked at its tensors one attribute at a time.  Host
// time of a call on an Arm core, through ctypes before: plan of 64 requests
// 4.0 us (10.8), append 3.0 (7.3), attention 5.7 (13.9), logits 4.3 (13).
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>
#include <string>

#include "dspark.h"

namespace {

using at::Tensor;

struct PyRaised {};              // a Python exception is set

[[noreturn]] void fail(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw PyRaised{};
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t) {
    return t == at::kInt ? "torch.int32" : t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16" : c10::toString(t);
}

// Address of a contiguous tensor of the given type and shape (no extents: any shape).
template <typename... Extent>
void* typed(PyObject* o, const char* name, at::ScalarType type, Extent... extents) {
    const Tensor& t = tensor(o, name);
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
    if constexpr (sizeof...(extents) > 0) {
        const int64_t want[] = {(int64_t)extents...};
        bool ok = t.dim() == (int64_t)sizeof...(extents);
        for (size_t i = 0; ok && i < sizeof...(extents); ++i) ok = t.size(i) == want[i];
        if (!ok) {
            std::string s = std::string(name) + " must have shape (";
            for (int64_t w : want) s += std::to_string(w) + ", ";
            fail(PyExc_ValueError, s + ")");
        }
    }
    if (!t.is_contiguous()) fail(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t.data_ptr();
}
template <typename... Extent>
void* typed_or_null(PyObject* o, const char* name, at::ScalarType type, Extent... extents) {
    return o == Py_None ? nullptr : typed(o, name, type, extents...);
}

const Tensor& of_dim(PyObject* o, const char* name, int64_t dim) {
    const Tensor& t = tensor(o, name);
    if (t.dim() != dim) fail(PyExc_ValueError, std::string(name) + " must have " + std::to_string(dim) + " dimensions");
    return t;
}

dspark_dtype dtype_of(const Tensor& t) {
    if (t.scalar_type() == at::kFloat) return DSPARK_F32;
    if (t.scalar_type() == at::kBFloat16) return DSPARK_BF16;
    fail(PyExc_TypeError, std::string("unsupported dtype ") + type_name(t.scalar_type()));
}

// An extent as the C functions take it.
int extent(int64_t n) {
    if (n > INT_MAX) fail(PyExc_ValueError, "a tensor is too large");
    return (int)n;
}
int integer(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyRaised{};
    if (v < INT_MIN || v > INT_MAX) fail(PyExc_ValueError, "an integer is out of range");
    return (int)v;
}
float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyRaised{};
    return (float)v;
}

// None: the current stream of the current device; a stream object or a handle.
void* stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* handle = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!handle) throw PyRaised{};
    void* s = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!s && PyErr_Occurred()) throw PyRaised{};
    return s;
}

struct Cache {
    void* k; void* v;
    dspark_dtype type;
    at::ScalarType scalar;
    int64_t pages, heads, page_size, dim;
    long long page_stride;
};

// Two caches [pages, kv_heads, page_size, head_dim] whose pages are contiguous.
Cache caches(PyObject* ko, PyObject* vo) {
    const Tensor &k = of_dim(ko, "k_cache", 4), &v = of_dim(vo, "v_cache", 4);
    if (k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type() || k.strides() != v.strides())
        fail(PyExc_ValueError, "k_cache and v_cache must share shape, dtype and strides");
    Cache c{nullptr, nullptr, dtype_of(k), k.scalar_type(), k.size(0), k.size(1), k.size(2), k.size(3), 0};
    // (the stride of an extent of one says nothing)
    if ((c.dim > 1 && k.stride(3) != 1) || (c.page_size > 1 && k.stride(2) != c.dim) ||
        (c.heads > 1 && k.stride(1) != c.page_size * c.dim))
        fail(PyExc_ValueError, "a page of the cache must be contiguous [kv_heads, page_size, head_dim]");
    c.page_stride = c.pages > 1 ? k.stride(0) : c.heads * c.page_size * c.dim;
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    return c;
}

// Elements between tokens of t [T, heads, head_dim], whose tokens are contiguous.
long long token_stride(const Tensor& t, const char* name) {
    if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != t.size(2)))
        fail(PyExc_ValueError, std::string("the heads of a token of ") + name + " must be contiguous");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

void* workspace(PyObject* o, size_t* bytes) {
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(o, "ws");
    if (bytes) *bytes = t.nbytes();
    return t.data_ptr();
}

// The status that `body` returns as a Python number, or its exception.
template <typename Body>
PyObject* call(Py_ssize_t given, Py_ssize_t wanted, Body&& body) {
    try {
        if (given != wanted) fail(PyExc_TypeError, "wrong number of arguments");
        return PyLong_FromLong(body());
    } catch (const PyRaised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
#define DSPARK_UNLOCKED(st, expr) \
    dspark_status st;             \
    Py_BEGIN_ALLOW_THREADS st = expr; Py_END_ALLOW_THREADS

// seq_len, n_new, owned, ring, ring_state, block_table, page_size, owned_out, ring_state_out, kv_len, q_off,
// tile_off, slot_map, positions, ws, stream
PyObject* cache_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 16, [&]() {
        const Tensor& table = of_dim(a[5], "block_table", 2);
        const int64_t B = table.size(0), T = of_dim(a[12], "slot_map", 1).size(0);
        int32_t* p[14];
        const char* const names[14] = {"seq_len", "n_new", "owned", "ring", "ring_state", "block_table", "", "owned_out",
                                       "ring_state_out", "kv_len", "q_off", "tile_off", "slot_map", "positions"};
        const int64_t extents[14] = {B, B, B, 0, 2, 0, 0, B, 2, B, B + 1, B + 1, T, T};
        for (int i = 0; i < 14; ++i)
            if (i != 6)              // (the ring and the table: any shape, and the one that B was taken from)
                p[i] = static_cast<int32_t*>(i == 3 || i == 5 ? typed(a[i], names[i], at::kInt) : typed(a[i], names[i], at::kInt, extents[i]));
        const int b = extent(B), pages = extent(tensor(a[3], "ring").numel()), width = extent(table.size(1)), tokens = extent(T);
        const int page_size = integer(a[6]);
        void *ws = workspace(a[14], nullptr), *s = stream_of(a[15]);
        DSPARK_UNLOCKED(st, dspark_cache_plan(p[0], p[1], p[2], b, p[3], p[4], pages, p[5], width, page_size, p[7], p[8], p[9],
                                              p[10], p[11], p[12], p[13], tokens, ws, s));
        return st;
    });
}

// k, v, slot_map, k_cache, v_cache, ws, stream
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 7, [&]() {
        const Tensor &k = of_dim(a[0], "k", 3), &v = of_dim(a[1], "v", 3);
        const Cache c = caches(a[3], a[4]);
        if (v.sizes() != k.sizes() || c.heads != k.size(1) || c.dim != k.size(2) || k.scalar_type() != c.scalar || v.scalar_type() != c.scalar)
            fail(PyExc_ValueError, "k and v must be [T, kv_heads, head_dim] of the cache's heads and dtype");
        const long long ks = token_stride(k, "k"), vs = token_stride(v, "v");
        const int T = extent(k.size(0)), pages = extent(c.pages), P = extent(c.page_size), H = extent(c.heads), D = extent(c.dim);
        const auto* slots = static_cast<const int32_t*>(typed(a[2], "slot_map", at::kInt, k.size(0)));
        const void *kp = k.data_ptr(), *vp = v.data_ptr();
        void *ws = workspace(a[5], nullptr), *s = stream_of(a[6]);
        DSPARK_UNLOCKED(st, dspark_cache_append(kp, vp, c.type, ks, vs, slots, T, c.k, c.v, c.page_stride, pages, P, H, D, ws, s));
        return st;
    });
}

// q, k_cache, v_cache, block_table, kv_len, q_off, tile_off, out, ws, max_new, scale, lse, stream
PyObject* cache_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 13, [&]() {
        const Tensor &q = of_dim(a[0], "q", 3), &table = of_dim(a[3], "block_table", 2), &out = tensor(a[7], "out");
        const Cache c = caches(a[1], a[2]);
        if (c.dim != q.size(2) || q.scalar_type() != c.scalar || out.scalar_type() != c.scalar || out.sizes() != q.sizes())
            fail(PyExc_ValueError, "q and out must be [N, q_heads, head_dim] of the cache's head_dim and dtype");
        if (!out.is_contiguous()) fail(PyExc_ValueError, "tensors must be contiguous");
        const int64_t B = table.size(0), N = q.size(0), Hq = q.size(1);
        const long long qs = token_stride(q, "q");
        const auto* tab = static_cast<const int32_t*>(typed(a[3], "block_table", at::kInt));
        const auto* len = static_cast<const int32_t*>(typed(a[4], "kv_len", at::kInt, B));
        const auto* q_off = static_cast<const int32_t*>(typed(a[5], "q_off", at::kInt, B + 1));
        const auto* tile_off = static_cast<const int32_t*>(typed(a[6], "tile_off", at::kInt, B + 1));
        auto* lse = static_cast<float*>(typed_or_null(a[11], "lse", at::kFloat, N, Hq));
        const int b = extent(B), nn = extent(N), width = extent(table.size(1)), hq = extent(Hq), pages = extent(c.pages),
                  P = extent(c.page_size), H = extent(c.heads), D = extent(c.dim), max_new = integer(a[9]);
        const float scale = a[10] == Py_None ? (float)std::pow((double)D, -0.5) : number(a[10]);
        const void* qp = q.data_ptr();
        void* op = out.data_ptr();
        size_t bytes = 0;
        void *ws = workspace(a[8], &bytes), *s = stream_of(a[12]);
        DSPARK_UNLOCKED(st, dspark_cache_attention(qp, qs, c.k, c.v, c.type, c.page_stride, pages, P, tab, width, len, q_off, tile_off,
                                                   b, nn, hq, H, D, max_new, scale, op, lse, ws, bytes, s));
        return st;
    });
}

// logits, out, ws, hist, hist_len, prompt_len, draft_tok, rep, freq, pres, bias_tok, bias_val, bias_off, mask, fill, live, stream
PyObject* logits_process(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 17, [&]() {
        const Tensor &x = of_dim(a[0], "logits", 3), &out = tensor(a[1], "out");
        if (out.sizes() != x.sizes() || out.scalar_type() != x.scalar_type())
            fail(PyExc_ValueError, "out must have the logits' shape and dtype");
        const int64_t B = x.size(0), R = x.size(1), V = x.size(2);
        long long rs = R > 1 ? x.stride(1) : x.stride(0);
        if (x.stride(2) != 1 || (B > 1 && x.stride(0) != R * rs)) fail(PyExc_ValueError, "the rows of logits must lie at one stride");
        if (B * R == 1) rs = V;
        if (!out.is_contiguous()) fail(PyExc_ValueError, "tensors must be contiguous");
        const dspark_dtype type = dtype_of(x);
        int drafts = 0, past = 0, biases = 0;
        if (a[6] != Py_None) {
            const Tensor& d = tensor(a[6], "draft_tok");
            if (d.dim() != 2 || d.size(0) != B || d.size(1) < R - 1) fail(PyExc_ValueError, "draft_tok must be [B, R-1] or wider");
            drafts = extent(d.size(1));
        }
        if ((a[3] == Py_None) != (a[4] == Py_None)) fail(PyExc_ValueError, "hist and hist_len go together");
        PyObject *hist_o = a[3], *len_o = a[4], *prompt_o = a[5];
        if (hist_o != Py_None) {
            past = extent(of_dim(hist_o, "hist", 2).size(1));
            if (past == 0) hist_o = len_o = prompt_o = Py_None;      // no history yet
        }
        if (a[12] != Py_None) {
            const int64_t entries = tensor(a[10], "bias_tok").numel();
            if (tensor(a[11], "bias_val").numel() != entries) fail(PyExc_ValueError, "bias_tok and bias_val must have one entry each");
            biases = extent(entries);
        }
        const auto* hist = static_cast<const int32_t*>(typed_or_null(hist_o, "hist", at::kInt, B, past));
        const auto* len = static_cast<const int32_t*>(typed_or_null(len_o, "hist_len", at::kInt, B));
        const auto* prompt = static_cast<const int32_t*>(typed_or_null(prompt_o, "prompt_len", at::kInt, B));
        const auto* draft = static_cast<const int32_t*>(typed_or_null(a[6], "draft_tok", at::kInt));
        const auto* rep = static_cast<const float*>(typed_or_null(a[7], "rep", at::kFloat, B));
        const auto* freq = static_cast<const float*>(typed_or_null(a[8], "freq", at::kFloat, B));
        const auto* pres = static_cast<const float*>(typed_or_null(a[9], "pres", at::kFloat, B));
        const auto* bias_off = static_cast<const int32_t*>(typed_or_null(a[12], "bias_off", at::kInt, B + 1));
        const auto* bias_tok = bias_off ? static_cast<const int32_t*>(typed(a[10], "bias_tok", at::kInt)) : nullptr;
        const auto* bias_val = bias_off ? static_cast<const float*>(typed(a[11], "bias_val", at::kFloat)) : nullptr;
        const auto* mask = static_cast<const uint32_t*>(typed_or_null(a[13], "mask", at::kInt, B, R, (V + 31) / 32));
        auto* live = static_cast<int32_t*>(typed_or_null(a[15], "live", at::kInt, B, R));
        const float fill = number(a[14]);
        const int b = extent(B), r = extent(R), v = extent(V);
        const void* xp = x.data_ptr();
        void* op = out.data_ptr();
        size_t bytes = 0;
        void *ws = workspace(a[2], &bytes), *s = stream_of(a[16]);
        DSPARK_UNLOCKED(st, dspark_logits_process(xp, type, rs, op, b, r, v, hist, past, len, prompt, draft, drafts, rep, freq, pres,
                                                  bias_tok, bias_val, bias_off, biases, mask, fill, live, ws, bytes, s));
        return st;
    });
}

PyMethodDef methods[] = {
    {"cache_plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_plan)), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_append)), METH_FASTCALL, nullptr},
    {"cache_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_attention)), METH_FASTCALL, nullptr},
    {"logits_process", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(logits_process)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", "The serving operators of libdspark.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__serve() { return PyModule_Create(&module); }
