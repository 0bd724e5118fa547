// The ordinary calls of decoder.py without Python's share of the time, as
// attn_marshal.cpp does it for attention.py: each function returns its
// results, or None for anything it does not take as it stands (another type
// or layout than the ABI describes, another GPU than the current one, a call
// that the library declines), which decoder.py then checks and reports.
#include "marshal.hpp"

#include <torch/csrc/Dtype.h>

#include <cmath>
#include <cstring>
#include <vector>

#include "igemm_decoder.h"

namespace {

// Entries of one loaded library (decoder.py's _entries).
struct Entries {
    int32_t (*ln_fwd)(const igc_layer_norm*, void*);
    int32_t (*ln_bwd)(const igc_layer_norm*, void*);
    size_t (*ln_bwd_ws)(const igc_layer_norm*);
    int32_t (*quant)(const igc_quantize_rows*, void*);
    int32_t (*linear)(const igc_linear_i8*, void*);
    int32_t (*cache_write)(const igc_kv_io*, void*);
    int32_t (*cache_read)(const igc_kv_io*, void*);
    int32_t (*cache_attn)(const igc_cache_attn*, void*);
    size_t (*cache_attn_ws)(const igc_cache_attn*);
};
constexpr int kEntries = 9;
constexpr const char* kCapsule = "igc_decoder_entries";

const Entries& entries(PyObject* o) {
    void* p = PyCapsule_GetPointer(o, kCapsule);
    if (!p) {
        PyErr_Clear();
        no();
    }
    return *static_cast<Entries*>(p);
}

// A number of Python's (one that is none is Python's to report).
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) no();
    return v;
}
int64_t whole(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) no();
    return v;
}

// Rows of a tensor [..., C] of one to four axes: its view, and its sizes.
igc_attn_view rows(const at::Tensor& t, int64_t n[3], int64_t* c) {
    const int64_t dim = t.dim();
    if (dim < 1 || dim > 4) no();
    *c = t.size(dim - 1);
    if (t.stride(dim - 1) != 1 && *c > 1) no();
    int64_t s[3] = {0, 0, 0};
    n[0] = n[1] = n[2] = 1;
    for (int64_t i = 0; i < dim - 1; ++i) {
        n[4 - dim + i] = t.size(i);
        s[4 - dim + i] = t.stride(i);
    }
    return {t.data_ptr(), s[0], s[1], s[2]};
}

// A 16-bit tensor of rows on the current GPU.
const at::Tensor& rows_on_gpu(PyObject* o, int64_t device) {
    const at::Tensor& t = tensor(o);
    if (!t.is_cuda() || t.get_device() != device || t.layout() != at::kStrided) no();
    type_code(t.scalar_type());
    return t;
}

igc_layer_norm ln_args(const at::Tensor& x, PyObject* weight, PyObject* eps, int64_t device) {
    igc_layer_norm a{};
    a.dtype = type_code(x.scalar_type());
    a.x = rows(x, a.n, &a.channels);
    if (given(weight)) a.weight = dense<float>(weight, at::kFloat, device, {a.channels});
    a.eps = number(eps);
    return a;
}

// (entries, x, weight, bias, eps, stream, device)
PyObject* layer_norm(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 7) no();
        const Entries& e = entries(o[0]);
        const int64_t device = whole(o[6]);
        const at::Tensor& x = rows_on_gpu(o[1], device);
        igc_layer_norm a = ln_args(x, o[2], o[4], device);
        if (given(o[3])) a.bias = dense<float>(o[3], at::kFloat, device, {a.channels});
        at::Tensor out = fresh(x);
        a.out = rows(out, a.n, &a.channels);
        if (e.ln_fwd(&a, PyLong_AsVoidPtr(o[5])) != 1) no();
        return THPVariable_Wrap(out);
    });
}

// (entries, dy, x, weight, eps, stream, device)
PyObject* layer_norm_bwd(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 7) no();
        const Entries& e = entries(o[0]);
        const int64_t device = whole(o[6]);
        const at::Tensor &g = rows_on_gpu(o[1], device), &x = rows_on_gpu(o[2], device);
        if (g.scalar_type() != x.scalar_type() || g.sizes() != x.sizes()) no();
        igc_layer_norm a = ln_args(x, o[3], o[4], device);
        a.grad = rows(g, a.n, &a.channels);
        at::Tensor dx = fresh(x), dw = floats(x, {a.channels}), db = floats(x, {a.channels}), ws;
        a.out = rows(dx, a.n, &a.channels);
        a.dweight = static_cast<float*>(dw.data_ptr());
        a.dbias = static_cast<float*>(db.data_ptr());
        if (const size_t need = e.ln_bwd_ws(&a)) {
            ws = bytes(x, need);
            a.workspace = ws.data_ptr();
            a.workspace_bytes = need;
        }
        if (e.ln_bwd(&a, PyLong_AsVoidPtr(o[5])) != 1) no();
        return wrap({dx, dw, db});
    });
}

// (entries, x, stream, device)
PyObject* quantize_rows(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 4) no();
        const Entries& e = entries(o[0]);
        const at::Tensor& x = rows_on_gpu(o[1], whole(o[3]));
        igc_quantize_rows a{};
        a.dtype = type_code(x.scalar_type());
        a.x = rows(x, a.n, &a.channels);
        const int64_t pitch = (a.channels + 15) / 16 * 16, last = x.dim() - 1;
        std::vector<int64_t> sizes(x.sizes().begin(), x.sizes().end());
        sizes[last] = pitch;
        at::Tensor q = at::empty(sizes, x.options().dtype(at::kChar));
        sizes.pop_back();
        at::Tensor scale = floats(x, sizes);
        a.q = {q.data_ptr(), a.n[1] * a.n[2] * pitch, a.n[2] * pitch, pitch};
        a.scale = static_cast<float*>(scale.data_ptr());
        if (e.quant(&a, PyLong_AsVoidPtr(o[2])) != 1) no();
        return wrap({pitch == a.channels ? q : q.narrow(last, 0, a.channels), scale});
    });
}

// An int8 matrix whose rows lie one pitch apart (decoder.py's _matrix).
const at::Tensor& matrix(PyObject* o, int64_t device, int64_t* m, int64_t* k, int64_t* pitch) {
    const at::Tensor& t = tensor(o);
    if (!t.is_cuda() || t.get_device() != device || t.scalar_type() != at::kChar || t.dim() < 1 ||
        t.layout() != at::kStrided)
        no();
    const int64_t last = t.dim() - 1;
    *k = t.size(last);
    if (t.stride(last) != 1 && *k > 1) no();
    *m = 1;
    *pitch = -1;
    for (int64_t i = last - 1; i >= 0; --i) {
        if (t.size(i) != 1 && *m) {
            if (*pitch < 0) *pitch = t.stride(i);
            else if (t.stride(i) != *pitch * *m) no();
        }
        *m *= t.size(i);
    }
    const int64_t k16 = (*k + 15) / 16 * 16;
    if (*pitch < 0) *pitch = k16;
    if (*m && *k % 16 &&
        t.storage_offset() + (*m - 1) * *pitch + k16 > (int64_t)t.storage().nbytes())
        no();
    return t;
}

// (entries, x, x_scale, w, w_scale, bias, dtype, stream, device)
PyObject* linear_i8(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 9 || !THPDtype_Check(o[6])) no();
        const Entries& e = entries(o[0]);
        const int64_t device = whole(o[8]);
        const at::ScalarType type = reinterpret_cast<THPDtype*>(o[6])->scalar_type;
        igc_linear_i8 a{};
        a.dtype = type_code(type);
        const at::Tensor& x = matrix(o[1], device, &a.m, &a.k, &a.x_pitch);
        int64_t wk = 0;
        const at::Tensor& w = matrix(o[3], device, &a.n, &wk, &a.w_pitch);
        if (w.dim() != 2 || wk != a.k) no();
        std::vector<int64_t> sizes(x.sizes().begin(), x.sizes().end());
        sizes.pop_back();
        a.x_scale = dense<float>(o[2], at::kFloat, device, sizes);
        a.w_scale = dense<float>(o[4], at::kFloat, device, {a.n});
        if (given(o[5])) a.bias = dense<float>(o[5], at::kFloat, device, {a.n});
        sizes.push_back(a.n);
        at::Tensor y = at::empty(sizes, x.options().dtype(type));
        a.x = static_cast<const int8_t*>(x.data_ptr());
        a.w = static_cast<const int8_t*>(w.data_ptr());
        a.y = y.data_ptr();
        a.y_pitch = a.n;
        if (e.linear(&a, PyLong_AsVoidPtr(o[7])) != 1) no();
        return THPVariable_Wrap(y);
    });
}

// The cache as KVCache packed it (its tensors are on `device`).
igc_kv_cache cache_of(PyObject* packed) {
    igc_kv_cache c;
    if (!PyBytes_Check(packed) || PyBytes_GET_SIZE(packed) != (Py_ssize_t)sizeof(c)) no();
    std::memcpy(&c, PyBytes_AS_STRING(packed), sizeof(c));
    return c;
}

const int32_t* page_table(PyObject* o, int64_t device, int64_t batch, int64_t* stride,
                          int64_t* entries) {
    const at::Tensor& t = on_gpu(o, at::kInt, device, 2);
    if (t.size(0) != batch || (t.stride(1) != 1 && t.size(1) > 1)) no();
    *stride = t.stride(0);
    *entries = t.size(1);
    return static_cast<const int32_t*>(t.data_ptr());
}

// (entries, cache, k, v, table, start, lens, stream, device)
PyObject* kv_cache_write(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 9) no();
        const Entries& e = entries(o[0]);
        const int64_t device = whole(o[8]);
        igc_kv_io a{};
        a.cache = cache_of(o[1]);
        const at::ScalarType type = tensor(o[2]).scalar_type();
        a.dtype = type_code(type);
        const at::Tensor &k = on_gpu(o[2], type, device, 4), &v = on_gpu(o[3], type, device, 4);
        if (k.sizes() != v.sizes() || k.size(2) != a.cache.kv_heads ||
            k.size(3) != a.cache.head_dim)
            no();
        a.batch = k.size(0);
        a.tokens = k.size(1);
        a.k = view(k);
        a.v = view(v);
        a.table = page_table(o[4], device, a.batch, &a.table_stride, &a.table_entries);
        a.start = dense<int32_t>(o[5], at::kInt, device, {a.batch});
        if (given(o[6])) a.lens = dense<int32_t>(o[6], at::kInt, device, {a.batch});
        if (e.cache_write(&a, PyLong_AsVoidPtr(o[7])) != 1) no();
        Py_RETURN_TRUE;
    });
}

// (entries, cache, table, start, tokens, lens, dtype, stream, device)
PyObject* kv_cache_read(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 9 || !THPDtype_Check(o[6])) no();
        const Entries& e = entries(o[0]);
        const int64_t device = whole(o[8]);
        const at::ScalarType type = reinterpret_cast<THPDtype*>(o[6])->scalar_type;
        igc_kv_io a{};
        a.cache = cache_of(o[1]);
        a.dtype = type_code(type);
        const at::Tensor& table = on_gpu(o[2], at::kInt, device, 2);
        a.batch = table.size(0);
        a.tokens = whole(o[4]);
        if (a.tokens < 0) no();
        a.table = page_table(o[2], device, a.batch, &a.table_stride, &a.table_entries);
        a.start = dense<int32_t>(o[3], at::kInt, device, {a.batch});
        if (given(o[5])) a.lens = dense<int32_t>(o[5], at::kInt, device, {a.batch});
        at::Tensor k = at::empty({a.batch, a.tokens, a.cache.kv_heads, a.cache.head_dim},
                                 table.options().dtype(type));
        at::Tensor v = at::empty_like(k);
        a.k = view(k);
        a.v = view(v);
        if (e.cache_read(&a, PyLong_AsVoidPtr(o[7])) != 1) no();
        return wrap({k, v});
    });
}

// (entries, q, cache, table, lens, causal, scale, return_lse, stream, device)
PyObject* cache_attention(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 10) no();
        const Entries& e = entries(o[0]);
        const int64_t device = whole(o[9]);
        igc_cache_attn a{};
        a.cache = cache_of(o[2]);
        const at::ScalarType type = tensor(o[1]).scalar_type();
        a.dtype = type_code(type);
        const at::Tensor& q = on_gpu(o[1], type, device, 4);
        if (q.size(3) != a.cache.head_dim) no();
        a.batch = q.size(0);
        a.q_len = q.size(1);
        a.q_heads = q.size(2);
        a.q = view(q);
        a.table = page_table(o[3], device, a.batch, &a.table_stride, &a.table_entries);
        a.lens = dense<int32_t>(o[4], at::kInt, device, {a.batch});
        a.causal = truth(o[5]);
        a.scale = given(o[6]) ? number(o[6]) : 1.0 / std::sqrt((double)a.cache.head_dim);
        at::Tensor out = fresh(q), lse, ws;
        a.out = view(out);
        const bool with_lse = truth(o[7]);
        if (with_lse) {
            lse = floats(q, {a.batch, a.q_heads, a.q_len});
            a.lse = static_cast<float*>(lse.data_ptr());
        }
        if (const size_t need = e.cache_attn_ws(&a)) {
            ws = bytes(q, need);
            a.workspace = ws.data_ptr();
            a.workspace_bytes = need;
        }
        if (e.cache_attn(&a, PyLong_AsVoidPtr(o[8])) != 1) no();
        return with_lse ? wrap({out, lse}) : THPVariable_Wrap(out);
    });
}

// Addresses of the entries -> capsule (held until the process ends).
PyObject* bind(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (n != kEntries) {
        PyErr_SetString(PyExc_TypeError, "nine addresses");
        return nullptr;
    }
    Entries* e = new (std::nothrow) Entries;
    if (!e) return PyErr_NoMemory();
    void** p = reinterpret_cast<void**>(e);
    for (int i = 0; i < kEntries; ++i) p[i] = PyLong_AsVoidPtr(o[i]);
    return PyCapsule_New(e, kCapsule, nullptr);
}

#define FAST(f) {#f, (PyCFunction)(void*)f, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST(bind),           FAST(layer_norm),    FAST(layer_norm_bwd),
                          FAST(quantize_rows),  FAST(linear_i8),     FAST(kv_cache_write),
                          FAST(kv_cache_read),  FAST(cache_attention),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_decoder_marshal", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decoder_marshal() { return PyModule_Create(&kModule); }
