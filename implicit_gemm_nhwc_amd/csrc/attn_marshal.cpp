// The ordinary calls of attention.py without Python's share of the time: a
// call's tensors are checked, its outputs and workspace allocated, and the C
// entry called, from C++ (a call of cross_attention: 8.9 -> 5.3 us of host
// time, of which the launch itself takes 3.0).
//
// Each function returns its results, or None for anything it does not take as
// it stands (another type or layout than the ABI describes, another GPU than
// the current one, a call that the library declines): attention.py then goes
// through its own checks, which say what is wrong.  Nothing is decided here
// that is not decided there.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "igemm_attn.h"

namespace {

// Entries of one loaded library (attention.py's _entries).
struct Entries {
    int32_t (*attn_fwd)(const igc_cross_attn*, void*);
    size_t (*attn_fwd_ws)(const igc_cross_attn*);
    int32_t (*attn_bwd)(const igc_cross_attn_grad*, void*);
    size_t (*attn_bwd_ws)(const igc_cross_attn_grad*);
    int32_t (*norm_fwd)(const igc_qk_norm*, void*);
    int32_t (*norm_bwd)(const igc_qk_norm*, void*);
    size_t (*norm_bwd_ws)(const igc_qk_norm*);
};

constexpr const char* kCapsule = "igc_attn_entries";

struct NotTaken {};   // thrown within this file only: the call returns None
[[noreturn]] void no() { throw NotTaken(); }

const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) no();
    return THPVariable_Unpack(o);
}

// A tensor of this type on the current GPU.
const at::Tensor& on_gpu(PyObject* o, at::ScalarType type, int64_t device, int64_t dim) {
    const at::Tensor& t = tensor(o);
    if (!t.is_cuda() || t.get_device() != device || t.scalar_type() != type || t.dim() != dim ||
        t.layout() != at::kStrided)
        no();
    return t;
}

igc_attn_view view(const at::Tensor& t) {
    if (t.stride(3) != 1 && t.size(3) > 1) no();
    return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

int64_t type_code(at::ScalarType t) {
    if (t == at::kBFloat16) return IGC_DTYPE_BF16;
    if (t == at::kHalf) return IGC_DTYPE_FP16;
    no();
}

bool given(PyObject* o) { return o != Py_None; }

// Truth value of an argument (one that has none is Python's to report).
bool truth(PyObject* o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) no();
    return t != 0;
}

template <typename T>
T* dense(PyObject* o, at::ScalarType type, int64_t device, at::IntArrayRef sizes) {
    const at::Tensor& t = on_gpu(o, type, device, (int64_t)sizes.size());
    if (t.sizes() != sizes || !t.is_contiguous()) no();
    return static_cast<T*>(t.data_ptr());
}

at::Tensor fresh(const at::Tensor& t) {
    return at::empty(t.sizes(), t.options().memory_format(at::MemoryFormat::Contiguous));
}
at::Tensor floats(const at::Tensor& t, at::IntArrayRef sizes) {
    return at::empty(sizes, t.options().dtype(at::kFloat));
}
at::Tensor bytes(const at::Tensor& t, size_t n) {
    return at::empty({(int64_t)n}, t.options().dtype(at::kByte));
}

// The arguments common to cross attention's passes; o = {q, k, v, scale,
// kv_lens, key_mask}.
igc_cross_attn attn_args(PyObject* q_, PyObject* k_, PyObject* v_, PyObject* scale,
                         PyObject* lens, PyObject* mask, int64_t device) {
    const at::Tensor& q = tensor(q_);
    const at::ScalarType type = q.scalar_type();
    igc_cross_attn a{};
    a.dtype = type_code(type);
    on_gpu(q_, type, device, 4);
    const at::Tensor& k = on_gpu(k_, type, device, 4);
    const at::Tensor& v = on_gpu(v_, type, device, 4);
    a.batch = q.size(0);
    a.q_len = q.size(1);
    a.q_heads = q.size(2);
    a.head_dim = q.size(3);
    a.kv_len = k.size(1);
    a.kv_heads = k.size(2);
    if (k.size(0) != a.batch || k.size(3) != a.head_dim || v.sizes() != k.sizes()) no();
    a.q = view(q);
    a.k = view(k);
    a.v = view(v);
    if (given(lens)) a.kv_lens = dense<int32_t>(lens, at::kInt, device, {a.batch});
    if (given(mask)) {
        const at::Tensor& m = tensor(mask);
        const at::ScalarType mt = m.scalar_type();
        if (mt != at::kByte && mt != at::kBool) no();
        on_gpu(mask, mt, device, 2);
        if (m.size(0) != a.batch || m.size(1) != a.kv_len || (m.stride(1) != 1 && a.kv_len > 1))
            no();
        a.key_mask = static_cast<const uint8_t*>(m.data_ptr());
        a.key_mask_stride = m.stride(0);
    }
    if (given(scale)) {
        a.scale = PyFloat_AsDouble(scale);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            no();
        }
    } else {
        a.scale = a.head_dim ? 1.0 / std::sqrt((double)a.head_dim) : 1.0;
    }
    return a;
}

const Entries& entries(PyObject* o) {
    void* p = PyCapsule_GetPointer(o, kCapsule);
    if (!p) {
        PyErr_Clear();
        no();
    }
    return *static_cast<Entries*>(p);
}

// Runs f, whose exceptions (ATen's too: the Python path meets the same
// condition and reports it) become None.
template <typename F>
PyObject* taken(F f) {
    try {
        return f();
    } catch (...) {
        if (PyErr_Occurred()) PyErr_Clear();
        Py_RETURN_NONE;
    }
}

PyObject* wrap(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o = Py_None;
        if (t.defined()) o = THPVariable_Wrap(t);
        else Py_INCREF(o);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// (entries, q, k, v, scale, kv_lens, key_mask, return_lse, stream, device)
PyObject* cross_attention(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 10) no();
        const Entries& e = entries(o[0]);
        const int64_t device = PyLong_AsLongLong(o[9]);
        igc_cross_attn a = attn_args(o[1], o[2], o[3], o[4], o[5], o[6], device);
        const at::Tensor& q = tensor(o[1]);
        at::Tensor out = fresh(q), lse, ws;
        a.out = view(out);
        const bool with_lse = truth(o[7]);
        if (with_lse) {
            lse = floats(q, {a.batch, a.q_heads, a.q_len});
            a.lse = static_cast<float*>(lse.data_ptr());
        }
        if (const size_t need = e.attn_fwd_ws(&a)) {
            ws = bytes(q, need);
            a.workspace = ws.data_ptr();
            a.workspace_bytes = need;
        }
        if (e.attn_fwd(&a, PyLong_AsVoidPtr(o[8])) != 1) no();
        return with_lse ? wrap({out, lse}) : THPVariable_Wrap(out);
    });
}

// (entries, dout, q, k, v, out, lse, scale, kv_lens, key_mask, stream, device)
PyObject* cross_attention_bwd(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 12) no();
        const Entries& e = entries(o[0]);
        const int64_t device = PyLong_AsLongLong(o[11]);
        igc_cross_attn_grad a{};
        a.fwd = attn_args(o[2], o[3], o[4], o[7], o[8], o[9], device);
        igc_cross_attn& f = a.fwd;
        const at::Tensor &q = tensor(o[2]), &k = tensor(o[3]), &v = tensor(o[4]);
        const at::Tensor& g = on_gpu(o[1], q.scalar_type(), device, 4);
        const at::Tensor& out = on_gpu(o[5], q.scalar_type(), device, 4);
        if (g.sizes() != q.sizes() || out.sizes() != q.sizes()) no();
        a.dout = view(g);
        f.out = view(out);
        f.lse = dense<float>(o[6], at::kFloat, device, {f.batch, f.q_heads, f.q_len});
        at::Tensor dq = fresh(q), dk = fresh(k), dv = fresh(v), ws;
        a.dq = view(dq);
        a.dk = view(dk);
        a.dv = view(dv);
        if (const size_t need = e.attn_bwd_ws(&a)) {
            ws = bytes(q, need);
            f.workspace = ws.data_ptr();
            f.workspace_bytes = need;
        }
        if (e.attn_bwd(&a, PyLong_AsVoidPtr(o[10])) != 1) no();
        return wrap({dq, dk, dv});
    });
}

// Sizes, input and side arrays of one part; o = x, weight, table, positions.
void qk_part(igc_qk_part* p, PyObject* x_, PyObject* weight, PyObject* table, PyObject* pos,
             at::ScalarType type, int64_t device, int64_t* d, int64_t* rot) {
    const at::Tensor& x = on_gpu(x_, type, device, 4);
    if (*d >= 0 && x.size(3) != *d) no();
    *d = x.size(3);
    p->batch = x.size(0);
    p->tokens = x.size(1);
    p->heads = x.size(2);
    p->x = view(x);
    if (given(weight)) p->weight = dense<float>(weight, at::kFloat, device, {*d});
    int64_t r = 0;
    if (given(table)) {
        const at::Tensor& t = on_gpu(table, at::kFloat, device, 2);
        if (!t.is_contiguous()) no();
        p->table = static_cast<const float*>(t.data_ptr());
        p->table_rows = t.size(0);
        r = t.size(1);
    }
    if (*rot >= 0 && *rot != r) no();
    *rot = r;
    if (given(pos)) {
        const at::Tensor& t = on_gpu(pos, at::kInt, device, 2);
        if (t.size(0) != p->batch || t.size(1) != p->tokens || (t.stride(1) != 1 && p->tokens > 1))
            no();
        p->positions = static_cast<const int32_t*>(t.data_ptr());
        p->positions_stride = t.stride(0);
    }
}

// o = q, k, q_weight, k_weight, q_table, k_table, q_positions, k_positions,
// eps, interleaved
igc_qk_norm norm_args(PyObject* const* o, int64_t device) {
    igc_qk_norm a{};
    const at::ScalarType type = tensor(o[0]).scalar_type();
    a.dtype = type_code(type);
    int64_t d = -1, rot = -1;
    qk_part(&a.q, o[0], o[2], o[4], o[6], type, device, &d, &rot);
    if (given(o[1])) qk_part(&a.k, o[1], o[3], o[5], o[7], type, device, &d, &rot);
    a.head_dim = d;
    a.rot_dim = rot;
    a.eps = PyFloat_AsDouble(o[8]);
    if (PyErr_Occurred()) no();
    a.interleaved = truth(o[9]);
    return a;
}

// (entries, q, k, ... interleaved, stream, device)
PyObject* qk_norm_rope(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 13) no();
        const Entries& e = entries(o[0]);
        igc_qk_norm a = norm_args(o + 1, PyLong_AsLongLong(o[12]));
        at::Tensor q = fresh(tensor(o[1])), k;
        a.q.out = view(q);
        if (given(o[2])) {
            k = fresh(tensor(o[2]));
            a.k.out = view(k);
        }
        if (e.norm_fwd(&a, PyLong_AsVoidPtr(o[11])) != 1) no();
        return k.defined() ? wrap({q, k}) : THPVariable_Wrap(q);
    });
}

// (entries, dq, dk, q, k, ... interleaved, stream, device)
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return taken([&]() -> PyObject* {
        if (n != 15) no();
        const Entries& e = entries(o[0]);
        const int64_t device = PyLong_AsLongLong(o[14]);
        igc_qk_norm a = norm_args(o + 3, device);
        const at::Tensor& xq = tensor(o[3]);
        at::Tensor out[2], dw[2], ws;
        igc_qk_part* parts[2] = {&a.q, &a.k};
        for (int i = 0; i < 2; ++i) {
            if (!given(o[3 + i])) continue;
            const at::Tensor& x = tensor(o[3 + i]);
            const at::Tensor& g = on_gpu(o[1 + i], x.scalar_type(), device, 4);
            if (g.sizes() != x.sizes()) no();
            parts[i]->grad = view(g);
            out[i] = fresh(x);
            parts[i]->out = view(out[i]);
            dw[i] = floats(x, {a.head_dim});
            parts[i]->dweight = static_cast<float*>(dw[i].data_ptr());
        }
        if (const size_t need = e.norm_bwd_ws(&a)) {
            ws = bytes(xq, need);
            a.workspace = ws.data_ptr();
            a.workspace_bytes = need;
        }
        if (e.norm_bwd(&a, PyLong_AsVoidPtr(o[13])) != 1) no();
        return wrap({out[0], out[1], dw[0], dw[1]});
    });
}

// Addresses of the seven entries -> capsule (held until the process ends).
PyObject* bind(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "seven addresses");
        return nullptr;
    }
    Entries* e = new (std::nothrow) Entries;
    if (!e) return PyErr_NoMemory();
    void** p = reinterpret_cast<void**>(e);
    for (int i = 0; i < 7; ++i) p[i] = PyLong_AsVoidPtr(o[i]);
    return PyCapsule_New(e, kCapsule, nullptr);
}

#define FAST(f) {#f, (PyCFunction)(void*)f, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST(bind),         FAST(cross_attention),  FAST(cross_attention_bwd),
                          FAST(qk_norm_rope), FAST(qk_norm_rope_bwd),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_attn_marshal", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_marshal() { return PyModule_Create(&kModule); }
