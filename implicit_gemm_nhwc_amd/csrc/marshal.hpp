// Pieces of the bindings' C++ parts (attn_marshal.cpp, decoder_marshal.cpp):
// checks of tensors, new tensors, results.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <new>

#include "igemm_attn.h"

namespace {

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

}  // namespace
