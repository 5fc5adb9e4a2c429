// bind.h -- what the compiled Python entries share: checks of tensors, the
// current stream, and status codes as exceptions.  Included by one source per
// module; everything here is internal to it.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "w4a8.h"

namespace {

struct Refused {};   // a Python exception is set

template <typename... A>
[[noreturn]] void refuse(PyObject* kind, const char* format, A... a) {
    PyErr_Format(kind, format, a...);
    throw Refused();
}

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kByte: return "uint8";
        case at::kInt: return "int32";
        case at::kLong: return "int64";
        case at::kFloat: return "float32";
        case at::kHalf: return "float16";
        case at::kBFloat16: return "bfloat16";
        default: return "16-bit float";
    }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch tensor", name);
    return THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type, at::Device dev) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be a %s tensor", name, type_name(type));
    if (t.device() != dev)
        refuse(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), dev.str().c_str());
    return t;
}
const at::Tensor& vector(PyObject* o, const char* name, at::ScalarType type, at::Device dev, int64_t n) {
    const at::Tensor& t = tensor(o, name, type, dev);
    if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous vector of %lld", name, (long long)n);
    return t;
}

// bf16 or fp16
w4a8_float float_kind(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return W4A8_BF16;
    if (t.scalar_type() == at::kHalf) return W4A8_FP16;
    refuse(PyExc_TypeError, "%s must be a bfloat16 or float16 tensor", name);
}

void on_gpu(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be on a GPU", name);
}

// the caller's output, or a new contiguous tensor
at::Tensor output(PyObject* o, const char* name, const at::Tensor& like, at::IntArrayRef shape, bool gpu) {
    if (o == Py_None) {
        if (!gpu) refuse(PyExc_ValueError, "%s needs a GPU", name);
        return at::empty(shape, like.options());
    }
    const at::Tensor& t = tensor(o, name, like.scalar_type(), like.device());
    if (t.sizes() != shape || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous tensor of the input's shape", name);
    return t;
}

const float* weight(PyObject* o, const char* name, at::Device dev, int64_t d) {
    return o == Py_None ? nullptr : vector(o, name, at::kFloat, dev, d).const_data_ptr<float>();
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}
int64_t integer(PyObject* o, const char* name, int64_t lo, int64_t hi) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    if (v < lo || v > hi) refuse(PyExc_ValueError, "%s must be from %lld to %lld", name, (long long)lo, (long long)hi);
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v != 0;
}
void arguments(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) refuse(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
}

void* stream(at::Device dev) { return (void*)c10::hip::getCurrentHIPStream(dev.index()).stream(); }

PyObject* hip_error;   // W4A8Error of binding.py, set by the Python module

void check(w4a8_status s, const char* what) {
    if (s == W4A8_OK) return;
    if (s == W4A8_ERR_HIP && hip_error) {
        PyObject* e = PyObject_CallFunction(hip_error, "is", (int)s, what);
        if (e) {
            PyErr_SetObject(hip_error, e);
            Py_DECREF(e);
        }
        throw Refused();
    }
    refuse(s == W4A8_ERR_HIP ? PyExc_RuntimeError : PyExc_ValueError, "%s: %s (status %d)", what, w4a8_status_string(s),
           (int)s);
}

PyObject* set_error(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 1);
    Py_XDECREF(hip_error);
    hip_error = Py_NewRef(a[0]);
    return Py_NewRef(Py_None);
}

// no exception leaves an entry: torch's become Python's
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(a, n);
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)(void))entry<F>, METH_FASTCALL, nullptr};
}

}  // namespace
