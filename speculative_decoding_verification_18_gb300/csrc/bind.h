// Checks of arguments that the bindings share (kvbind.cpp, lpbind.cpp).

#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>
#include <string>

#include "specverify.h"

namespace {

struct Refused {
    PyObject* type;
    std::string why;
};
[[noreturn]] void value(const std::string& why) { throw Refused{PyExc_ValueError, why}; }
[[noreturn]] void type(const std::string& why) { throw Refused{PyExc_TypeError, why}; }

std::string shape_of(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// The call's tensors are all on the current device: looked at last, once the rest is right.
struct Devices {
    int first = 0;
    bool any = false;
    void add(const at::Tensor& t, const char* name) {
        if (!t.is_cuda()) value(std::string(name) + " must be a CUDA tensor");
        const int d = t.get_device();
        if (any && d != first) value(std::string(name) + " is on another device than the others");
        first = d;
        any = true;
    }
    void check(int cache = -1) const {
        const int now = c10::cuda::current_device();
        if ((cache >= 0 && cache != now) || (any && first != now))
            value("tensors must be on the current device (cuda:" + std::to_string(now) + ")");
    }
};

// A contiguous tensor of this shape and type, or None.
void* vector(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType t,
             at::ScalarType also) {
    if (o == Py_None) return nullptr;
    const at::Tensor& x = tensor(o, name);
    if (x.scalar_type() != t && x.scalar_type() != also)
        type(std::string(name) + " must be " + c10::toString(t) + ", not " +
             c10::toString(x.scalar_type()));
    if (x.sizes() != shape)
        value(std::string(name) + " has shape " + shape_of(x.sizes()) + ", not " +
              shape_of(shape));
    if (!x.is_contiguous()) value(std::string(name) + " must be contiguous");
    return x.data_ptr();
}
void* ints(PyObject* o, const char* name, at::IntArrayRef shape) {
    return vector(o, name, shape, at::kInt, at::kInt);
}
cudaStream_t stream_of(PyObject* o) {
    return o == Py_None ? c10::cuda::getCurrentCUDAStream().stream()
                        : static_cast<cudaStream_t>(PyLong_AsVoidPtr(o));
}
int number(PyObject* o, const char* name) {
    const long long x = PyLong_AsLongLong(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        type(std::string(name) + " must be a whole number");
    }
    if (x < INT_MIN || x > INT_MAX) value(std::string(name) + " is too large");
    return (int)x;
}

template <typename F> PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        const sv_status st = f();
        return PyErr_Occurred() ? nullptr : PyLong_FromLong(st);
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.why.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

void add(Devices& d, PyObject* o, const char* name) {
    if (o != Py_None) d.add(THPVariable_Unpack(o), name);
}

}  // namespace
