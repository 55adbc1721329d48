// What the tensor-level calls of the Python binding share: Python arguments, errors,
// outputs and workspaces. Host code only, included by binding.cpp.
#pragma once

#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <limits>
#include <optional>
#include <string>

#include "rmsnorm.h"

namespace {

PyObject* g_error = nullptr;  // RMSNormError(status, what)

// Raised as the Python exception it stands for.
struct Refused {
    int status;  // 0: a ValueError
    std::string what;
};
[[noreturn]] void refuse(std::string what) { throw Refused{RMSNORM_ERR_INVALID_ARG, std::move(what)}; }
[[noreturn]] void bad_value(std::string what) { throw Refused{0, std::move(what)}; }

PyObject* raise(const Refused& r) {
    if (r.status == 0) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
        return nullptr;
    }
    PyObject* e = PyObject_CallFunction(g_error, "is", r.status, r.what.c_str());
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

using Optional = std::optional<at::Tensor>;

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) bad_value(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}
Optional optional(PyObject* o, const char* name) {
    if (o == Py_None) return std::nullopt;
    return tensor(o, name);
}
int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

std::string text(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t n : t.sizes()) s += std::to_string(n) + ", ";
    return s + ") " + c10::toString(t.scalar_type());
}

// dtype code of activations of type t beside weights of type u
int pair_code(at::ScalarType t, at::ScalarType u) {
    const bool wide = u == at::kFloat && t != at::kFloat;
    if (u == t || wide) {
        if (t == at::kFloat) return RMSNORM_F32;
        if (t == at::kBFloat16) return wide ? RMSNORM_BF16_W_F32 : RMSNORM_BF16;
        if (t == at::kHalf) return wide ? RMSNORM_F16_W_F32 : RMSNORM_F16;
    }
    refuse(std::string("unsupported dtypes x=") + c10::toString(t) + " w=" + c10::toString(u));
}
int dtype_code(const at::Tensor& x, const Optional& w) {
    return pair_code(x.scalar_type(), w ? w->scalar_type() : x.scalar_type());
}

void same_device(const at::Tensor& x, const at::Tensor& t) {
    if (t.device() != x.device()) refuse("tensors on " + t.device().str() + " and " + x.device().str());
}
void same_device(const at::Tensor& x, const Optional& t) {
    if (t) same_device(x, *t);
}
void on_gpu(const at::Tensor& x) {
    if (!x.is_cuda()) bad_value("tensor argument on " + x.device().str() + ": the library takes CUDA tensors");
}
void dense(const at::Tensor& t) {
    if (!t.is_contiguous())
        bad_value("tensor argument is not contiguous: the library takes dense row-major tensors "
                  "(call .contiguous() first)");
}
void dense(const Optional& t) {
    if (t) dense(*t);
}
const void* data(const Optional& t) { return t ? t->const_data_ptr() : nullptr; }

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
    return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

// The call's device, stream and workspace. A stream that is given is the current
// one meanwhile: the caching allocator then gives memory ordered on it, for the
// outputs as for the workspace.
struct Run {
    c10::cuda::CUDAGuard guard;
    std::optional<c10::cuda::CUDAStreamGuard> on;
    cudaStream_t stream;
    void* ws = nullptr;
    Run(const at::Tensor& x, PyObject* s) : guard(x.device()) {
        const auto device = x.get_device();
        stream = c10::cuda::getCurrentCUDAStream(device).stream();
        if (s == Py_None) return;
        const cudaStream_t there = reinterpret_cast<cudaStream_t>(integer(s));
        if (there == stream) return;
        on.emplace(there == nullptr ? c10::cuda::getDefaultCUDAStream(device)
                                    : c10::cuda::getStreamFromExternal(there, device));
        stream = there;
    }
    ~Run() {
        if (ws != nullptr) c10::cuda::CUDACachingAllocator::raw_delete(ws);
    }
    Run(const Run&) = delete;
    Run& operator=(const Run&) = delete;
    void* workspace(size_t need) {
        if (need > 0) ws = c10::cuda::CUDACachingAllocator::raw_alloc(need);
        return ws;
    }
};

template <typename Call>
void check(const char* what, Call call) {
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = call();
    Py_END_ALLOW_THREADS;
    if (st != RMSNORM_OK) throw Refused{st, what};
}

template <typename F>
PyObject* guarded(F f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refused& r) {
        return raise(r);
    }
    END_HANDLE_TH_ERRORS
}

PyObject* wrap(const Optional& t) {
    if (!t) Py_RETURN_NONE;
    return THPVariable_Wrap(*t);
}
template <typename... T>
PyObject* tuple(const T&... t) {
    PyObject* items[] = {wrap(Optional(t))...};
    constexpr Py_ssize_t n = sizeof...(T);
    PyObject* out = PyTuple_New(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (out != nullptr && items[i] != nullptr) PyTuple_SET_ITEM(out, i, items[i]);
        else Py_XDECREF(items[i]);
    }
    return out;
}

}  // namespace
