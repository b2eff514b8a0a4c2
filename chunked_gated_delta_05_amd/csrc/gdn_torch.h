// What the native entries of binding.py share: their arguments, checks, errors,
// devices and streams. Every translation unit of _native.so has its own copy.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <string>
#include <vector>

#include "gdn.h"

namespace gdn_torch {
namespace {

using at::ScalarType;
using at::Tensor;

[[noreturn]] void invalid(const std::string& msg) { throw std::invalid_argument(msg); }

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

std::string dtype_text(ScalarType t) {
    switch (t) {
        case ScalarType::Float: return "torch.float32";
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Half: return "torch.float16";
        case ScalarType::Double: return "torch.float64";
        case ScalarType::Int: return "torch.int32";
        case ScalarType::Byte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

int32_t dtype_code(ScalarType t) {
    if (t == ScalarType::BFloat16) return GDN_DTYPE_BF16;
    if (t == ScalarType::Float) return GDN_DTYPE_F32;
    invalid("unsupported dtype " + dtype_text(t));
}

// ---- arguments
struct Raised {};   // Python's own error is set

struct Arguments {
    PyObject* const* a;
    Py_ssize_t n;
    const char* name;

    void count(Py_ssize_t want) const {
        if (n != want) invalid(std::string(name) + ": expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
    }
    bool none(int i) const { return a[i] == Py_None; }
    Tensor tensor(int i, const char* what) const {   // undefined for None
        if (none(i)) return Tensor();
        if (!THPVariable_Check(a[i])) invalid(std::string(what) + " must be a tensor");
        return THPVariable_Unpack(a[i]);
    }
    bool flag(int i) const {
        const int x = PyObject_IsTrue(a[i]);
        if (x < 0) throw Raised();
        return x == 1;
    }
    int64_t integer(int i) const {
        const long long x = PyLong_AsLongLong(a[i]);
        if (x == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            invalid(std::string(name) + ": an integer is expected");
        }
        return x;
    }
    float scale(int i, int64_t K) const {   // None: 1 / sqrt(K)
        if (none(i)) return (float)(1.0 / std::sqrt((double)K));
        const double x = PyFloat_AsDouble(a[i]);
        if (x == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            invalid("scale must be a number");
        }
        return (float)x;
    }
    // an output's dtype: given, else the given buffer's, else the inputs'
    ScalarType o_dtype(int i, const Tensor& out, ScalarType in) const {
        dtype_code(in);
        ScalarType t = in;
        if (!none(i)) {
            if (!THPDtype_Check(a[i])) invalid("o_dtype must be a torch dtype");
            t = reinterpret_cast<THPDtype*>(a[i])->scalar_type;
        } else if (out.defined()) {
            t = out.scalar_type();
        }
        if (t != ScalarType::Float && t != ScalarType::BFloat16) invalid("unsupported output dtype " + dtype_text(t));
        return t;
    }
};

void check_tensor(const char* name, const Tensor& t, ScalarType dtype, at::IntArrayRef shape) {
    if (t.scalar_type() != dtype) invalid(std::string(name) + " must be " + dtype_text(dtype) + ", got " + dtype_text(t.scalar_type()));
    if (t.sizes() != shape) invalid(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    if (!t.is_contiguous()) invalid(std::string(name) + " must be contiguous");
}

// An output given by the caller may not be one of the inputs: workgroups read
// them while others write it. Of strided inputs everything from the first
// value to the last counts (their strides are not negative).
void check_apart(const Tensor& out, std::initializer_list<std::pair<const char*, const Tensor*>> others) {
    if (!out.defined() || out.numel() == 0) return;
    const uintptr_t a = reinterpret_cast<uintptr_t>(out.data_ptr()), a_end = a + out.nbytes();
    for (const auto& [name, t] : others) {
        if (!t->defined() || t->numel() == 0) continue;
        int64_t last = 0;
        for (int64_t i = 0; i < t->dim(); ++i) last += (t->size(i) - 1) * t->stride(i);
        const uintptr_t b = reinterpret_cast<uintptr_t>(t->data_ptr());
        if (a < b + (last + 1) * t->element_size() && b < a_end) invalid(std::string("out overlaps ") + name);
    }
}

void check_device(const char* name, const Tensor& t, c10::Device dev) {
    if (t.defined() && t.device() != dev) invalid(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
}

void need_gpu(const char* name, const Tensor& t) {
    if (!t.is_cuda()) invalid(std::string(name) + " must be GPU tensors, got " + t.device().str());
}

void check(gdn_status st, const char* what) {
    if (st == GDN_OK) return;
    const std::string msg = std::string(what) + ": libgdn status " + std::to_string((int)st);
    if (st == GDN_ERR_INVALID || st == GDN_ERR_CAPACITY) invalid(msg);
    if (st == GDN_ERR_UNSUPPORTED) throw std::logic_error(msg);
    throw std::runtime_error(msg);
}

template <typename P = void>
P* ptr(const Tensor& t) {
    return t.defined() ? static_cast<P*>(t.data_ptr()) : nullptr;
}

// What a call has written in place of what the caller's tensors held: autograd
// then refuses a gradient that needs the old values. Tensors made in inference
// mode have no version.
void written(std::initializer_list<const Tensor*> tensors) {
    for (const Tensor* t : tensors)
        if (t->defined() && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// A call launches on its tensors' device, whichever is current. (Where it is
// that one already, a c10::DeviceGuard would set it again at the end.)
struct Guard {
    c10::OptionalDeviceGuard other;
    explicit Guard(c10::Device dev) {
        if (c10::hip::current_device() != dev.index()) other.reset_device(dev);
    }
};

hipStream_t stream_of(c10::Device dev) { return c10::hip::getCurrentHIPStream(dev.index()).stream(); }

// (token, head) strides in elements of [B,T,h,D] or [tokens,h,D] rows that
// are contiguous and 16-byte aligned, batch rows at T token strides
void row_strides(const char* name, const Tensor& t, int64_t* out) {
    const auto n = t.sizes(), s = t.strides();
    const int64_t d = t.dim(), W = n[d - 1];
    if (W > 1 && s[d - 1] != 1) invalid(std::string(name) + ": the values of a row must be contiguous");
    int64_t ts = s[d - 3], hs = s[d - 2];
    if (n[d - 2] == 1) hs = W;   // strides of axes of length one are not used
    if (d == 4) {
        const int64_t B = n[0], T = n[1];
        if (B * T <= 1) ts = n[2] * hs;
        else if (T == 1) ts = s[0];
        else if (B > 1 && s[0] != T * ts) invalid(std::string(name) + ": batch rows must follow each other at the token stride");
    } else if (n[0] <= 1) {
        ts = n[1] * hs;
    }
    const int64_t es = t.element_size();
    if ((ts * es) % 16 || (hs * es) % 16 || reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 || ts < 0 || hs < 0)
        invalid(std::string(name) + ": rows must be 16-byte aligned");
    out[0] = ts;
    out[1] = hs;
}

int32_t narrow(int64_t x, const char* what) {
    if (x > INT32_MAX) invalid(std::string(what) + " is too large");
    return (int32_t)x;
}

Tensor workspace_of(const Tensor& given, size_t need, c10::Device dev) {
    if (!given.defined()) return at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(dev));
    if (given.scalar_type() != ScalarType::Byte || given.device() != dev || !given.is_contiguous() ||
        given.numel() < (int64_t)need)
        invalid("workspace must be a uint8 tensor of at least " + std::to_string(need) + " bytes on " + dev.str());
    return given;
}

// ---- entries
void out_of_memory(const char* what) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, what);   // else the import's own error is set
    Py_XDECREF(type);
    Py_XDECREF(torch);
}

template <PyObject* (*F)(const Arguments&)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        return F(Arguments{args, n, "native entry"});
    } catch (const Raised&) {
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::logic_error& e) {
        PyErr_SetString(PyExc_NotImplementedError, e.what());
    } catch (const c10::OutOfMemoryError& e) {   // torch.OutOfMemoryError, as from any allocation
        out_of_memory(e.what_without_backtrace());
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <PyObject* (*F)(const Arguments&)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F>)), METH_FASTCALL, nullptr};
}

}  // namespace
}  // namespace gdn_torch
