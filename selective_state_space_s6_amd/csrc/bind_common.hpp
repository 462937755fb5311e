// bind_common.hpp -- what the sources of the compiled Python binding share: checks of tensors and
// numbers, outputs and workspaces, Python's errors.  Everything is local to the source that
// includes it; some of it is used by one of them alone.
#pragma once
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <initializer_list>
#include <string>
#include <tuple>

#include "../../include/ssm_longctx.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

// Thrown with the Python error set; caught where a function returns to the interpreter.
struct Refused {};

[[noreturn]] void refuse(PyObject *kind, const std::string &text) {
    PyErr_SetString(kind, text.c_str());
    throw Refused{};
}

std::string show(IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const char *show(ScalarType t) {
    switch (t) {
        case ScalarType::Float: return "torch.float32";
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Int: return "torch.int32";
        case ScalarType::Long: return "torch.int64";
        case ScalarType::Byte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + ": a tensor is required");
    return THPVariable_Unpack(o);
}

// what a call's tensors have in common, from its first one
struct Call {
    c10::Device dev;
    c10::TensorOptions options;
    explicit Call(const Tensor &t) : dev(t.device()), options(t.options().requires_grad(false)) {}
    bool gpu() const { return dev.is_cuda(); }

    void check(const Tensor &t, const char *name, ScalarType dtype, IntArrayRef shape) const {
        if (t.scalar_type() != dtype)
            refuse(PyExc_TypeError, std::string(name) + ": dtype " + show(t.scalar_type()) + ", expected " + show(dtype));
        if (t.sizes() != shape)
            refuse(PyExc_ValueError, std::string(name) + ": shape " + show(t.sizes()) + ", expected " + show(shape));
        if (t.device() != dev)
            refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
    }
    // a contiguous tensor's address
    void *whole(PyObject *o, const char *name, ScalarType dtype, std::initializer_list<int64_t> shape) const {
        const Tensor &t = tensor(o, name);
        check(t, name, dtype, IntArrayRef(shape.begin(), shape.size()));
        if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
        return t.data_ptr();
    }
    // the address of a tensor whose last dim has stride 1
    void *view(const Tensor &t, const char *name, ScalarType dtype, IntArrayRef shape) const {
        check(t, name, dtype, shape);
        if (t.stride(-1) != 1 && shape.back() != 1 && t.numel() > 0)
            refuse(PyExc_ValueError, std::string(name) + ": the last dim must have stride 1");
        return t.data_ptr();
    }
    // an output: the caller's, or a new one
    Tensor out(PyObject *o, const char *name, ScalarType dtype, std::initializer_list<int64_t> shape) const {
        if (o == Py_None) return make(dtype, shape);
        whole(o, name, dtype, shape);
        return THPVariable_Unpack(o);
    }
    Tensor make(ScalarType dtype, std::initializer_list<int64_t> shape) const {
        if (!gpu()) refuse(PyExc_ValueError, "tensors are on " + dev.str() + ", expected a GPU");
        return at::empty(IntArrayRef(shape.begin(), shape.size()), options.dtype(dtype));
    }
    // new outputs in one allocation, each from a multiple of 16 bytes on: an allocation costs
    // more than the rest of a small call's checks
    struct Wanted { ScalarType dtype; std::initializer_list<int64_t> shape; };
    template <size_t N> std::array<Tensor, N> make_together(const Wanted (&want)[N]) const {
        int64_t at[N], bytes = 0;
        for (size_t i = 0; i < N; ++i) {
            at[i] = bytes;
            int64_t n = (int64_t)c10::elementSize(want[i].dtype);
            for (int64_t d : want[i].shape) n *= d;
            bytes += (n + 15) / 16 * 16;
        }
        const Tensor all = make(ScalarType::Byte, {bytes});
        std::array<Tensor, N> r;
        for (size_t i = 0; i < N; ++i) {
            r[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                            c10::scalarTypeToTypeMeta(want[i].dtype));
            r[i].unsafeGetTensorImpl()->set_storage_offset(at[i] / (int64_t)c10::elementSize(want[i].dtype));
            r[i].unsafeGetTensorImpl()->set_sizes_contiguous(IntArrayRef(want[i].shape.begin(), want[i].shape.size()));
        }
        return r;
    }
    // few enough (up to 4 MiB) that outputs which stay alive do not hold much of each other's memory
    static bool few(int64_t elements) { return elements <= (1 << 20); }
    Tensor workspace(PyObject *o, size_t need) const {
        if (o == Py_None) return make(ScalarType::Byte, {(int64_t)need});
        const Tensor &t = tensor(o, "workspace");
        if (t.device() != dev || !t.is_contiguous())
            refuse(PyExc_ValueError, "workspace must be a contiguous tensor on the inputs' device");
        return t;
    }
    hipStream_t stream() const {
        if (!gpu()) refuse(PyExc_ValueError, "tensors are on " + dev.str() + ", expected a GPU");
        return c10::hip::getCurrentHIPStream(dev.index()).stream();
    }
};

ssm_dtype_t head_dtype(const Tensor &t, const char *name) {
    if (t.scalar_type() == ScalarType::Float) return SSM_F32;
    if (t.scalar_type() == ScalarType::BFloat16) return SSM_BF16;
    refuse(PyExc_TypeError, std::string(name) + ": dtype " + show(t.scalar_type()) + ", expected float32 or bfloat16");
}

void dims(const Tensor &t, const char *name, int64_t n, const char *form) {
    if (t.dim() != n) refuse(PyExc_ValueError, std::string(name) + ": shape " + show(t.sizes()) + ", expected " + form);
}

int64_t whole_number(PyObject *o, const char *name) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_TypeError, std::string(name) + ": a whole number is required");
    }
    return v;
}
uint32_t flag_bits(PyObject *o) {
    const int64_t v = whole_number(o, "flags");
    if (v < 0 || v > 0xffffffffLL) refuse(PyExc_ValueError, "flags: " + std::to_string(v) + " has bits that no flag has");
    return (uint32_t)v;
}
float number(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_TypeError, std::string(name) + ": a number is required");
    }
    return (float)v;
}

void set(PyObject *dict, const char *name, const Tensor &t) {
    PyObject *v = THPVariable_Wrap(t);
    PyDict_SetItemString(dict, name, v);
    Py_DECREF(v);
}

// Runs a function's body: its refusals and torch's errors (out of memory) become Python's.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F body) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused &) {
        return nullptr;
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject *pair(const Tensor &x, const Tensor &y) {
    PyObject *t = PyTuple_New(2);
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(x));
    if (y.defined()) {
        PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(y));
    } else {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(t, 1, Py_None);
    }
    return t;
}

// a pair of caches (pages, page_size, kv_heads, headdim) with the same strides
struct Caches {
    void *k, *v;
    int64_t pages, page_size, Hk, d, sp, st, sh;
    ssm_kv_dtype_t kv;
    Caches(const Call &c, PyObject *ok, PyObject *ov) {
        const Tensor &tk = tensor(ok, "k_cache"), &tv = tensor(ov, "v_cache");
        switch (tk.scalar_type()) {
            case ScalarType::Float: kv = SSM_KV_F32; break;
            case ScalarType::BFloat16: kv = SSM_KV_BF16; break;
            case ScalarType::Float8_e4m3fn: kv = SSM_KV_F8E4M3; break;
            default:
                refuse(PyExc_TypeError, std::string("k_cache: dtype ") + show(tk.scalar_type()) +
                                            ", expected float32, bfloat16 or float8_e4m3fn");
        }
        dims(tk, "k_cache", 4, "(pages, page_size, kv_heads, headdim)");
        k = c.view(tk, "k_cache", tk.scalar_type(), tk.sizes());
        v = c.view(tv, "v_cache", tk.scalar_type(), tk.sizes());
        if (tk.strides() != tv.strides())
            refuse(PyExc_ValueError, "v_cache: strides " + show(tv.strides()) + ", expected k_cache's " + show(tk.strides()));
        pages = tk.size(0); page_size = tk.size(1); Hk = tk.size(2); d = tk.size(3);
        sp = tk.stride(0); st = tk.stride(1); sh = tk.stride(2);
    }
};

}  // namespace
