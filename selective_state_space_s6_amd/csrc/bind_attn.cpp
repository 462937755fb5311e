// bind_attn.cpp -- the Python binding of include/ssm_attn.h's entry points as a CPython
// module, in place of ctypes: one decode step makes three of these calls a layer, each a few
// microseconds of GPU work, and checking and passing a dozen tensors in Python took the host
// 14 to 22 us a call where this takes 4.2 to 5.1 (each of the five entry points, 4 tokens, outputs
// allocated).
//
// It only marshals: dtype, shape, stride and device of every tensor are checked, missing
// outputs and workspaces allocated with torch, and addresses and the current stream handed to
// the library, which checks everything else.  Functions take positional arguments from
// attn.py, raise TypeError or ValueError for what they check, and return the library's
// negative status as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <initializer_list>
#include <string>
#include <tuple>

#include "../../include/ssm_attn.h"

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
        if (t.stride(-1) != 1 && shape.back() != 1)
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

PyObject *pages_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const Tensor &len_old = tensor(a[0], "len_old"), &table = tensor(a[2], "block_table"), &ring = tensor(a[3], "free_ring");
        const Call c(len_old);
        dims(table, "block_table", 2, "(batch, max_pages)");
        dims(ring, "free_ring", 1, "(n_pages,)");
        const int64_t batch = table.size(0), max_pages = table.size(1), n_pages = ring.size(0);
        const int64_t page_size = whole_number(a[5], "page_size"), tokens = whole_number(a[6], "n_tokens");
        const auto i32 = ScalarType::Int;
        auto *p_old = (const int32_t *)c.whole(a[0], "len_old", i32, {batch});
        auto *p_new = (const int32_t *)c.whole(a[1], "len_new", i32, {batch});
        auto *p_table = (int32_t *)c.view(table, "block_table", i32, table.sizes());
        auto *p_free = (int32_t *)c.whole(a[3], "free_ring", i32, {n_pages});
        auto *p_ring = (const int32_t *)c.whole(a[4], "ring", i32, {2});
        const hipStream_t stream = c.stream();
        const int64_t room = tokens > 0 ? tokens : 0;
        Tensor slots, request, positions, len, starts, ring_out, denied;
        if (c.few(4 * room)) {
            std::tie(slots, request, positions, len, starts, ring_out, denied) = std::tuple_cat(c.make_together<7>(
                {{ScalarType::Long, {room}}, {i32, {room}}, {i32, {room}}, {i32, {batch}}, {i32, {batch + 1}}, {i32, {2}}, {i32, {1}}}));
        } else {    // len and ring go on to the next step, the tokens' maps need not
            std::tie(slots, request, positions) = std::tuple_cat(c.make_together<3>({{ScalarType::Long, {room}}, {i32, {room}}, {i32, {room}}}));
            std::tie(len, starts, ring_out, denied) = std::tuple_cat(c.make_together<4>({{i32, {batch}}, {i32, {batch + 1}}, {i32, {2}}, {i32, {1}}}));
        }
        const int rc = ssm_kv_pages_step(
            p_old, p_new, p_table, p_free, p_ring, (int32_t *)ring_out.data_ptr(), (int32_t *)len.data_ptr(),
            (int32_t *)starts.data_ptr(), (int32_t *)request.data_ptr(), (int32_t *)positions.data_ptr(),
            (int64_t *)slots.data_ptr(), (int32_t *)denied.data_ptr(), batch, max_pages,
            batch > 1 ? table.stride(0) : max_pages, n_pages, page_size, tokens, stream);
        if (rc != SSM_OK) return PyLong_FromLong(rc);
        PyObject *d = PyDict_New();
        set(d, "ring", ring_out); set(d, "len", len); set(d, "starts", starts); set(d, "request", request);
        set(d, "positions", positions); set(d, "slots", slots); set(d, "denied", denied);
        return d;
    });
}

// the arguments that the norm and rotation calls share: q, k, wq, wk, inv_freq, positions
struct Rope {
    Call c;
    ScalarType type;
    ssm_dtype_t dtype;
    int64_t T, H, Hk = 0, d, rot;
    const void *q, *k = nullptr;
    const float *wq = nullptr, *wk = nullptr, *inv_freq;
    const int32_t *positions;
    int64_t q_st, q_sh, k_st = 0, k_sh = 0;
    bool norm;
    Rope(PyObject *const *a, uint32_t flags) : c(tensor(a[0], "q")) {
        const Tensor &tq = tensor(a[0], "q");
        dims(tq, "q", 3, "(tokens, heads, headdim)");
        dtype = head_dtype(tq, "q");
        type = tq.scalar_type();
        T = tq.size(0); H = tq.size(1); d = tq.size(2);
        q = c.view(tq, "q", type, tq.sizes());
        q_st = tq.stride(0); q_sh = tq.stride(1);
        if (a[1] != Py_None) {
            const Tensor &tk = tensor(a[1], "k");
            dims(tk, "k", 3, "(tokens, kv_heads, headdim)");
            Hk = tk.size(1);
            k = c.view(tk, "k", type, {T, Hk, d});
            k_st = tk.stride(0); k_sh = tk.stride(1);
        }
        norm = (flags & SSM_QK_NO_NORM) == 0;
        if (norm) {
            wq = (const float *)c.whole(a[2], "wq", ScalarType::Float, {d});
            if (k) wk = (const float *)c.whole(a[3], "wk", ScalarType::Float, {d});
        }
        const Tensor &f = tensor(a[4], "inv_freq");
        dims(f, "inv_freq", 1, "(rot/2,)");
        rot = 2 * f.size(0);
        inv_freq = (const float *)c.whole(a[4], "inv_freq", ScalarType::Float, {f.size(0)});
        positions = (const int32_t *)c.whole(a[5], "positions", ScalarType::Int, {T});
        if (k != nullptr && Hk == 0) refuse(PyExc_ValueError, "k: no heads");
    }
};

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

PyObject *rope_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const float eps = number(a[6], "eps");
        const uint32_t flags = flag_bits(a[7]);
        const Rope r(a, flags);
        Tensor qo, ko;
        if (a[1] != Py_None && a[8] == Py_None && a[9] == Py_None && r.c.few(r.T * (r.H + r.Hk) * r.d)) {
            std::tie(qo, ko) = std::tuple_cat(r.c.make_together<2>({{r.type, {r.T, r.H, r.d}}, {r.type, {r.T, r.Hk, r.d}}}));
        } else {
            qo = r.c.out(a[8], "q_out", r.type, {r.T, r.H, r.d});
            if (a[1] != Py_None) ko = r.c.out(a[9], "k_out", r.type, {r.T, r.Hk, r.d});
        }
        const int rc = ssm_qk_norm_rope_fwd(r.q, r.k, r.wq, r.wk, r.inv_freq, r.positions, qo.data_ptr(),
                                            ko.defined() ? ko.data_ptr() : nullptr, r.T, r.H, r.Hk, r.d, r.rot, r.q_st, r.q_sh,
                                            r.k_st, r.k_sh, eps, r.dtype, flags, r.c.stream());
        return rc != SSM_OK ? PyLong_FromLong(rc) : pair(qo, ko);
    });
}

PyObject *rope_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject * {
        const float eps = number(a[8], "eps");
        const uint32_t flags = flag_bits(a[9]);
        const Rope r(a, flags);
        const bool has_k = a[1] != Py_None;
        const Tensor &gq = tensor(a[6], "dq_out");
        const void *pgq = r.c.view(gq, "dq_out", r.type, {r.T, r.H, r.d}), *pgk = nullptr;
        int64_t gk_st = 0, gk_sh = 0;
        if (has_k) {
            const Tensor &gk = tensor(a[7], "dk_out");
            pgk = r.c.view(gk, "dk_out", r.type, {r.T, r.Hk, r.d});
            gk_st = gk.stride(0); gk_sh = gk.stride(1);
        }
        const size_t need = ssm_qk_norm_rope_bwd_workspace_size(r.T, r.H, r.Hk, r.d, flags);
        const auto f32 = ScalarType::Float;
        Tensor dq, dk, dwq, dwk, ws;
        bool given = !has_k || !r.norm;
        for (int i = 10; i < 15; ++i) given = given || a[i] != Py_None;
        if (!given && r.c.few(r.T * (r.H + r.Hk) * r.d)) {
            // (of few tokens the workspace is a part of the outputs' size)
            std::tie(dq, dk, dwq, dwk, ws) = std::tuple_cat(
                r.c.make_together<5>({{r.type, {r.T, r.H, r.d}}, {r.type, {r.T, r.Hk, r.d}}, {f32, {r.d}}, {f32, {r.d}},
                                      {ScalarType::Byte, {(int64_t)need}}}));
        } else {
            dq = r.c.out(a[10], "dq", r.type, {r.T, r.H, r.d});
            if (has_k) dk = r.c.out(a[11], "dk", r.type, {r.T, r.Hk, r.d});
            if (r.norm && has_k && a[12] == Py_None && a[13] == Py_None) {
                std::tie(dwq, dwk) = std::tuple_cat(r.c.make_together<2>({{f32, {r.d}}, {f32, {r.d}}}));
            } else if (r.norm) {
                dwq = r.c.out(a[12], "dwq", f32, {r.d});
                if (has_k) dwk = r.c.out(a[13], "dwk", f32, {r.d});
            }
            ws = r.c.workspace(a[14], need);
        }
        auto at_ = [](const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
        const int rc = ssm_qk_norm_rope_bwd(r.q, r.k, r.wq, r.wk, r.inv_freq, r.positions, pgq, pgk, at_(dq), at_(dk),
                                            (float *)at_(dwq), (float *)at_(dwk), r.T, r.H, r.Hk, r.d, r.rot, r.q_st, r.q_sh,
                                            r.k_st, r.k_sh, gq.stride(0), gq.stride(1), gk_st, gk_sh, eps, r.dtype, flags,
                                            ws.data_ptr(), ws.nbytes(), r.c.stream());
        if (rc != SSM_OK) return PyLong_FromLong(rc);
        PyObject *d = PyDict_New();
        set(d, "dq", dq);
        if (dk.defined()) set(d, "dk", dk); else PyDict_SetItemString(d, "dk", Py_None);
        if (dwq.defined()) set(d, "dwq", dwq); else PyDict_SetItemString(d, "dwq", Py_None);
        if (dwk.defined()) set(d, "dwk", dwk); else PyDict_SetItemString(d, "dwk", Py_None);
        return d;
    });
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

PyObject *rope_cache_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject * {
        const float eps = number(a[10], "eps"), k_scale = number(a[11], "k_scale"), v_scale = number(a[12], "v_scale");
        const uint32_t flags = flag_bits(a[13]);
        const Rope r(a, flags);
        const Tensor &v = tensor(a[6], "v");
        const void *pv = r.c.view(v, "v", r.type, {r.T, r.Hk, r.d});
        auto *ps = (const int64_t *)r.c.whole(a[7], "slots", ScalarType::Long, {r.T});
        const Caches k(r.c, a[8], a[9]);
        if (k.Hk != r.Hk || k.d != r.d)
            refuse(PyExc_ValueError, "k_cache: shape " + show({k.pages, k.page_size, k.Hk, k.d}) + ", expected (pages, page_size, " +
                                         std::to_string(r.Hk) + ", " + std::to_string(r.d) + ")");
        const Tensor qo = r.c.out(a[14], "q_out", r.type, {r.T, r.H, r.d});
        const int rc = ssm_qk_norm_rope_cache_fwd(
            r.q, r.k, pv, r.wq, r.wk, r.inv_freq, r.positions, ps, qo.data_ptr(), k.k, k.v, r.T, r.H, r.Hk, r.d, r.rot, k.pages,
            k.page_size, r.q_st, r.q_sh, r.k_st, r.k_sh, v.stride(0), v.stride(1), k.sp, k.st, k.sh, eps, k_scale, v_scale, r.dtype,
            k.kv, flags, r.c.stream());
        return rc != SSM_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(qo);
    });
}

PyObject *attn_decode_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject * {
        const Tensor &q = tensor(a[0], "q"), &table = tensor(a[3], "block_table");
        const Call c(q);
        dims(q, "q", 3, "(batch, heads, headdim)");
        const ssm_dtype_t dtype = head_dtype(q, "q");
        const ScalarType type = q.scalar_type();
        const int64_t B = q.size(0), H = q.size(1), d = q.size(2);
        const void *pq = c.view(q, "q", type, q.sizes());
        const Caches k(c, a[1], a[2]);
        if (k.d != d)
            refuse(PyExc_ValueError, "k_cache: shape " + show({k.pages, k.page_size, k.Hk, k.d}) + ", expected headdim " +
                                         std::to_string(d));
        dims(table, "block_table", 2, "(batch, max_pages)");
        const int64_t cols = table.size(1);
        auto *pt = (const int32_t *)c.view(table, "block_table", ScalarType::Int, {B, cols});
        auto *pl = (const int32_t *)c.whole(a[4], "lens", ScalarType::Int, {B});
        const float scale = number(a[5], "scale"), k_scale = number(a[7], "k_scale"), v_scale = number(a[8], "v_scale");
        const int64_t window = whole_number(a[6], "window");
        const int asked = PyObject_IsTrue(a[9]);
        if (asked < 0) throw Refused{};          // with the error that its truth raised
        const bool want_lse = a[11] != Py_None || asked == 1;
        Tensor o, lse;
        if (want_lse && a[10] == Py_None && a[11] == Py_None && c.few(B * H * d)) {
            std::tie(o, lse) = std::tuple_cat(c.make_together<2>({{type, {B, H, d}}, {ScalarType::Float, {B, H}}}));
        } else {
            o = c.out(a[10], "o", type, {B, H, d});
            if (want_lse) lse = c.out(a[11], "lse", ScalarType::Float, {B, H});
        }
        const Tensor ws = c.workspace(a[12], ssm_paged_attn_decode_fwd_workspace_size(B, H, k.Hk, d, cols, k.page_size));
        const int rc = ssm_paged_attn_decode_fwd(
            pq, k.k, k.v, pt, pl, o.data_ptr(), want_lse ? (float *)lse.data_ptr() : nullptr, B, H, k.Hk, d, cols,
            B > 1 ? table.stride(0) : cols, k.pages, k.page_size, q.stride(0), q.stride(1), k.sp, k.st, k.sh, scale, window, k_scale,
            v_scale, dtype, k.kv, ws.data_ptr(), ws.nbytes(), c.stream());
        if (rc != SSM_OK) return PyLong_FromLong(rc);
        return want_lse ? pair(o, lse) : THPVariable_Wrap(o);
    });
}

PyMethodDef methods[] = {
    {"pages_step", (PyCFunction)(void (*)(void))pages_step, METH_FASTCALL, nullptr},
    {"rope_fwd", (PyCFunction)(void (*)(void))rope_fwd, METH_FASTCALL, nullptr},
    {"rope_bwd", (PyCFunction)(void (*)(void))rope_bwd, METH_FASTCALL, nullptr},
    {"rope_cache_fwd", (PyCFunction)(void (*)(void))rope_cache_fwd, METH_FASTCALL, nullptr},
    {"attn_decode_fwd", (PyCFunction)(void (*)(void))attn_decode_fwd, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_bind(void) { return PyModule_Create(&module); }
