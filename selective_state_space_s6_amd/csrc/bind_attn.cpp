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
#include "bind_common.hpp"
#include "bind_longctx.hpp"

namespace {

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
    {"prefix_attn_fwd", (PyCFunction)(void (*)(void))ssm_bind::prefix_attn_fwd, METH_FASTCALL, nullptr},
    {"page_bounds", (PyCFunction)(void (*)(void))ssm_bind::page_bounds, METH_FASTCALL, nullptr},
    {"page_select", (PyCFunction)(void (*)(void))ssm_bind::page_select, METH_FASTCALL, nullptr},
    {"select_attn_fwd", (PyCFunction)(void (*)(void))ssm_bind::select_attn_fwd, METH_FASTCALL, nullptr},
    {"mass_update", (PyCFunction)(void (*)(void))ssm_bind::mass_update, METH_FASTCALL, nullptr},
    {"evict", (PyCFunction)(void (*)(void))ssm_bind::evict, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_bind(void) { return PyModule_Create(&module); }
