// bind_longctx.cpp -- the Python binding of include/ssm_longctx.h's entry points, in the manner and
// the module of bind_attn.cpp.
#include "bind_common.hpp"
#include "bind_longctx.hpp"

namespace {

constexpr auto kI32 = ScalarType::Int;
constexpr auto kF32 = ScalarType::Float;

// q (rows, heads, headdim) beside a cache
struct Queries {
    ScalarType type;
    ssm_dtype_t dtype;
    int64_t rows, H, d, sr, sh;
    const void *p;
    Queries(const Call &c, const Tensor &q, const char *form) {
        dims(q, "q", 3, form);
        dtype = head_dtype(q, "q");
        type = q.scalar_type();
        rows = q.size(0); H = q.size(1); d = q.size(2);
        p = c.view(q, "q", type, q.sizes());
        sr = q.stride(0); sh = q.stride(1);
    }
    void match(int64_t pages, int64_t page_size, int64_t Hk, int64_t kd) const {
        if (kd != d)
            refuse(PyExc_ValueError, "k_cache: shape " + show({pages, page_size, Hk, kd}) + ", expected headdim " + std::to_string(d));
    }
};

// an int32 table of pages (rows, cols), rows strided
struct Table {
    const int32_t *p;
    int64_t rows, cols, stride;
    Table(const Call &c, PyObject *o, const char *name, const char *form) {
        const Tensor &t = tensor(o, name);
        dims(t, name, 2, form);
        rows = t.size(0); cols = t.size(1);
        p = (const int32_t *)c.view(t, name, kI32, t.sizes());
        stride = rows > 1 ? t.stride(0) : cols;
    }
    void count(int64_t want, const char *name) const {
        if (rows != want) refuse(PyExc_ValueError, std::string(name) + ": " + std::to_string(rows) + " rows, expected " + std::to_string(want));
    }
};

// the key cache alone
struct Keys {
    const void *p;
    int64_t pages, page_size, Hk, d, sp, st, sh;
    ScalarType type;
    ssm_kv_dtype_t kv;
    Keys(const Call &c, PyObject *o) {
        const Tensor &t = tensor(o, "k_cache");
        type = t.scalar_type();
        kv = kv_type(type, "k_cache");
        dims(t, "k_cache", 4, "(pages, page_size, kv_heads, headdim)");
        p = c.view(t, "k_cache", type, t.sizes());
        pages = t.size(0); page_size = t.size(1); Hk = t.size(2); d = t.size(3);
        sp = t.stride(0); st = t.stride(1); sh = t.stride(2);
    }
    static ssm_kv_dtype_t kv_type(ScalarType t, const char *name) {
        switch (t) {
            case ScalarType::Float: return SSM_KV_F32;
            case ScalarType::BFloat16: return SSM_KV_BF16;
            case ScalarType::Float8_e4m3fn: return SSM_KV_F8E4M3;
            default: refuse(PyExc_TypeError, std::string(name) + ": dtype " + show(t) + ", expected float32, bfloat16 or float8_e4m3fn");
        }
    }
};

// o and (asked for, or given) lse of an attention call
struct Outputs {
    Tensor o, lse;
    bool want;
    Outputs(const Call &c, const Queries &q, PyObject *asked_for, PyObject *po, PyObject *pl) {
        const int asked = PyObject_IsTrue(asked_for);
        if (asked < 0) throw Refused{};          // with the error that its truth raised
        want = pl != Py_None || asked == 1;
        if (want && po == Py_None && pl == Py_None && c.few(q.rows * q.H * q.d)) {
            std::tie(o, lse) = std::tuple_cat(c.make_together<2>({{q.type, {q.rows, q.H, q.d}}, {kF32, {q.rows, q.H}}}));
        } else {
            o = c.out(po, "o", q.type, {q.rows, q.H, q.d});
            if (want) lse = c.out(pl, "lse", kF32, {q.rows, q.H});
        }
    }
    float *at_lse() const { return want ? (float *)lse.data_ptr() : nullptr; }
    PyObject *result(int rc) const {
        if (rc != SSM_OK) return PyLong_FromLong(rc);
        return want ? pair(o, lse) : THPVariable_Wrap(o);
    }
};

}  // namespace

namespace ssm_bind {

PyObject *prefix_attn_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject * {
        const Tensor &tq = tensor(a[0], "q");
        const Call c(tq);
        const Queries q(c, tq, "(batch, heads, headdim)");
        const Caches k(c, a[1], a[2]);
        q.match(k.pages, k.page_size, k.Hk, k.d);
        auto *prefix = (const int32_t *)c.whole(a[3], "prefix", kI32, {q.rows});
        const Table pt(c, a[4], "prefix_table", "(prefixes, max_prefix_pages)"), bt(c, a[6], "block_table", "(batch, max_pages)");
        bt.count(q.rows, "block_table");
        auto *plens = (const int32_t *)c.whole(a[5], "prefix_lens", kI32, {pt.rows});
        auto *lens = (const int32_t *)c.whole(a[7], "lens", kI32, {q.rows});
        const float scale = number(a[8], "scale"), k_scale = number(a[9], "k_scale"), v_scale = number(a[10], "v_scale");
        const Outputs out(c, q, a[11], a[12], a[13]);
        const Tensor ws = c.workspace(a[14], ssm_prefix_attn_decode_fwd_workspace_size(q.rows, q.H, k.Hk, q.d, pt.cols, bt.cols, k.page_size));
        return out.result(ssm_prefix_attn_decode_fwd(
            q.p, k.k, k.v, prefix, pt.p, plens, bt.p, lens, out.o.data_ptr(), out.at_lse(), q.rows, q.H, k.Hk, q.d, pt.rows, pt.cols,
            pt.stride, bt.cols, bt.stride, k.pages, k.page_size, q.sr, q.sh, k.sp, k.st, k.sh, scale, k_scale, v_scale, q.dtype,
            k.kv, ws.data_ptr(), ws.nbytes(), c.stream()));
    });
}

PyObject *page_bounds(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject * {
        const Call c(tensor(a[0], "k_cache"));
        const Keys k(c, a[0]);
        void *bounds = c.whole(a[1], "bounds", k.type, {k.pages, k.Hk, 2, k.d});
        const Table bt(c, a[2], "block_table", "(batch, max_pages)");
        auto *old = (const int32_t *)c.whole(a[3], "len_old", kI32, {bt.rows});
        auto *lens = (const int32_t *)c.whole(a[4], "lens", kI32, {bt.rows});
        return PyLong_FromLong(ssm_kv_page_bounds_update(k.p, bounds, bt.p, old, lens, bt.rows, k.Hk, k.d, bt.cols, bt.stride, k.pages,
                                                         k.page_size, k.sp, k.st, k.sh, k.kv, c.stream()));
    });
}

PyObject *page_select(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const Tensor &tq = tensor(a[0], "q"), &b = tensor(a[1], "bounds");
        const Call c(tq);
        const Queries q(c, tq, "(batch, heads, headdim)");
        dims(b, "bounds", 4, "(pages, kv_heads, 2, headdim)");
        const int64_t pages = b.size(0), Hk = b.size(1);
        const ssm_kv_dtype_t kv = Keys::kv_type(b.scalar_type(), "bounds");
        const void *bounds = c.whole(a[1], "bounds", b.scalar_type(), {pages, Hk, 2, q.d});
        const Table bt(c, a[2], "block_table", "(batch, max_pages)");
        bt.count(q.rows, "block_table");
        auto *lens = (const int32_t *)c.whole(a[3], "lens", kI32, {q.rows});
        const int64_t page_size = whole_number(a[4], "page_size"), top_k = whole_number(a[5], "top_k"),
                      first = whole_number(a[6], "first"), last = whole_number(a[7], "last");
        if (top_k < 1 || top_k > (1 << 20)) refuse(PyExc_ValueError, "top_k: " + std::to_string(top_k) + ", expected 1 to 2^20");
        const Tensor out = c.out(a[8], "selected", kI32, {q.rows, Hk, top_k});
        const Tensor ws = c.workspace(a[9], ssm_kv_page_select_fwd_workspace_size(q.rows, Hk, bt.cols, top_k));
        const int rc = ssm_kv_page_select_fwd(q.p, bounds, bt.p, lens, (int32_t *)out.data_ptr(), q.rows, q.H, Hk, q.d, bt.cols, bt.stride,
                                              pages, page_size, top_k, first, last, q.sr, q.sh, q.dtype, kv, ws.data_ptr(), ws.nbytes(),
                                              c.stream());
        return rc != SSM_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
    });
}

PyObject *select_attn_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject * {
        const Tensor &tq = tensor(a[0], "q"), &sel = tensor(a[5], "selected");
        const Call c(tq);
        const Queries q(c, tq, "(batch, heads, headdim)");
        const Caches k(c, a[1], a[2]);
        q.match(k.pages, k.page_size, k.Hk, k.d);
        const Table bt(c, a[3], "block_table", "(batch, max_pages)");
        bt.count(q.rows, "block_table");
        auto *lens = (const int32_t *)c.whole(a[4], "lens", kI32, {q.rows});
        dims(sel, "selected", 3, "(batch, kv_heads, top_k)");
        const int64_t top_k = sel.size(2);
        auto *ps = (const int32_t *)c.whole(a[5], "selected", kI32, {q.rows, k.Hk, top_k});
        const float scale = number(a[6], "scale"), k_scale = number(a[7], "k_scale"), v_scale = number(a[8], "v_scale");
        const Outputs out(c, q, a[9], a[10], a[11]);
        const Tensor ws = c.workspace(a[12], ssm_select_attn_decode_fwd_workspace_size(q.rows, q.H, k.Hk, q.d, bt.cols, k.page_size, top_k));
        return out.result(ssm_select_attn_decode_fwd(
            q.p, k.k, k.v, bt.p, lens, ps, out.o.data_ptr(), out.at_lse(), q.rows, q.H, k.Hk, q.d, bt.cols, bt.stride, k.pages,
            k.page_size, top_k, q.sr, q.sh, k.sp, k.st, k.sh, scale, k_scale, v_scale, q.dtype, k.kv, ws.data_ptr(), ws.nbytes(),
            c.stream()));
    });
}

PyObject *mass_update(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject * {
        const Tensor &tq = tensor(a[0], "q");
        const Call c(tq);
        const Queries q(c, tq, "(tokens, heads, headdim)");
        const Keys k(c, a[1]);
        q.match(k.pages, k.page_size, k.Hk, k.d);
        auto *lse = (const float *)c.whole(a[2], "lse", kF32, {q.rows, q.H});
        auto *mass = (float *)c.whole(a[3], "mass", kF32, {k.pages, k.Hk, k.page_size});
        const Table bt(c, a[4], "block_table", "(batch, max_pages)");
        auto *starts = (const int32_t *)c.whole(a[5], "starts", kI32, {bt.rows + 1});
        auto *positions = (const int32_t *)c.whole(a[6], "positions", kI32, {q.rows});
        auto *old = (const int32_t *)c.whole(a[7], "len_old", kI32, {bt.rows});
        auto *lens = (const int32_t *)c.whole(a[8], "lens", kI32, {bt.rows});
        const float scale = number(a[9], "scale"), k_scale = number(a[10], "k_scale");
        return PyLong_FromLong(ssm_kv_mass_update(q.p, k.p, lse, mass, bt.p, starts, positions, old, lens, q.rows, bt.rows, q.H, k.Hk,
                                                  q.d, bt.cols, bt.stride, k.pages, k.page_size, q.sr, q.sh, k.sp, k.st, k.sh, scale,
                                                  k_scale, q.dtype, k.kv, c.stream()));
    });
}

PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const Call c(tensor(a[0], "k_cache"));
        const Caches k(c, a[0], a[1]);
        auto *mass = (float *)c.whole(a[2], "mass", kF32, {k.pages, k.Hk, k.page_size});
        const Table bt(c, a[3], "block_table", "(batch, max_pages)");
        auto *lens = (const int32_t *)c.whole(a[4], "lens", kI32, {bt.rows});
        const int64_t budget = whole_number(a[5], "budget"), recent = whole_number(a[6], "recent");
        if (budget < 1 || budget > (1 << 30)) refuse(PyExc_ValueError, "budget: " + std::to_string(budget) + ", expected 1 to 2^30");
        const Tensor len_out = c.out(a[7], "len_out", kI32, {bt.rows}), kept = c.out(a[8], "kept", kI32, {bt.rows, k.Hk, budget});
        const int rc = ssm_kv_evict(k.k, k.v, mass, bt.p, lens, (int32_t *)len_out.data_ptr(), (int32_t *)kept.data_ptr(), bt.rows, k.Hk,
                                    k.d, bt.cols, bt.stride, k.pages, k.page_size, budget, recent, k.sp, k.st, k.sh, k.kv, c.stream());
        return rc != SSM_OK ? PyLong_FromLong(rc) : pair(len_out, kept);
    });
}

}  // namespace ssm_bind
