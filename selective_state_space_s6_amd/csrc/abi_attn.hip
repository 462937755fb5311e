// abi_attn.hip -- the extern "C" boundary of include/ssm_attn.h: argument
// validation, workspace sizing, and dispatch to the kernel launchers.  Every
// check runs before any HIP call.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ssm_attn.h"
#include "abi_common.hpp"
#include "attn_launchers.hpp"

using ssm::fail;
using ssm::launched;
using ssm::too_big;

namespace {

constexpr int64_t k2p31 = int64_t(1) << 31;

#define REQUIRE_NOT_NEG(entry, v)                                                                 \
    do {                                                                                          \
        if ((v) < 0) return fail(SSM_ERR_INVALID_ARG, "%s: %s must be >= 0 (got %lld)", entry, #v, \
                                 (long long)(v));                                                 \
    } while (0)

// two tensors of one call that may not share their first element
struct Named { const void *p; const char *name; };
int check_alias(const char *E, const Named *outs, int no, const Named *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        if (outs[i].p == nullptr) continue;
        for (int j = 0; j < ni; ++j)
            if (outs[i].p == ins[j].p) return fail(SSM_ERR_INVALID_ARG, "%s: %s aliases %s", E, outs[i].name, ins[j].name);
        for (int j = i + 1; j < no; ++j)
            if (outs[i].p == outs[j].p) return fail(SSM_ERR_INVALID_ARG, "%s: %s aliases %s", E, outs[i].name, outs[j].name);
    }
    return SSM_OK;
}

// elements of `dtype` start at multiples of their size
int check_element(const char *E, const void *p, const char *name, int esize) {
    if (((uintptr_t)p & (uintptr_t)(esize - 1)) != 0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: %s is not aligned to its elements", E, name);
    return SSM_OK;
}

// heads (n_tokens, n_heads, headdim) without a gap; strides of a dim of one entry are not used
bool gapless(int64_t n_tokens, int64_t n_heads, int64_t headdim, int64_t st, int64_t sh) {
    return (n_heads == 1 || sh == headdim) && (n_tokens == 1 || st == n_heads * headdim);
}

// what the norm and rotation entry points have in common; n_kv_heads may be 0
int check_rope(const char *E, const void *q, const void *k, const float *wq, const float *wk, const float *inv_freq,
               const int32_t *positions, int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
               int64_t rot_dim, float eps, ssm_dtype_t dtype, uint32_t flags) {
    REQUIRE_NOT_NEG(E, n_tokens); REQUIRE_POS(E, n_heads); REQUIRE_NOT_NEG(E, n_kv_heads); REQUIRE_POS(E, headdim);
    if (dtype != SSM_F32 && dtype != SSM_BF16)
        return fail(SSM_ERR_INVALID_ARG, "%s: dtype %d is not SSM_F32 or SSM_BF16", E, (int)dtype);
    if ((flags & ~(SSM_ROPE_INTERLEAVED | SSM_QK_NO_NORM)) != 0)
        return fail(SSM_ERR_INVALID_ARG, "%s: flags 0x%x: only SSM_ROPE_INTERLEAVED and SSM_QK_NO_NORM apply", E, flags);
    if (headdim > SSM_ATTN_MAX_HEADDIM)
        return fail(SSM_ERR_UNSUPPORTED, "%s: headdim %lld > %d", E, (long long)headdim, SSM_ATTN_MAX_HEADDIM);
    if (rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > headdim)
        return fail(SSM_ERR_INVALID_ARG, "%s: rot_dim %lld must be even, >= 0 and <= headdim %lld", E,
                    (long long)rot_dim, (long long)headdim);
    if (n_tokens >= k2p31 / 4 || n_heads > 65536 || n_kv_heads > 65536 || too_big(n_tokens, n_heads + n_kv_heads, headdim, 1))
        return fail(SSM_ERR_UNSUPPORTED, "%s: problem too large", E);
    const bool norm = (flags & SSM_QK_NO_NORM) == 0;
    if (norm && !(eps >= 0.0f && eps < INFINITY))
        return fail(SSM_ERR_INVALID_ARG, "%s: eps must be >= 0 and finite", E);
    if (n_tokens == 0) return SSM_OK;
    REQUIRE_PTR(E, q);
    if (n_kv_heads > 0) REQUIRE_PTR(E, k);
    if (norm) {
        REQUIRE_PTR(E, wq);
        if (n_kv_heads > 0) REQUIRE_PTR(E, wk);
    }
    if (rot_dim > 0) { REQUIRE_PTR(E, inv_freq); REQUIRE_PTR(E, positions); }
    return SSM_OK;
}

// cache strides: rows must not overlap by sign, and every offset must fit the kernels' arithmetic
int check_cache(const char *E, int64_t n_pages, int64_t page_size, int64_t n_kv_heads, int64_t headdim,
                int64_t sp, int64_t st, int64_t sh, int esize) {
    REQUIRE_POS(E, n_pages); REQUIRE_POS(E, page_size);
    if (n_pages >= k2p31 || page_size >= k2p31 || n_pages * page_size >= k2p31)
        return fail(SSM_ERR_UNSUPPORTED, "%s: n_pages * page_size must be below 2^31", E);
    if (sp < 0 || st < 0 || sh < 0)
        return fail(SSM_ERR_INVALID_ARG, "%s: cache strides must be >= 0", E);
    const double extent = ((double)(n_pages - 1) * (double)sp + (double)(page_size - 1) * (double)st +
                           (double)(n_kv_heads - 1) * (double)sh + (double)headdim) * esize;
    if (extent >= 68719476736.0) return fail(SSM_ERR_UNSUPPORTED, "%s: a cache's extent must be below 2^36 bytes", E);
    return SSM_OK;
}

}  // namespace

extern "C" {

int ssm_kv_pages_step(const int32_t *len_old, const int32_t *len_new, int32_t *block_table,
                      int32_t *free_ring, const int32_t *ring, int32_t *ring_out, int32_t *len_out,
                      int32_t *starts, int32_t *request, int32_t *positions, int64_t *slots, int32_t *denied,
                      int64_t batch, int64_t max_pages, int64_t table_stride, int64_t n_pages,
                      int64_t page_size, int64_t n_tokens, hipStream_t stream) {
    const char *E = "ssm_kv_pages_step";
    REQUIRE_PTR(E, len_old); REQUIRE_PTR(E, len_new); REQUIRE_PTR(E, block_table); REQUIRE_PTR(E, free_ring);
    REQUIRE_PTR(E, ring); REQUIRE_PTR(E, ring_out); REQUIRE_PTR(E, len_out); REQUIRE_PTR(E, starts);
    REQUIRE_PTR(E, denied);
    REQUIRE_POS(E, batch); REQUIRE_POS(E, max_pages); REQUIRE_POS(E, n_pages); REQUIRE_POS(E, page_size);
    REQUIRE_NOT_NEG(E, n_tokens);
    if (batch > SSM_KV_MAX_BATCH)
        return fail(SSM_ERR_UNSUPPORTED, "%s: batch %lld > %d", E, (long long)batch, SSM_KV_MAX_BATCH);
    if (table_stride < max_pages)
        return fail(SSM_ERR_INVALID_ARG, "%s: table_stride %lld < max_pages %lld", E, (long long)table_stride,
                    (long long)max_pages);
    if (max_pages >= k2p31 / batch || n_pages >= k2p31 || page_size >= k2p31 || n_pages * page_size >= k2p31 ||
        n_tokens >= k2p31 || table_stride >= (int64_t(1) << 40))
        return fail(SSM_ERR_UNSUPPORTED, "%s: problem too large", E);
    if (n_tokens > 0) { REQUIRE_PTR(E, request); REQUIRE_PTR(E, positions); REQUIRE_PTR(E, slots); }
    REQUIRE_ALIGN(E, request); REQUIRE_ALIGN(E, positions); REQUIRE_ALIGN(E, slots);
    const Named outs[] = {{block_table, "block_table"}, {free_ring, "free_ring"}, {ring_out, "ring_out"},
                          {len_out, "len_out"}, {starts, "starts"}, {request, "request"}, {positions, "positions"},
                          {slots, "slots"}, {denied, "denied"}};
    const Named ins[] = {{len_old, "len_old"}, {len_new, "len_new"}, {ring, "ring"}};
    const int rc = check_alias(E, outs, 9, ins, 3);
    if (rc != SSM_OK) return rc;
    ssm::KvPagesArgs a{len_old, len_new, block_table, free_ring, ring, ring_out, len_out, starts, request, positions,
                       slots, denied, (int32_t)batch, (int32_t)max_pages, table_stride, (int32_t)n_pages,
                       (int32_t)page_size, (int32_t)n_tokens};
    const char *kn = "kv_pages_kernel";
    return launched(E, ssm::launch_kv_pages(a, stream, &kn), kn);
}

int ssm_qk_norm_rope_fwd(const void *q, const void *k, const float *wq, const float *wk,
                         const float *inv_freq, const int32_t *positions, void *q_out, void *k_out,
                         int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads, int64_t headdim, int64_t rot_dim,
                         int64_t q_stride_token, int64_t q_stride_head,
                         int64_t k_stride_token, int64_t k_stride_head,
                         float eps, ssm_dtype_t dtype, uint32_t flags, hipStream_t stream) {
    const char *E = "ssm_qk_norm_rope_fwd";
    int rc = check_rope(E, q, k, wq, wk, inv_freq, positions, n_tokens, n_heads, n_kv_heads, headdim, rot_dim, eps,
                        dtype, flags);
    if (rc != SSM_OK || n_tokens == 0) return rc;
    REQUIRE_PTR(E, q_out);
    if (n_kv_heads > 0) REQUIRE_PTR(E, k_out);
    const int es = dtype == SSM_BF16 ? 2 : 4;
    const Named ts[] = {{q, "q"}, {k, "k"}, {q_out, "q_out"}, {k_out, "k_out"}};
    for (const Named &t : ts)
        if ((rc = check_element(E, t.p, t.name, es)) != SSM_OK) return rc;
    // in place only where the layout is the output's
    if (q_out == q && !gapless(n_tokens, n_heads, headdim, q_stride_token, q_stride_head))
        return fail(SSM_ERR_INVALID_ARG, "%s: q_out aliases a q that is not contiguous", E);
    if (n_kv_heads > 0 && k_out == k && !gapless(n_tokens, n_kv_heads, headdim, k_stride_token, k_stride_head))
        return fail(SSM_ERR_INVALID_ARG, "%s: k_out aliases a k that is not contiguous", E);
    if (n_kv_heads > 0 && (q_out == k || k_out == q || q_out == k_out))
        return fail(SSM_ERR_INVALID_ARG, "%s: an output aliases the other tensor", E);
    const bool norm = (flags & SSM_QK_NO_NORM) == 0;
    const Named outs[] = {{q_out, "q_out"}, {n_kv_heads > 0 ? k_out : nullptr, "k_out"}};
    const Named ins[] = {{norm ? wq : nullptr, "wq"}, {norm && n_kv_heads > 0 ? wk : nullptr, "wk"}, {rot_dim > 0 ? inv_freq : nullptr, "inv_freq"},
                         {rot_dim > 0 ? positions : nullptr, "positions"}};
    if ((rc = check_alias(E, outs, 2, ins, 4)) != SSM_OK) return rc;
    ssm::QkRopeArgs a{};
    a.q = q; a.k = k; a.wq = wq; a.wk = wk; a.inv_freq = inv_freq; a.positions = positions;
    a.q_out = q_out; a.k_out = k_out;
    a.n_tokens = n_tokens; a.n_heads = n_heads; a.n_kv_heads = n_kv_heads;
    a.headdim = (int)headdim; a.rot_dim = (int)rot_dim;
    a.q_st = n_tokens > 1 ? q_stride_token : 0; a.q_sh = n_heads > 1 ? q_stride_head : 0;
    a.k_st = n_tokens > 1 ? k_stride_token : 0; a.k_sh = n_kv_heads > 1 ? k_stride_head : 0;
    a.eps = eps; a.bf16 = dtype == SSM_BF16; a.flags = flags;
    const char *kn = "qk_rope_kernel";
    return launched(E, ssm::launch_qk_rope(a, stream, &kn), kn);
}

size_t ssm_qk_norm_rope_bwd_workspace_size(int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads,
                                           int64_t headdim, uint32_t flags) {
    if (n_tokens <= 0 || n_heads <= 0 || n_kv_heads < 0 || headdim <= 0) return 0;
    return ssm::qk_rope_bwd_workspace_bytes(n_tokens, n_heads, n_kv_heads, headdim, flags);
}

int ssm_qk_norm_rope_bwd(const void *q, const void *k, const float *wq, const float *wk,
                         const float *inv_freq, const int32_t *positions,
                         const void *dq_out, const void *dk_out, void *dq, void *dk, float *dwq, float *dwk,
                         int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads, int64_t headdim, int64_t rot_dim,
                         int64_t q_stride_token, int64_t q_stride_head,
                         int64_t k_stride_token, int64_t k_stride_head,
                         int64_t dq_stride_token, int64_t dq_stride_head,
                         int64_t dk_stride_token, int64_t dk_stride_head,
                         float eps, ssm_dtype_t dtype, uint32_t flags,
                         void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const char *E = "ssm_qk_norm_rope_bwd";
    int rc = check_rope(E, q, k, wq, wk, inv_freq, positions, n_tokens, n_heads, n_kv_heads, headdim, rot_dim, eps,
                        dtype, flags);
    if (rc != SSM_OK) return rc;
    const bool norm = (flags & SSM_QK_NO_NORM) == 0, has_k = n_kv_heads > 0;
    if (norm) {
        REQUIRE_PTR(E, dwq);
        if (has_k) REQUIRE_PTR(E, dwk);
    }
    if (n_tokens == 0 && !norm) return SSM_OK;
    if (n_tokens > 0) {
        REQUIRE_PTR(E, dq_out); REQUIRE_PTR(E, dq);
        if (has_k) { REQUIRE_PTR(E, dk_out); REQUIRE_PTR(E, dk); }
    }
    const int es = dtype == SSM_BF16 ? 2 : 4;
    const Named ts[] = {{q, "q"}, {k, "k"}, {dq_out, "dq_out"}, {dk_out, "dk_out"}, {dq, "dq"}, {dk, "dk"}};
    for (const Named &t : ts)
        if ((rc = check_element(E, t.p, t.name, es)) != SSM_OK) return rc;
    if (n_tokens > 0 && dq == dq_out && !gapless(n_tokens, n_heads, headdim, dq_stride_token, dq_stride_head))
        return fail(SSM_ERR_INVALID_ARG, "%s: dq aliases a dq_out that is not contiguous", E);
    if (n_tokens > 0 && has_k && dk == dk_out && !gapless(n_tokens, n_kv_heads, headdim, dk_stride_token, dk_stride_head))
        return fail(SSM_ERR_INVALID_ARG, "%s: dk aliases a dk_out that is not contiguous", E);
    const size_t need = ssm_qk_norm_rope_bwd_workspace_size(n_tokens, n_heads, n_kv_heads, headdim, flags);
    const Named outs[] = {{dq, "dq"}, {has_k ? dk : nullptr, "dk"}, {norm ? dwq : nullptr, "dwq"},
                          {norm && has_k ? dwk : nullptr, "dwk"}, {need > 0 ? workspace : nullptr, "workspace"}};
    const Named ins[] = {{q, "q"}, {has_k ? k : nullptr, "k"}, {norm ? wq : nullptr, "wq"}, {norm && has_k ? wk : nullptr, "wk"},
                         {rot_dim > 0 ? inv_freq : nullptr, "inv_freq"}, {rot_dim > 0 ? positions : nullptr, "positions"}};
    if ((rc = check_alias(E, outs, 5, ins, 6)) != SSM_OK) return rc;
    // a side's blocks may overwrite their own cotangents, not those that the other side's still read
    const Named gq = {dq_out, "dq_out"}, gk = {has_k ? dk_out : nullptr, "dk_out"}, both[] = {gq, gk};
    if ((rc = check_alias(E, outs, 1, &gk, 1)) != SSM_OK) return rc;
    if ((rc = check_alias(E, outs + 1, 1, &gq, 1)) != SSM_OK) return rc;
    if ((rc = check_alias(E, outs + 2, 3, both, 2)) != SSM_OK) return rc;
    REQUIRE_ALIGN(E, workspace);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", E, need,
                    workspace ? workspace_bytes : (size_t)0);
    ssm::QkRopeBwdArgs a{q, k, wq, wk, inv_freq, positions, dq_out, dk_out, dq, dk, dwq, dwk,
                         n_tokens, n_heads, n_kv_heads, (int)headdim, (int)rot_dim,
                         n_tokens > 1 ? q_stride_token : 0, n_heads > 1 ? q_stride_head : 0,
                         n_tokens > 1 ? k_stride_token : 0, n_kv_heads > 1 ? k_stride_head : 0,
                         n_tokens > 1 ? dq_stride_token : 0, n_heads > 1 ? dq_stride_head : 0,
                         n_tokens > 1 ? dk_stride_token : 0, n_kv_heads > 1 ? dk_stride_head : 0,
                         eps, dtype == SSM_BF16, flags, workspace};
    const char *kn = "qk_rope_bwd_kernel";
    return launched(E, ssm::launch_qk_rope_bwd(a, stream, &kn), kn);
}

int ssm_qk_norm_rope_cache_fwd(const void *q, const void *k, const void *v, const float *wq, const float *wk,
                               const float *inv_freq, const int32_t *positions, const int64_t *slots,
                               void *q_out, void *k_cache, void *v_cache,
                               int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                               int64_t rot_dim, int64_t n_pages, int64_t page_size,
                               int64_t q_stride_token, int64_t q_stride_head,
                               int64_t k_stride_token, int64_t k_stride_head,
                               int64_t v_stride_token, int64_t v_stride_head,
                               int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                               float eps, float k_scale, float v_scale, ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype,
                               uint32_t flags, hipStream_t stream) {
    const char *E = "ssm_qk_norm_rope_cache_fwd";
    REQUIRE_POS(E, n_kv_heads);
    int rc = check_rope(E, q, k, wq, wk, inv_freq, positions, n_tokens, n_heads, n_kv_heads, headdim, rot_dim, eps,
                        dtype, flags);
    if (rc != SSM_OK) return rc;
    if (!(dtype == SSM_F32 ? kv_dtype == SSM_KV_F32 : kv_dtype == SSM_KV_BF16 || kv_dtype == SSM_KV_F8E4M3))
        return fail(SSM_ERR_UNSUPPORTED, "%s: kv_dtype %d does not go with dtype %d", E, (int)kv_dtype, (int)dtype);
    const bool f8 = kv_dtype == SSM_KV_F8E4M3;
    if (f8 && !(k_scale > 0.0f && k_scale < INFINITY && v_scale > 0.0f && v_scale < INFINITY))
        return fail(SSM_ERR_INVALID_ARG, "%s: k_scale and v_scale must be > 0 and finite", E);
    const int es = dtype == SSM_BF16 ? 2 : 4, ce = f8 ? 1 : es;
    if ((rc = check_cache(E, n_pages, page_size, n_kv_heads, headdim, cache_stride_page, cache_stride_token,
                          cache_stride_head, ce)) != SSM_OK) return rc;
    if (n_tokens == 0) return SSM_OK;
    REQUIRE_PTR(E, v); REQUIRE_PTR(E, slots); REQUIRE_PTR(E, q_out); REQUIRE_PTR(E, k_cache); REQUIRE_PTR(E, v_cache);
    const Named ts[] = {{q, "q"}, {k, "k"}, {v, "v"}, {q_out, "q_out"}};
    for (const Named &t : ts)
        if ((rc = check_element(E, t.p, t.name, es)) != SSM_OK) return rc;
    if ((rc = check_element(E, k_cache, "k_cache", ce)) != SSM_OK) return rc;
    if ((rc = check_element(E, v_cache, "v_cache", ce)) != SSM_OK) return rc;
    if (q_out == q && !gapless(n_tokens, n_heads, headdim, q_stride_token, q_stride_head))
        return fail(SSM_ERR_INVALID_ARG, "%s: q_out aliases a q that is not contiguous", E);
    const Named outs[] = {{q_out, "q_out"}, {k_cache, "k_cache"}, {v_cache, "v_cache"}};
    const bool norm = (flags & SSM_QK_NO_NORM) == 0;
    const Named ins[] = {{k, "k"}, {v, "v"}, {norm ? wq : nullptr, "wq"}, {norm ? wk : nullptr, "wk"},
                         {rot_dim > 0 ? inv_freq : nullptr, "inv_freq"}, {rot_dim > 0 ? positions : nullptr, "positions"},
                         {slots, "slots"}};
    if ((rc = check_alias(E, outs, 3, ins, 7)) != SSM_OK) return rc;
    if (k_cache == q || v_cache == q) return fail(SSM_ERR_INVALID_ARG, "%s: a cache aliases q", E);
    ssm::QkRopeArgs a{};
    a.q = q; a.k = k; a.v = v; a.wq = wq; a.wk = wk; a.inv_freq = inv_freq; a.positions = positions; a.slots = slots;
    a.q_out = q_out; a.k_out = k_cache; a.v_cache = v_cache;
    a.n_tokens = n_tokens; a.n_heads = n_heads; a.n_kv_heads = n_kv_heads;
    a.headdim = (int)headdim; a.rot_dim = (int)rot_dim;
    a.q_st = n_tokens > 1 ? q_stride_token : 0; a.q_sh = n_heads > 1 ? q_stride_head : 0;
    a.k_st = n_tokens > 1 ? k_stride_token : 0; a.k_sh = n_kv_heads > 1 ? k_stride_head : 0;
    a.v_st = n_tokens > 1 ? v_stride_token : 0; a.v_sh = n_kv_heads > 1 ? v_stride_head : 0;
    a.n_pages = n_pages; a.page_size = page_size;
    a.c_sp = n_pages > 1 ? cache_stride_page : 0; a.c_st = page_size > 1 ? cache_stride_token : 0;
    a.c_sh = n_kv_heads > 1 ? cache_stride_head : 0;
    a.eps = eps; a.k_scale = k_scale; a.v_scale = v_scale;
    a.bf16 = dtype == SSM_BF16; a.kv_dtype = (int)kv_dtype; a.flags = flags;
    const char *kn = "qk_rope_kernel";
    return launched(E, ssm::launch_qk_rope(a, stream, &kn), kn);
}

size_t ssm_paged_attn_decode_fwd_workspace_size(int64_t batch, int64_t n_heads, int64_t n_kv_heads,
                                                int64_t headdim, int64_t max_pages, int64_t page_size) {
    if (batch <= 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 || headdim <= 0 ||
        max_pages <= 0 || page_size <= 0)
        return 0;
    return ssm::paged_attn_workspace_bytes(batch, n_heads, n_kv_heads, headdim, max_pages, page_size);
}

int ssm_paged_attn_decode_fwd(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *block_table, const int32_t *lens, void *o, float *lse,
                              int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                              int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                              int64_t q_stride_row, int64_t q_stride_head,
                              int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                              float scale, int64_t window, float k_scale, float v_scale,
                              ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype,
                              void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const char *E = "ssm_paged_attn_decode_fwd";
    REQUIRE_NOT_NEG(E, batch); REQUIRE_POS(E, n_heads); REQUIRE_POS(E, n_kv_heads); REQUIRE_POS(E, headdim);
    REQUIRE_POS(E, max_pages); REQUIRE_NOT_NEG(E, window);
    if (n_heads % n_kv_heads != 0)
        return fail(SSM_ERR_INVALID_ARG, "%s: n_heads %lld is not a multiple of n_kv_heads %lld", E, (long long)n_heads,
                    (long long)n_kv_heads);
    if (dtype != SSM_F32 && dtype != SSM_BF16)
        return fail(SSM_ERR_INVALID_ARG, "%s: dtype %d is not SSM_F32 or SSM_BF16", E, (int)dtype);
    if (!(dtype == SSM_F32 ? kv_dtype == SSM_KV_F32 : kv_dtype == SSM_KV_BF16 || kv_dtype == SSM_KV_F8E4M3))
        return fail(SSM_ERR_UNSUPPORTED, "%s: kv_dtype %d does not go with dtype %d", E, (int)kv_dtype, (int)dtype);
    const bool f8 = kv_dtype == SSM_KV_F8E4M3;
    if (f8 && !(k_scale > 0.0f && k_scale < INFINITY && v_scale > 0.0f && v_scale < INFINITY))
        return fail(SSM_ERR_INVALID_ARG, "%s: k_scale and v_scale must be > 0 and finite", E);
    if (!(scale > -INFINITY && scale < INFINITY))
        return fail(SSM_ERR_INVALID_ARG, "%s: scale must be finite", E);
    if (headdim > SSM_ATTN_MAX_HEADDIM)
        return fail(SSM_ERR_UNSUPPORTED, "%s: headdim %lld > %d", E, (long long)headdim, SSM_ATTN_MAX_HEADDIM);
    if (headdim % (f8 ? 16 : 8) != 0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: headdim %lld is not a multiple of %d", E, (long long)headdim, f8 ? 16 : 8);
    if (table_stride < max_pages)
        return fail(SSM_ERR_INVALID_ARG, "%s: table_stride %lld < max_pages %lld", E, (long long)table_stride,
                    (long long)max_pages);
    const int qe = dtype == SSM_BF16 ? 2 : 4, ce = f8 ? 1 : qe;
    int rc = check_cache(E, n_pages, page_size, n_kv_heads, headdim, cache_stride_page, cache_stride_token,
                         cache_stride_head, ce);
    if (rc != SSM_OK) return rc;
    if (batch > 65536 * 16 || n_heads > 65535 || table_stride >= (int64_t(1) << 40) ||
        (double)max_pages * (double)page_size > 1073741824.0 ||
        ssm::paged_attn_max_units(batch, n_heads, n_kv_heads, max_pages, page_size) >= 2147483648.0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: problem too large", E);
    if (batch == 0) return SSM_OK;
    REQUIRE_PTR(E, q); REQUIRE_PTR(E, k_cache); REQUIRE_PTR(E, v_cache); REQUIRE_PTR(E, block_table);
    REQUIRE_PTR(E, lens); REQUIRE_PTR(E, o);
    REQUIRE_ALIGN(E, q); REQUIRE_ALIGN(E, k_cache); REQUIRE_ALIGN(E, v_cache); REQUIRE_ALIGN(E, o);
    REQUIRE_ALIGN(E, workspace);
    // strides of a dim of one entry are not used
    const int64_t q_sr = batch > 1 ? q_stride_row : 0, q_sh = n_heads > 1 ? q_stride_head : 0;
    const int64_t sp = n_pages > 1 ? cache_stride_page : 0, st = page_size > 1 ? cache_stride_token : 0,
                  sh = n_kv_heads > 1 ? cache_stride_head : 0;
    if ((q_sr * qe) % 16 != 0 || (q_sh * qe) % 16 != 0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: a stride of q is not a multiple of 16 bytes", E);
    if ((sp * ce) % 16 != 0 || (st * ce) % 16 != 0 || (sh * ce) % 16 != 0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: a stride of the caches is not a multiple of 16 bytes", E);
    const Named outs[] = {{o, "o"}, {lse, "lse"}, {workspace, "workspace"}};
    const Named ins[] = {{q, "q"}, {k_cache, "k_cache"}, {v_cache, "v_cache"}, {block_table, "block_table"}, {lens, "lens"}};
    if ((rc = check_alias(E, outs, 3, ins, 5)) != SSM_OK) return rc;
    const size_t need = ssm_paged_attn_decode_fwd_workspace_size(batch, n_heads, n_kv_heads, headdim, max_pages, page_size);
    if (workspace == nullptr || workspace_bytes < need)
        return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", E, need,
                    workspace ? workspace_bytes : (size_t)0);
    ssm::PagedAttnArgs a{q, k_cache, v_cache, block_table, lens, o, lse, batch, n_heads, n_kv_heads, (int)headdim,
                         max_pages, table_stride, n_pages, page_size, q_sr, q_sh, sp, st, sh,
                         scale, k_scale, v_scale, window, (int)kv_dtype, workspace};
    const char *kn = "paged_attn_kernel";
    return launched(E, ssm::launch_paged_attn(a, stream, &kn), kn);
}

}  // extern "C"
