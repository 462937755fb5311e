// abi_attn_common.hpp -- argument checks that the entry points of include/ssm_attn.h and
// include/ssm_longctx.h share.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ssm_attn.h"
#include "abi_common.hpp"

#define REQUIRE_NOT_NEG(entry, v)                                                                 \
    do {                                                                                          \
        if ((v) < 0) return ssm::fail(SSM_ERR_INVALID_ARG, "%s: %s must be >= 0 (got %lld)", entry, #v, \
                                 (long long)(v));                                                 \
    } while (0)

namespace ssm {

constexpr int64_t k2p31 = int64_t(1) << 31;

// two tensors of one call that may not share their first element
struct Named { const void *p; const char *name; };
inline int check_alias(const char *E, const Named *outs, int no, const Named *ins, int ni) {
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
inline int check_element(const char *E, const void *p, const char *name, int esize) {
    if (((uintptr_t)p & (uintptr_t)(esize - 1)) != 0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: %s is not aligned to its elements", E, name);
    return SSM_OK;
}

// cache strides: rows must not overlap by sign, and every offset must fit the kernels' arithmetic
inline int check_cache(const char *E, int64_t n_pages, int64_t page_size, int64_t n_kv_heads, int64_t headdim,
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

// what the kernels that walk a paged cache ask of it: types that go together, headdim, a table, strides
// that are multiples of 16 bytes.  Strides of a dim of one entry are not used and come back as 0.
inline int check_paged(const char *E, int64_t batch, int64_t headdim, int64_t max_pages, int64_t table_stride, int64_t n_pages,
                       int64_t page_size, int64_t n_kv_heads, int64_t &sp, int64_t &st, int64_t &sh, ssm_kv_dtype_t kv_dtype) {
    REQUIRE_NOT_NEG(E, batch); REQUIRE_POS(E, n_kv_heads); REQUIRE_POS(E, headdim); REQUIRE_POS(E, max_pages);
    if (kv_dtype != SSM_KV_F32 && kv_dtype != SSM_KV_BF16 && kv_dtype != SSM_KV_F8E4M3)
        return fail(SSM_ERR_INVALID_ARG, "%s: kv_dtype %d is not SSM_KV_F32, SSM_KV_BF16 or SSM_KV_F8E4M3", E, (int)kv_dtype);
    const int ce = kv_dtype == SSM_KV_F32 ? 4 : kv_dtype == SSM_KV_BF16 ? 2 : 1, mult = ce == 1 ? 16 : 8;
    if (headdim > SSM_ATTN_MAX_HEADDIM)
        return fail(SSM_ERR_UNSUPPORTED, "%s: headdim %lld > %d", E, (long long)headdim, SSM_ATTN_MAX_HEADDIM);
    if (headdim % mult != 0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: headdim %lld is not a multiple of %d", E, (long long)headdim, mult);
    if (table_stride < max_pages)
        return fail(SSM_ERR_INVALID_ARG, "%s: table_stride %lld < max_pages %lld", E, (long long)table_stride,
                    (long long)max_pages);
    const int rc = check_cache(E, n_pages, page_size, n_kv_heads, headdim, sp, st, sh, ce);
    if (rc != SSM_OK) return rc;
    if (batch > (1 << 20) || n_kv_heads > 65535 || table_stride >= (int64_t(1) << 40) ||
        (double)batch * (double)n_kv_heads > 1048576.0 || (double)max_pages * (double)page_size > 1073741824.0 ||
        (double)batch * (double)n_kv_heads * (double)max_pages >= 2147483648.0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: problem too large", E);
    sp = n_pages > 1 ? sp : 0; st = page_size > 1 ? st : 0; sh = n_kv_heads > 1 ? sh : 0;
    if ((sp * ce) % 16 != 0 || (st * ce) % 16 != 0 || (sh * ce) % 16 != 0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: a stride of the caches is not a multiple of 16 bytes", E);
    return SSM_OK;
}

// q beside such a cache
inline int check_heads(const char *E, int64_t rows, int64_t n_heads, int64_t n_kv_heads, int64_t &q_sr, int64_t &q_sh,
                       ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype) {
    REQUIRE_NOT_NEG(E, rows); REQUIRE_POS(E, n_heads); REQUIRE_POS(E, n_kv_heads);
    if (n_heads % n_kv_heads != 0)
        return fail(SSM_ERR_INVALID_ARG, "%s: n_heads %lld is not a multiple of n_kv_heads %lld", E, (long long)n_heads,
                    (long long)n_kv_heads);
    if (dtype != SSM_F32 && dtype != SSM_BF16)
        return fail(SSM_ERR_INVALID_ARG, "%s: dtype %d is not SSM_F32 or SSM_BF16", E, (int)dtype);
    if (!(dtype == SSM_F32 ? kv_dtype == SSM_KV_F32 : kv_dtype == SSM_KV_BF16 || kv_dtype == SSM_KV_F8E4M3))
        return fail(SSM_ERR_UNSUPPORTED, "%s: kv_dtype %d does not go with dtype %d", E, (int)kv_dtype, (int)dtype);
    if (rows >= k2p31 || n_heads > 65535 || (double)rows * (double)n_heads >= 1073741824.0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: problem too large", E);
    const int qe = dtype == SSM_BF16 ? 2 : 4;
    q_sr = rows > 1 ? q_sr : 0; q_sh = n_heads > 1 && rows > 0 ? q_sh : 0;
    if ((q_sr * qe) % 16 != 0 || (q_sh * qe) % 16 != 0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: a stride of q is not a multiple of 16 bytes", E);
    return SSM_OK;
}

inline int check_scales(const char *E, float scale, float k_scale, float v_scale, ssm_kv_dtype_t kv_dtype) {
    if (kv_dtype == SSM_KV_F8E4M3 && !(k_scale > 0.0f && k_scale < INFINITY && v_scale > 0.0f && v_scale < INFINITY))
        return fail(SSM_ERR_INVALID_ARG, "%s: k_scale and v_scale must be > 0 and finite", E);
    if (!(scale > -INFINITY && scale < INFINITY))
        return fail(SSM_ERR_INVALID_ARG, "%s: scale must be finite", E);
    return SSM_OK;
}

}  // namespace ssm
