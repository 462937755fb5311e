// abi_longctx.hip -- the extern "C" boundary of include/ssm_longctx.h: argument
// validation, workspace sizing, and dispatch to the kernel launchers.  Every
// check runs before any HIP call.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ssm_longctx.h"
#include "abi_attn_common.hpp"
#include "attn_launchers.hpp"

using namespace ssm;

namespace {

int check_workspace(const char *E, const void *workspace, size_t bytes, size_t need) {
    REQUIRE_ALIGN(E, workspace);
    if (need > 0 && (workspace == nullptr || bytes < need))
        return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", E, need, workspace ? bytes : (size_t)0);
    return SSM_OK;
}

// the work of the attention kernels is counted in 32 bits
int check_units(const char *E, int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t max_pages, int64_t page_size) {
    if (paged_attn_max_units(batch, n_heads, n_kv_heads, max_pages, page_size) >= 2147483648.0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: problem too large", E);
    return SSM_OK;
}

bool sizes_ok(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim, int64_t max_pages, int64_t page_size) {
    return batch > 0 && n_heads > 0 && n_kv_heads > 0 && n_heads % n_kv_heads == 0 && headdim > 0 && max_pages > 0 && page_size > 0;
}

#define TRY(call)                          \
    do {                                   \
        const int rc_ = (call);            \
        if (rc_ != SSM_OK) return rc_;     \
    } while (0)

int elem(ssm_kv_dtype_t kv) { return kv == SSM_KV_F32 ? 4 : kv == SSM_KV_BF16 ? 2 : 1; }

}  // namespace

extern "C" {

size_t ssm_prefix_attn_decode_fwd_workspace_size(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                                 int64_t max_prefix_pages, int64_t max_pages, int64_t page_size) {
    if (!sizes_ok(batch, n_heads, n_kv_heads, headdim, max_pages, page_size) || max_prefix_pages <= 0) return 0;
    return prefix_attn_workspace_bytes(batch, n_heads, n_kv_heads, headdim, max_prefix_pages, max_pages, page_size);
}

int ssm_prefix_attn_decode_fwd(const void *q, const void *k_cache, const void *v_cache,
                               const int32_t *prefix, const int32_t *prefix_table, const int32_t *prefix_lens,
                               const int32_t *block_table, const int32_t *lens, void *o, float *lse,
                               int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                               int64_t n_prefixes, int64_t max_prefix_pages, int64_t prefix_stride,
                               int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                               int64_t q_stride_row, int64_t q_stride_head,
                               int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                               float scale, float k_scale, float v_scale, ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype,
                               void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const char *E = "ssm_prefix_attn_decode_fwd";
    int64_t sp = cache_stride_page, st = cache_stride_token, sh = cache_stride_head, q_sr = q_stride_row, q_sh = q_stride_head;
    TRY(check_heads(E, batch, n_heads, n_kv_heads, q_sr, q_sh, dtype, kv_dtype));
    TRY(check_scales(E, scale, k_scale, v_scale, kv_dtype));
    TRY(check_paged(E, batch, headdim, max_pages, table_stride, n_pages, page_size, n_kv_heads, sp, st, sh, kv_dtype));
    REQUIRE_POS(E, n_prefixes); REQUIRE_POS(E, max_prefix_pages);
    if (prefix_stride < max_prefix_pages)
        return fail(SSM_ERR_INVALID_ARG, "%s: prefix_stride %lld < max_prefix_pages %lld", E, (long long)prefix_stride,
                    (long long)max_prefix_pages);
    TRY(check_units(E, batch, n_heads, n_kv_heads, max_pages, page_size));
    if (n_prefixes >= k2p31 || prefix_stride >= (int64_t(1) << 40) || batch * n_heads >= (1 << 24) ||
        (double)max_prefix_pages * (double)page_size > 1073741824.0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: problem too large", E);
    // (the prefixes of a block's rows, 64 at most, stand in one line of tiles of 16 tokens or more, counted in 32 bits)
    if ((n_prefixes < 64 ? n_prefixes : 64) * ((max_prefix_pages * page_size + 15) / 16) >= k2p31)
        return fail(SSM_ERR_UNSUPPORTED, "%s: prefixes of up to %lld tokens are too long together", E,
                    (long long)(max_prefix_pages * page_size));
    if (batch == 0) return SSM_OK;
    REQUIRE_PTR(E, q); REQUIRE_PTR(E, k_cache); REQUIRE_PTR(E, v_cache); REQUIRE_PTR(E, prefix); REQUIRE_PTR(E, prefix_table);
    REQUIRE_PTR(E, prefix_lens); REQUIRE_PTR(E, block_table); REQUIRE_PTR(E, lens); REQUIRE_PTR(E, o);
    REQUIRE_ALIGN(E, q); REQUIRE_ALIGN(E, k_cache); REQUIRE_ALIGN(E, v_cache); REQUIRE_ALIGN(E, o);
    const Named outs[] = {{o, "o"}, {lse, "lse"}, {workspace, "workspace"}};
    const Named ins[] = {{q, "q"}, {k_cache, "k_cache"}, {v_cache, "v_cache"}, {prefix, "prefix"}, {prefix_table, "prefix_table"},
                         {prefix_lens, "prefix_lens"}, {block_table, "block_table"}, {lens, "lens"}};
    TRY(check_alias(E, outs, 3, ins, 8));
    TRY(check_workspace(E, workspace, workspace_bytes,
                        prefix_attn_workspace_bytes(batch, n_heads, n_kv_heads, headdim, max_prefix_pages, max_pages, page_size)));
    PrefixAttnArgs a{};
    a.own = {q, k_cache, v_cache, block_table, lens, o, lse, batch, n_heads, n_kv_heads, (int)headdim,
             max_pages, table_stride, n_pages, page_size, q_sr, q_sh, sp, st, sh,
             scale, k_scale, v_scale, 0, (int)kv_dtype, workspace, nullptr, 0, false};
    a.prefix = prefix; a.prefix_table = prefix_table; a.prefix_lens = prefix_lens;
    a.n_prefixes = n_prefixes; a.max_prefix_pages = max_prefix_pages; a.prefix_stride = prefix_stride;
    const char *kn = "prefix_attn_kernel";
    return launched(E, launch_prefix_attn(a, stream, &kn), kn);
}

int ssm_kv_page_bounds_update(const void *k_cache, void *bounds, const int32_t *block_table,
                              const int32_t *len_old, const int32_t *lens,
                              int64_t batch, int64_t n_kv_heads, int64_t headdim,
                              int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                              int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                              ssm_kv_dtype_t kv_dtype, hipStream_t stream) {
    const char *E = "ssm_kv_page_bounds_update";
    int64_t sp = cache_stride_page, st = cache_stride_token, sh = cache_stride_head;
    TRY(check_paged(E, batch, headdim, max_pages, table_stride, n_pages, page_size, n_kv_heads, sp, st, sh, kv_dtype));
    if (batch > SSM_KV_MAX_BATCH)
        return fail(SSM_ERR_UNSUPPORTED, "%s: batch %lld > %d", E, (long long)batch, SSM_KV_MAX_BATCH);
    if (batch == 0) return SSM_OK;
    REQUIRE_PTR(E, k_cache); REQUIRE_PTR(E, bounds); REQUIRE_PTR(E, block_table); REQUIRE_PTR(E, len_old); REQUIRE_PTR(E, lens);
    REQUIRE_ALIGN(E, k_cache); REQUIRE_ALIGN(E, bounds);
    const Named outs[] = {{bounds, "bounds"}};
    const Named ins[] = {{k_cache, "k_cache"}, {block_table, "block_table"}, {len_old, "len_old"}, {lens, "lens"}};
    TRY(check_alias(E, outs, 1, ins, 4));
    const int ce = elem(kv_dtype);
    KvBoundsArgs a{(const char *)k_cache, (char *)bounds, block_table, len_old, lens, table_stride, sp * ce, st * ce, sh * ce,
                   (int)batch, (int)n_kv_heads, (int)headdim * ce, (int)max_pages, (int)n_pages, (int)page_size, (int)kv_dtype};
    const char *kn = "kv_bounds_kernel";
    return launched(E, launch_kv_bounds(a, stream, &kn), kn);
}

size_t ssm_kv_page_select_fwd_workspace_size(int64_t batch, int64_t n_kv_heads, int64_t max_pages, int64_t top_k) {
    if (batch <= 0 || n_kv_heads <= 0 || max_pages <= 0 || top_k <= 0) return 0;
    return page_select_workspace_bytes(batch, n_kv_heads, max_pages, top_k);
}

int ssm_kv_page_select_fwd(const void *q, const void *bounds, const int32_t *block_table, const int32_t *lens,
                           int32_t *selected, int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                           int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                           int64_t top_k, int64_t first, int64_t last, int64_t q_stride_row, int64_t q_stride_head,
                           ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype,
                           void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const char *E = "ssm_kv_page_select_fwd";
    int64_t sp = 0, st = 0, sh = 0, q_sr = q_stride_row, q_sh = q_stride_head;
    TRY(check_heads(E, batch, n_heads, n_kv_heads, q_sr, q_sh, dtype, kv_dtype));
    TRY(check_paged(E, batch, headdim, max_pages, table_stride, n_pages, page_size, n_kv_heads, sp, st, sh, kv_dtype));
    REQUIRE_POS(E, top_k); REQUIRE_NOT_NEG(E, first); REQUIRE_NOT_NEG(E, last);
    if (first > top_k || last > top_k || first + last > top_k)
        return fail(SSM_ERR_INVALID_ARG, "%s: first %lld + last %lld > top_k %lld", E, (long long)first, (long long)last,
                    (long long)top_k);
    if (top_k > (1 << 20) || (double)batch * (double)n_kv_heads * (double)top_k >= 2147483648.0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: top_k %lld is too large", E, (long long)top_k);
    if (batch == 0) return SSM_OK;
    REQUIRE_PTR(E, q); REQUIRE_PTR(E, bounds); REQUIRE_PTR(E, block_table); REQUIRE_PTR(E, lens); REQUIRE_PTR(E, selected);
    REQUIRE_ALIGN(E, q); REQUIRE_ALIGN(E, bounds);
    const size_t need = page_select_workspace_bytes(batch, n_kv_heads, max_pages, top_k);
    const Named outs[] = {{selected, "selected"}, {need > 0 ? workspace : nullptr, "workspace"}};
    const Named ins[] = {{q, "q"}, {bounds, "bounds"}, {block_table, "block_table"}, {lens, "lens"}};
    TRY(check_alias(E, outs, 2, ins, 4));
    TRY(check_workspace(E, workspace, workspace_bytes, need));
    PageSelectArgs a{q, (const char *)bounds, block_table, lens, selected, (uint32_t *)workspace, table_stride, q_sr, q_sh,
                     (int)batch, (int)n_heads, (int)n_kv_heads, (int)headdim, (int)max_pages, (int)n_pages, (int)page_size,
                     (int)top_k, (int)first, (int)last, (int)kv_dtype, dtype == SSM_BF16};
    const char *kn = "page_select_kernel";
    return launched(E, launch_page_select(a, stream, &kn), kn);
}

size_t ssm_select_attn_decode_fwd_workspace_size(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                                 int64_t max_pages, int64_t page_size, int64_t top_k) {
    if (!sizes_ok(batch, n_heads, n_kv_heads, headdim, max_pages, page_size) || top_k <= 0) return 0;
    return paged_attn_workspace_bytes(batch, n_heads, n_kv_heads, headdim, top_k < max_pages ? top_k : max_pages, page_size);
}

int ssm_select_attn_decode_fwd(const void *q, const void *k_cache, const void *v_cache,
                               const int32_t *block_table, const int32_t *lens, const int32_t *selected,
                               void *o, float *lse,
                               int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                               int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size, int64_t top_k,
                               int64_t q_stride_row, int64_t q_stride_head,
                               int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                               float scale, float k_scale, float v_scale, ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype,
                               void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const char *E = "ssm_select_attn_decode_fwd";
    int64_t sp = cache_stride_page, st = cache_stride_token, sh = cache_stride_head, q_sr = q_stride_row, q_sh = q_stride_head;
    TRY(check_heads(E, batch, n_heads, n_kv_heads, q_sr, q_sh, dtype, kv_dtype));
    TRY(check_scales(E, scale, k_scale, v_scale, kv_dtype));
    TRY(check_paged(E, batch, headdim, max_pages, table_stride, n_pages, page_size, n_kv_heads, sp, st, sh, kv_dtype));
    REQUIRE_POS(E, top_k);
    if (top_k > (1 << 20) || (double)batch * (double)n_kv_heads * (double)top_k >= 2147483648.0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: top_k %lld is too large", E, (long long)top_k);
    TRY(check_units(E, batch, n_heads, n_kv_heads, top_k < max_pages ? top_k : max_pages, page_size));
    if (batch == 0) return SSM_OK;
    REQUIRE_PTR(E, q); REQUIRE_PTR(E, k_cache); REQUIRE_PTR(E, v_cache); REQUIRE_PTR(E, block_table); REQUIRE_PTR(E, lens);
    REQUIRE_PTR(E, selected); REQUIRE_PTR(E, o);
    REQUIRE_ALIGN(E, q); REQUIRE_ALIGN(E, k_cache); REQUIRE_ALIGN(E, v_cache); REQUIRE_ALIGN(E, o);
    const Named outs[] = {{o, "o"}, {lse, "lse"}, {workspace, "workspace"}};
    const Named ins[] = {{q, "q"}, {k_cache, "k_cache"}, {v_cache, "v_cache"}, {block_table, "block_table"}, {lens, "lens"},
                         {selected, "selected"}};
    TRY(check_alias(E, outs, 3, ins, 6));
    TRY(check_workspace(E, workspace, workspace_bytes,
                        ssm_select_attn_decode_fwd_workspace_size(batch, n_heads, n_kv_heads, headdim, max_pages, page_size, top_k)));
    PagedAttnArgs a{q, k_cache, v_cache, block_table, lens, o, lse, batch, n_heads, n_kv_heads, (int)headdim,
                    max_pages, table_stride, n_pages, page_size, q_sr, q_sh, sp, st, sh,
                    scale, k_scale, v_scale, 0, (int)kv_dtype, workspace, selected, top_k, false};
    const char *kn = "paged_attn_kernel";
    return launched(E, launch_select_attn(a, stream, &kn), kn);
}

int ssm_kv_mass_update(const void *q, const void *k_cache, const float *lse, float *mass,
                       const int32_t *block_table, const int32_t *starts, const int32_t *positions,
                       const int32_t *len_old, const int32_t *lens,
                       int64_t n_tokens, int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                       int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                       int64_t q_stride_token, int64_t q_stride_head,
                       int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                       float scale, float k_scale, ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype, hipStream_t stream) {
    const char *E = "ssm_kv_mass_update";
    int64_t sp = cache_stride_page, st = cache_stride_token, sh = cache_stride_head, q_st = q_stride_token, q_sh = q_stride_head;
    TRY(check_heads(E, n_tokens, n_heads, n_kv_heads, q_st, q_sh, dtype, kv_dtype));
    TRY(check_scales(E, scale, k_scale, 1.0f, kv_dtype));
    TRY(check_paged(E, batch, headdim, max_pages, table_stride, n_pages, page_size, n_kv_heads, sp, st, sh, kv_dtype));
    if (batch > SSM_KV_MAX_BATCH)
        return fail(SSM_ERR_UNSUPPORTED, "%s: batch %lld > %d", E, (long long)batch, SSM_KV_MAX_BATCH);
    TRY(check_units(E, batch, n_heads, n_kv_heads, max_pages, page_size));
    if ((double)n_pages * (double)n_kv_heads * (double)page_size >= 2147483648.0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: problem too large", E);
    if (batch == 0) return SSM_OK;
    if (n_tokens > 0) { REQUIRE_PTR(E, q); REQUIRE_PTR(E, lse); REQUIRE_PTR(E, positions); }
    REQUIRE_PTR(E, k_cache); REQUIRE_PTR(E, mass); REQUIRE_PTR(E, block_table); REQUIRE_PTR(E, starts);
    REQUIRE_PTR(E, len_old); REQUIRE_PTR(E, lens);
    REQUIRE_ALIGN(E, q); REQUIRE_ALIGN(E, k_cache);
    TRY(check_element(E, mass, "mass", 4));
    const Named outs[] = {{mass, "mass"}};
    const Named ins[] = {{q, "q"}, {k_cache, "k_cache"}, {lse, "lse"}, {block_table, "block_table"}, {starts, "starts"},
                         {positions, "positions"}, {len_old, "len_old"}, {lens, "lens"}};
    TRY(check_alias(E, outs, 1, ins, 8));
    KvMassArgs a{q, k_cache, lse, mass, block_table, starts, positions, len_old, lens, n_tokens, batch, n_heads, n_kv_heads,
                 (int)headdim, max_pages, table_stride, n_pages, page_size, q_st, q_sh, sp, st, sh, scale, k_scale, (int)kv_dtype};
    const char *kn = "kv_mass_kernel";
    return launched(E, launch_kv_mass(a, stream, &kn), kn);
}

int ssm_kv_evict(void *k_cache, void *v_cache, float *mass, const int32_t *block_table, const int32_t *lens,
                 int32_t *len_out, int32_t *kept, int64_t batch, int64_t n_kv_heads, int64_t headdim,
                 int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                 int64_t budget, int64_t recent,
                 int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                 ssm_kv_dtype_t kv_dtype, hipStream_t stream) {
    const char *E = "ssm_kv_evict";
    int64_t sp = cache_stride_page, st = cache_stride_token, sh = cache_stride_head;
    TRY(check_paged(E, batch, headdim, max_pages, table_stride, n_pages, page_size, n_kv_heads, sp, st, sh, kv_dtype));
    REQUIRE_POS(E, budget); REQUIRE_NOT_NEG(E, recent);
    if (recent > budget)
        return fail(SSM_ERR_INVALID_ARG, "%s: recent %lld > budget %lld", E, (long long)recent, (long long)budget);
    if (budget > (int64_t(1) << 30) || (double)batch * (double)n_kv_heads * (double)budget >= 2147483648.0 ||
        (double)n_pages * (double)n_kv_heads * (double)page_size >= 2147483648.0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: problem too large", E);
    if (batch == 0) return SSM_OK;
    REQUIRE_PTR(E, k_cache); REQUIRE_PTR(E, v_cache); REQUIRE_PTR(E, mass); REQUIRE_PTR(E, block_table); REQUIRE_PTR(E, lens);
    REQUIRE_PTR(E, len_out); REQUIRE_PTR(E, kept);
    REQUIRE_ALIGN(E, k_cache); REQUIRE_ALIGN(E, v_cache);
    TRY(check_element(E, mass, "mass", 4));
    const Named outs[] = {{k_cache, "k_cache"}, {v_cache, "v_cache"}, {mass, "mass"}, {len_out, "len_out"}, {kept, "kept"}};
    const Named ins[] = {{block_table, "block_table"}, {lens, "lens"}};
    TRY(check_alias(E, outs, 5, ins, 2));
    const int ce = elem(kv_dtype);
    KvEvictArgs a{(char *)k_cache, (char *)v_cache, mass, block_table, lens, len_out, kept, table_stride, sp * ce, st * ce, sh * ce,
                  (int)batch, (int)n_kv_heads, (int)headdim * ce, (int)max_pages, (int)n_pages, (int)page_size,
                  (int)budget, (int)recent};
    const char *kn = "evict_pick_kernel";
    return launched(E, launch_kv_evict(a, stream, &kn), kn);
}

}  // extern "C"
