// attn_launchers.hpp -- host-side kernel launchers behind include/ssm_attn.h.
// Arguments have been validated by abi_attn.hip before any of these is called.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ssm_attn.h"

namespace ssm {

// one scheduling step of a paged cache (kv_pages.hip)
struct KvPagesArgs {
    const int32_t *len_old; const int32_t *len_new; int32_t *block_table; int32_t *free_ring;
    const int32_t *ring; int32_t *ring_out; int32_t *len_out; int32_t *starts;
    int32_t *request; int32_t *positions; int64_t *slots; int32_t *denied;
    int32_t batch, max_pages; int64_t table_stride; int32_t n_pages, page_size, n_tokens;
};
hipError_t launch_kv_pages(const KvPagesArgs &a, hipStream_t stream, const char **kernel_name);

// norm and rotation of q and k heads, and its form that writes a cache (qk_rope.hip).
// Strides in elements; the cache's are those of page, token and head.
struct QkRopeArgs {
    const void *q; const void *k; const void *v;
    const float *wq; const float *wk; const float *inv_freq; const int32_t *positions; const int64_t *slots;
    void *q_out; void *k_out;          // k_out: contiguous k, or the k cache when slots is set
    void *v_cache;
    int64_t n_tokens, n_heads, n_kv_heads; int headdim, rot_dim;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;
    int64_t n_pages, page_size, c_sp, c_st, c_sh;
    float eps, k_scale, v_scale; bool bf16; int kv_dtype; uint32_t flags;
};
hipError_t launch_qk_rope(const QkRopeArgs &a, hipStream_t stream, const char **kernel_name);

struct QkRopeBwdArgs {
    const void *q; const void *k; const float *wq; const float *wk; const float *inv_freq;
    const int32_t *positions; const void *dq_out; const void *dk_out; void *dq; void *dk; float *dwq; float *dwk;
    int64_t n_tokens, n_heads, n_kv_heads; int headdim, rot_dim;
    int64_t q_st, q_sh, k_st, k_sh, dq_st, dq_sh, dk_st, dk_sh;
    float eps; bool bf16; uint32_t flags; void *workspace;
};
size_t qk_rope_bwd_workspace_bytes(int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                   uint32_t flags);
hipError_t launch_qk_rope_bwd(const QkRopeBwdArgs &a, hipStream_t stream, const char **kernel_name);

// attention of one new token over a paged cache (paged_attn.hip); cache strides in elements
struct PagedAttnArgs {
    const void *q; const void *k_cache; const void *v_cache; const int32_t *block_table; const int32_t *lens;
    void *o; float *lse;
    int64_t batch, n_heads, n_kv_heads; int headdim;
    int64_t max_pages, table_stride, n_pages, page_size, q_sr, q_sh, c_sp, c_st, c_sh;
    float scale, k_scale, v_scale; int64_t window; int kv_dtype; void *workspace;
};
size_t paged_attn_workspace_bytes(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                  int64_t max_pages, int64_t page_size);
// units of work of the longest rows: must stay below 2^31
double paged_attn_max_units(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t max_pages, int64_t page_size);
hipError_t launch_paged_attn(const PagedAttnArgs &a, hipStream_t stream, const char **kernel_name);

}  // namespace ssm
