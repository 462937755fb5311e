/*
 * ssm_longctx.h -- C interface of libssmscan.so for long contexts in the paged
 * key-value cache of ssm_attn.h: attention of rows that share a long prefix,
 * attention over the pages that a cheap score selects, and eviction of the tokens
 * that gathered the least attention weight.
 *
 * The conventions are those of ssm_attn.h: caller-owned device buffers, strided
 * tensors with a last stride of 1, nothing allocated, nothing synchronised, work
 * enqueued on `stream`, every argument checked before any HIP call,
 * ssm_last_error() after a negative status, results that are bitwise reproducible
 * run to run (no floating-point atomics), a workspace that aliases nothing else.
 * Caches, their types and scales, block tables and lengths are those of
 * ssm_paged_attn_decode_fwd: token j of request r is row j % page_size of page
 * block_table[r, j / page_size]; a length is cut to max_pages * page_size, and a
 * negative one counts as 0; pages outside [0, n_pages) hold no token.
 * Limits of all of them: batch * n_kv_heads at most 2^20, batch * n_kv_heads *
 * max_pages below 2^31, max_pages * page_size at most 2^30, rows of queries times
 * n_heads below 2^30, n_heads at most 65535; the others stand at each.
 * All of these are operators of serving; none has a gradient.
 *
 * The definitions are the common ones of decoder models and are not taken from
 * the pages that ssm_scan.h cites.
 */
#ifndef SSM_LONGCTX_H
#define SSM_LONGCTX_H

#include "ssm_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --------------- attention of one new token a row, with shared prefixes ----
 * Row r attends to the tokens of prefix p = prefix[r] and then to its own:
 * tokens [0, prefix_lens[p]) through prefix_table[p, ..], and tokens
 * [0, lens[r]) through block_table[r, ..] (which counts from the prefix's end;
 * a cache for n tokens behind the prefix has lens = n).  A prefix[r] outside
 * [0, n_prefixes) is no prefix.  With s over both sets of tokens, o and lse are
 * as in ssm_paged_attn_decode_fwd, also for a row that has no token at all
 * (o = 0, lse = -inf).
 *
 * A prefix's keys and values are read once for 16 to 128 (row, query head)
 * pairs of a kv head whose rows stand next to each other: rows of one prefix cost
 * least side by side, and any order is right.
 * Arithmetic: as ssm_paged_attn_decode_fwd.
 *
 * Layouts: prefix (batch) int32; prefix_table (n_prefixes, max_prefix_pages)
 * int32, row stride prefix_stride; prefix_lens (n_prefixes) int32; the others as
 * in ssm_paged_attn_decode_fwd.  No output may alias an input.
 * Limits: those of ssm_paged_attn_decode_fwd; n_prefixes from 1 to 2^31 - 1,
 * max_prefix_pages * page_size at most 2^30, and min(n_prefixes, 64) times that / 16
 * (rounded up) below 2^31; batch * n_heads below 2^24.
 * Workspace: ssm_prefix_attn_decode_fwd_workspace_size() bytes, 16-byte aligned. */
size_t ssm_prefix_attn_decode_fwd_workspace_size(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                                 int64_t max_prefix_pages, int64_t max_pages, int64_t page_size);

int ssm_prefix_attn_decode_fwd(const void *q, const void *k_cache, const void *v_cache,
                               const int32_t *prefix, const int32_t *prefix_table, const int32_t *prefix_lens,
                               const int32_t *block_table, const int32_t *lens, void *o, float *lse,
                               int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                               int64_t n_prefixes, int64_t max_prefix_pages, int64_t prefix_stride,
                               int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                               int64_t q_stride_row, int64_t q_stride_head,
                               int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                               float scale, float k_scale, float v_scale, ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype,
                               void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------- smallest and largest keys of pages ----
 * For each request r with len_old[r] < lens[r], and each page that its tokens
 * [len_old[r], lens[r]) stand on: bounds[page, g, 0, :] and bounds[page, g, 1, :]
 * become the smallest and the largest value, dim by dim, of the page's keys of kv
 * head g: of the new tokens alone where the page's first token is one of them,
 * and of them and of what bounds held else.  Values are those that the cache
 * stores (before k_scale), so bounds have its type and are exact; of NaN keys a
 * page has NaN bounds.  Other pages' bounds are left as they are.  (len_old = 0
 * forms them anew, after an eviction for instance.)
 * Layouts: k_cache as above; bounds (n_pages, n_kv_heads, 2, headdim) [kv_dtype]
 * contiguous, updated in place; block_table, len_old, lens (batch) int32.  A page
 * that new tokens stand on belongs to one request, and stands once in its table.
 * Limits: batch <= SSM_KV_MAX_BATCH; headdim and the cache's strides as in
 * ssm_paged_attn_decode_fwd; bounds 16-byte aligned.  No workspace. */
int ssm_kv_page_bounds_update(const void *k_cache, void *bounds, const int32_t *block_table,
                              const int32_t *len_old, const int32_t *lens,
                              int64_t batch, int64_t n_kv_heads, int64_t headdim,
                              int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                              int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                              ssm_kv_dtype_t kv_dtype, hipStream_t stream);

/* ------------------------------------------------ choice of a row's pages ----
 * For each row r, of n = ceil(lens[r] / page_size) pages, and kv head g:
 *   score(i) = max over the query heads h of g of
 *              sum_d max(q[r,h,d], 0) hi_d + min(q[r,h,d], 0) lo_d,
 * lo and hi the bounds of page block_table[r, i]: no key between the bounds has a
 * larger product with q.  selected[r, g, :] lists the chosen pages i in rising
 * order, then -1:
 *   - all n pages if n <= top_k;
 *   - else the first `first` and the last `last` pages, and of the others the
 *     top_k - first - last with the largest scores, the lower i of equal ones.
 * Arithmetic: products and sums in 64 bits, a sum rounded once to 32 (the order of
 * scores that lie close together depends on nothing else).  A NaN is larger than
 * any number; a page outside [0, n_pages) has score -inf.
 * Layouts: q (batch, n_heads, headdim) [dtype] strided; bounds as above
 * [kv_dtype]; block_table; lens; selected (batch, n_kv_heads, top_k) int32.
 * Limits: n_heads % n_kv_heads == 0; first, last >= 0, first + last <= top_k, 1 <=
 * top_k <= 2^20; batch * n_kv_heads * top_k below 2^31; headdim a multiple of 8 (16
 * for 8 bits), <= SSM_ATTN_MAX_HEADDIM; q and bounds 16-byte aligned, strides of q
 * multiples of 16 bytes.
 * Workspace: ssm_kv_page_select_fwd_workspace_size() bytes, 16-byte aligned (the
 * scores). */
size_t ssm_kv_page_select_fwd_workspace_size(int64_t batch, int64_t n_kv_heads, int64_t max_pages, int64_t top_k);

int ssm_kv_page_select_fwd(const void *q, const void *bounds, const int32_t *block_table, const int32_t *lens,
                           int32_t *selected, int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                           int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                           int64_t top_k, int64_t first, int64_t last, int64_t q_stride_row, int64_t q_stride_head,
                           ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype,
                           void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------- attention of one new token over a row's chosen pages ----
 * ssm_paged_attn_decode_fwd over the tokens j < lens[r] whose page j / page_size
 * is listed in selected[r, g, 0 .. m), m = min(top_k, ceil(lens[r] / page_size)),
 * for the query heads of kv head g.  Entries below 0, or of pages that the row
 * does not have, are no page; a page listed twice counts twice.
 * Arithmetic, layouts and limits are those of ssm_paged_attn_decode_fwd (with
 * min(top_k, max_pages) in place of max_pages where it counts work); selected
 * (batch, n_kv_heads, top_k) int32 contiguous.
 * Workspace: ssm_select_attn_decode_fwd_workspace_size() bytes, 16-byte aligned. */
size_t ssm_select_attn_decode_fwd_workspace_size(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                                 int64_t max_pages, int64_t page_size, int64_t top_k);

int ssm_select_attn_decode_fwd(const void *q, const void *k_cache, const void *v_cache,
                               const int32_t *block_table, const int32_t *lens, const int32_t *selected,
                               void *o, float *lse,
                               int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                               int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size, int64_t top_k,
                               int64_t q_stride_row, int64_t q_stride_head,
                               int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                               float scale, float k_scale, float v_scale, ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype,
                               void *workspace, size_t workspace_bytes, hipStream_t stream);

/* --------------------------- attention weight that cached tokens gathered ----
 * Adds the softmax weights of a step's queries to a running sum for each cached
 * token and kv head.  Request r has the query rows t in [starts[r], starts[r+1])
 * of n_tokens (what ssm_kv_pages_step numbers), row t at place positions[t] of
 * its cache; rows whose place is outside [0, lens[r]) (a refused request's) add
 * nothing.  For each token j < lens[r] and kv head g:
 *   w = sum over rows t with j <= positions[t] and query heads h of g of
 *       exp(scale * k_scale * q[t,h] . k[j,g] - lse[t,h])
 *   mass[page, g, j % page_size] = w + (j < len_old[r] ? mass[page, g, j % page_size] : 0)
 * with lse what attention of the same rows over all the tokens that they see gave
 * (a row with lse = -inf adds nothing): ssm_paged_attn_decode_fwd without a window,
 * where each of a prompt's rows is a row of its own, with its request's line of the
 * table and the length positions[t] + 1; or ssm_prefix_attn_decode_fwd, whose rows' own
 * tokens then gather their shares of the whole.  Not that of attention over chosen
 * pages or a window: tokens that it left out would gather weights of any size.  Tokens from len_old[r] on are new: what their place held is dropped.
 * A request without a row that counts keeps its mass for the tokens below len_old.
 * Arithmetic: products as in ssm_paged_attn_decode_fwd, exponentials and sums in
 * fp32, in an order fixed by the shapes.
 * Layouts: q (n_tokens, n_heads, headdim) [dtype] strided; lse (n_tokens, n_heads)
 * fp32; mass (n_pages, n_kv_heads, page_size) fp32 contiguous, updated in place;
 * starts (batch + 1), positions (n_tokens), len_old, lens (batch) int32.  starts
 * outside [0, n_tokens] are cut to it.  A page belongs to one request here, and
 * stands once in its table.
 * Limits: batch <= SSM_KV_MAX_BATCH; those of ssm_paged_attn_decode_fwd, and n_pages *
 * n_kv_heads * page_size below 2^31.  n_tokens may be 0 (q, lse and positions may then be NULL).  No
 * workspace. */
int ssm_kv_mass_update(const void *q, const void *k_cache, const float *lse, float *mass,
                       const int32_t *block_table, const int32_t *starts, const int32_t *positions,
                       const int32_t *len_old, const int32_t *lens,
                       int64_t n_tokens, int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                       int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                       int64_t q_stride_token, int64_t q_stride_head,
                       int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                       float scale, float k_scale, ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype, hipStream_t stream);

/* ------------------------------- eviction of the tokens with least weight ----
 * For each request r with more than `budget` tokens, and each kv head g: keeps
 * the last `recent` tokens, and of the earlier ones the budget - recent with the
 * largest mass, the earlier of equal ones (a NaN is larger than any number, and
 * a token on a page outside [0, n_pages) has mass -inf).  The kept tokens move, in
 * their order, to the tokens 0 .. budget - 1 of the request's cache, k, v and
 * mass alike; what stands behind them is left.  Each kv head keeps tokens of its own.
 *   len_out[r] = min(max(lens[r], 0), budget)   (lens cut to max_pages * page_size)
 *   kept[r, g, i] = the place that token i had before, -1 from len_out[r] on
 * A request of up to `budget` tokens is left as it is.  len_out as the len_new
 * (with lens as the len_old) of ssm_kv_pages_step gives the freed pages back.  Keys
 * that were rotated keep the positions that they were rotated by.
 * A token whose old or new place is on a page outside [0, n_pages) is not moved.
 * Layouts: k_cache, v_cache as above, mass (n_pages, n_kv_heads, page_size) fp32
 * contiguous, all updated in place; block_table, lens; len_out (batch), kept
 * (batch, n_kv_heads, budget) int32.  A page belongs to one request here, and
 * stands once in its table.
 * Limits: 1 <= budget <= 2^30, 0 <= recent <= budget; batch * n_kv_heads * budget and
 * n_pages * n_kv_heads * page_size below 2^31; headdim and strides as in
 * ssm_paged_attn_decode_fwd, and different rows of a cache in different places.  No
 * workspace. */
int ssm_kv_evict(void *k_cache, void *v_cache, float *mass, const int32_t *block_table, const int32_t *lens,
                 int32_t *len_out, int32_t *kept, int64_t batch, int64_t n_kv_heads, int64_t headdim,
                 int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                 int64_t budget, int64_t recent,
                 int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                 ssm_kv_dtype_t kv_dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SSM_LONGCTX_H */
