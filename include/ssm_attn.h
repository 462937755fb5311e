/*
 * ssm_attn.h -- C interface of libssmscan.so for the attention layers that hybrid
 * models put between their state-space layers: a paged key-value cache, the
 * norm and position rotation of the heads that enter it, and attention of one
 * new token over it.
 *
 * The conventions are those of ssm_scan.h: caller-owned device buffers, nothing
 * allocated, nothing synchronised, work enqueued on `stream`, every argument
 * checked before any HIP call, ssm_last_error() after a negative status, and
 * results that are bitwise reproducible run to run (no floating-point atomics).
 * Two of them are widened here, because q, k and v usually are slices of one
 * projection's rows and a cache usually is a view: tensors may be strided (the
 * strides are in elements, the last dimension has stride 1), and pointers need
 * only their element's alignment unless a limit below asks for more.  A
 * workspace is an output: it may alias no other argument.
 *
 * What the operators compute stands at each of them; the definitions are the
 * common ones of decoder models and are not taken from the pages that
 * ssm_scan.h cites.
 */
#ifndef SSM_ATTN_H
#define SSM_ATTN_H

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element type of a key-value cache */
typedef enum {
    SSM_KV_F32 = 0,      /* with SSM_F32 heads */
    SSM_KV_BF16 = 1,     /* with SSM_BF16 heads */
    SSM_KV_F8E4M3 = 2    /* with SSM_BF16 heads: OCP e4m3 (no infinities, largest 448), value = stored * scale */
} ssm_kv_dtype_t;

/* flags of the norm and rotation entry points */
#define SSM_ROPE_INTERLEAVED 0x1u   /* pairs (2j, 2j+1); default: pairs (j, j + rot_dim/2) */
#define SSM_QK_NO_NORM       0x2u   /* rotation only; wq and wk are then not read */

/* Largest head size of these entry points, and most requests of one page step. */
#define SSM_ATTN_MAX_HEADDIM 256
#define SSM_KV_MAX_BATCH 4096

/* ------------------------------------------- pages of a key-value cache ----
 * One scheduling step of a paged cache, on the device: requests grow, shrink
 * or end, pages are taken from a ring of free pages and given back to it, and
 * the new tokens get their request, position and cache slot.
 *
 * A cache has n_pages pages of page_size tokens.  Request r keeps its pages in
 * block_table[r, 0 .. ceil(len_old[r] / page_size)).  The free pages stand in
 * free_ring (n_pages entries) from place `head`, `free` of them, wrapping;
 * ring = {head, free}.  With have = ceil(len_old / page_size) and
 * want = ceil(len_new / page_size):
 *   - request r is refused if want > max_pages, or if it needs pages and the
 *     needs of the requests up to it (those over max_pages left out) exceed
 *     `free`.  It keeps its length and pages, and its new tokens get slot -1.
 *   - the others take want - have pages from the ring's head, in request order
 *     and page order, into block_table[r, have ..), or give back the pages
 *     block_table[r, want .. have) behind the ring's last entry.  Pages given
 *     back can be taken by the next step, not by this one.
 *   - new tokens are numbered request by request: request r has the
 *     max(len_new - len_old, 0) tokens from starts[r] on (a refused request has
 *     them too), at positions len_old[r] onwards; token t of request r at
 *     position p gets slot = page * page_size + p % page_size with page =
 *     block_table[r, p / page_size].  Tokens past the last one have request,
 *     position and slot -1, and tokens past n_tokens are not written.
 * Table entries that no request holds are left as they are.
 *
 * Layouts: len_old, len_new (batch) int32 (negative counts as 0); block_table
 * (batch, max_pages) int32, row stride table_stride, updated in place;
 * free_ring (n_pages) int32, updated in place; ring, ring_out (2) int32;
 * len_out (batch) int32: the length each request has now; starts (batch + 1)
 * int32: first token of each request, and their number; request, positions
 * (n_tokens) int32; slots (n_tokens) int64; denied (1) int32: refused requests.
 * request, positions and slots may be NULL when n_tokens is 0.  No output may
 * alias an input or another output (block_table and free_ring are both).
 * Limits: batch <= SSM_KV_MAX_BATCH; batch * max_pages, n_tokens and n_pages *
 * page_size below 2^31; the new tokens' number below 2^31.  request, positions
 * and slots 16-byte aligned.  No workspace. */
int ssm_kv_pages_step(const int32_t *len_old, const int32_t *len_new, int32_t *block_table,
                      int32_t *free_ring, const int32_t *ring, int32_t *ring_out, int32_t *len_out,
                      int32_t *starts, int32_t *request, int32_t *positions, int64_t *slots, int32_t *denied,
                      int64_t batch, int64_t max_pages, int64_t table_stride, int64_t n_pages,
                      int64_t page_size, int64_t n_tokens, hipStream_t stream);

/* ------------------------- norm of q and k heads with position rotation ----
 * For each token t and each head x of q and of k (headdim values):
 *   y = x * w / sqrt(mean(x^2) + eps)       (y = x under SSM_QK_NO_NORM)
 *   theta_j = positions[t] * inv_freq[j],   j < rot_dim / 2
 *   (out[a], out[b]) = (y[a] cos theta_j - y[b] sin theta_j, y[b] cos theta_j + y[a] sin theta_j)
 * with (a, b) = (j, j + rot_dim/2), or (2j, 2j+1) under SSM_ROPE_INTERLEAVED;
 * out = y from rot_dim on.  w is wq for q heads and wk for k heads.
 * Arithmetic: fp32, the angle formed and reduced to a turn in fp64 (off by 2^-24
 * at most at positions up to 2^28, by 5e-7 at 2^31), outputs rounded once.
 *
 * Layouts: q (n_tokens, n_heads, headdim), k (n_tokens, n_kv_heads, headdim)
 * [dtype] with the given strides; wq, wk (headdim) fp32; inv_freq (rot_dim/2)
 * fp32; positions (n_tokens) int32; q_out, k_out [dtype] contiguous.  q_out may
 * be q and k_out may be k where those are contiguous; no other aliasing.
 * Limits: headdim <= SSM_ATTN_MAX_HEADDIM; rot_dim even, 0 <= rot_dim <=
 * headdim (0: inv_freq and positions may be NULL); n_kv_heads may be 0 (k,
 * k_out, wk may be NULL).  No workspace. */
int ssm_qk_norm_rope_fwd(const void *q, const void *k, const float *wq, const float *wk,
                         const float *inv_freq, const int32_t *positions, void *q_out, void *k_out,
                         int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads, int64_t headdim, int64_t rot_dim,
                         int64_t q_stride_token, int64_t q_stride_head,
                         int64_t k_stride_token, int64_t k_stride_head,
                         float eps, ssm_dtype_t dtype, uint32_t flags, hipStream_t stream);

/* Gradients of ssm_qk_norm_rope_fwd given dq_out, dk_out: with g the cotangent
 * turned back by -theta, r = 1/sqrt(mean(x^2) + eps) and n = x r,
 *   dx = r (w g - n mean(w g n)),   dw = sum over tokens and heads of g n
 * (dx = g under SSM_QK_NO_NORM; dwq and dwk are then not written).
 * Layouts: q, k, dq_out, dk_out [dtype] strided; dq, dk [dtype] contiguous (dq
 * may be dq_out and dk may be dk_out where those are contiguous); dwq, dwk
 * (headdim) fp32, or NULL under SSM_QK_NO_NORM.  The sums are held in fp32 over
 * at most 32 heads of a lane and over a block's lanes, and in fp64 else, in an
 * order fixed by the shape: their error does not grow with the tokens.
 * Limits as for the forward.
 * Workspace: ssm_qk_norm_rope_bwd_workspace_size() bytes, 16-byte aligned (the
 * blocks' shares of dwq and dwk; 0 under SSM_QK_NO_NORM). */
size_t ssm_qk_norm_rope_bwd_workspace_size(int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads,
                                           int64_t headdim, uint32_t flags);

int ssm_qk_norm_rope_bwd(const void *q, const void *k, const float *wq, const float *wk,
                         const float *inv_freq, const int32_t *positions,
                         const void *dq_out, const void *dk_out, void *dq, void *dk, float *dwq, float *dwk,
                         int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads, int64_t headdim, int64_t rot_dim,
                         int64_t q_stride_token, int64_t q_stride_head,
                         int64_t k_stride_token, int64_t k_stride_head,
                         int64_t dq_stride_token, int64_t dq_stride_head,
                         int64_t dk_stride_token, int64_t dk_stride_head,
                         float eps, ssm_dtype_t dtype, uint32_t flags,
                         void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------ the same pass with k and v written into the cache ----
 * q_out as ssm_qk_norm_rope_fwd; the normed and rotated k and the unchanged v
 * of token t go to slot slots[t] of the cache, slot = page * page_size + place.
 * Tokens whose slot lies outside [0, n_pages * page_size) write nothing into
 * the cache (their q_out is written).  Two tokens with one slot: which of them
 * is kept is not defined.
 * An SSM_KV_F8E4M3 cache stores k / k_scale and v / v_scale, clamped to
 * [-448, 448] and rounded once from fp32 (NaN stays NaN); the other types store
 * the values (k_scale and v_scale are then not read).
 *
 * Layouts: q, k, v [dtype] strided; slots (n_tokens) int64; k_cache, v_cache
 * (n_pages, page_size, n_kv_heads, headdim) [kv_dtype], any strides with the
 * last one 1, the same strides for both.  The rest as ssm_qk_norm_rope_fwd.
 * Limits: n_kv_heads >= 1; n_pages * page_size below 2^31.  No workspace. */
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
                               uint32_t flags, hipStream_t stream);

/* ------------------------ attention of one new token over the cache ----
 * For each row r (one new token of a request) and query head h, with kv head
 * g = h * n_kv_heads / n_heads and the cached tokens j in [lo, len), len =
 * lens[r] and lo = max(0, len - window) (0 without a window):
 *   s_j = scale * k_scale * q[r,h] . k[j,g]
 *   o[r,h] = v_scale * sum_j exp(s_j) v[j,g] / sum_j exp(s_j),   lse[r,h] = log sum_j exp(s_j)
 * where token j is row j % page_size of page block_table[r, j / page_size].
 * lens counts the new token too if its k and v are in the cache already.  A row
 * with no token (len <= 0, or every score -inf) has o = 0 and lse = -inf.
 * len is cut to max_pages * page_size.  Tokens on a page outside [0, n_pages)
 * are left out, and cache rows outside the row's tokens are never used,
 * whatever they hold (NaN included).  Rows may share pages and requests: the
 * tokens of a prompt are rows with growing lens.
 * Arithmetic: products on the matrix cores (bf16 products are exact in fp32;
 * 8-bit caches are widened to bf16, which is exact; fp32 stays fp32), sums,
 * maxima and exponentials in fp32; exp(s_j) enters its product with v with all
 * its bits (as the sum of three bf16 values where v is bf16 or 8-bit), and the
 * output is rounded once.
 *
 * Layouts: q (batch, n_heads, headdim) [dtype] strided; k_cache, v_cache as
 * above [kv_dtype]; block_table (batch, max_pages) int32, row stride
 * table_stride; lens (batch) int32; o (batch, n_heads, headdim) [dtype]
 * contiguous; lse (batch, n_heads) fp32 or NULL.  No output may alias an input.
 * Limits: n_heads % n_kv_heads == 0; headdim a multiple of 8 (of 16 for an
 * 8-bit cache), <= SSM_ATTN_MAX_HEADDIM; q, o, k_cache, v_cache 16-byte aligned
 * and every stride of q and of the caches a multiple of 16 bytes; max_pages *
 * page_size at most 2^30, n_pages * page_size below 2^31; a cache's extent below
 * 2^36 bytes; batch * n_kv_heads * max_pages * page_size / 16 below 2^31 (all
 * times the passes).
 * The cache is read once per 16 query heads of a kv head.  Work is cut by
 * length, not by row, into equal shares over the chip, whatever the lengths
 * are, and the shares of a row are joined by their maxima and sums; where the
 * table or the window keeps every row short, a row's head is one share (one
 * launch instead of two).  Which of the two follows from the arguments, not
 * from lens.  An infinite v gives NaN where the formula may give an infinity.
 * Workspace: ssm_paged_attn_decode_fwd_workspace_size() bytes, 16-byte aligned
 * (the rows' places in the work, and the unjoined shares). */
size_t ssm_paged_attn_decode_fwd_workspace_size(int64_t batch, int64_t n_heads, int64_t n_kv_heads,
                                                int64_t headdim, int64_t max_pages, int64_t page_size);

int ssm_paged_attn_decode_fwd(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *block_table, const int32_t *lens, void *o, float *lse,
                              int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                              int64_t max_pages, int64_t table_stride, int64_t n_pages, int64_t page_size,
                              int64_t q_stride_row, int64_t q_stride_head,
                              int64_t cache_stride_page, int64_t cache_stride_token, int64_t cache_stride_head,
                              float scale, int64_t window, float k_scale, float v_scale,
                              ssm_dtype_t dtype, ssm_kv_dtype_t kv_dtype,
                              void *workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SSM_ATTN_H */
