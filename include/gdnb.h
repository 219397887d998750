/*
 * gdnb.h -- C-ABI of libgdn's decoder-block operators: what joins the layers of
 * a hybrid model (gdn.h, gdna.h) into blocks, and its attention layers' prompts.
 *
 *     gdnb_residual_norm   the norm after a block, its gate and residual scale,
 *                          and the norm before the next, in one pass
 *     gdnb_attn_prompt     causal attention over whole prompts: packed sequences
 *                          of different lengths, over the paged cache or over
 *                          rows that were never stored
 *     gdnb_attn_shared     a decode step of requests that share a long prefix,
 *                          whose keys are read once for all of them
 *
 * Conventions are gdna.h's: device pointers the caller owns, strides in ELEMENTS,
 * asynchronous on `stream`, nothing allocated, arguments checked on the host
 * before anything is launched, status codes GDN_OK / GDN_ERR_*.  Sizes of zero
 * (batch, rows, q_len) are valid empty calls: no CUDA call is made and nothing is
 * written.  Values that live on the device (lengths, starts, page numbers) cannot
 * be checked on the host; the kernels check them, and none makes a kernel leave
 * its buffers.  The cache, its types and its addressing are gdna.h's.
 */
#ifndef GDNB_H
#define GDNB_H

#include "gdna.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gdnb_residual_norm -- per row of C elements:
 *     u  = post * y / sqrt(mean y^2 + eps)            (u = y if post is NULL)
 *     x' = x + scale * gate * u                       (no gate if NULL; x' = x if y is NULL)
 *     h  = pre * x' / sqrt(mean x'^2 + eps)           (pre NULL: weights of 1)
 *   x, x_dtype   [rows] rows of C, stride x_stride: the residual stream (F32, F16
 *                or BF16).
 *   y, y_dtype   NULL, or [rows] rows of C, stride y_stride: the block's output.
 *   gate         NULL, or [rows] rows of C of type y_dtype, stride gate_stride;
 *                gate_stride 0: one row for all.
 *   post, pre    [C] fp32 weights, or NULL.
 *   x_out        NULL, or rows of type x_dtype, stride x_out_stride.  May be x
 *                itself (same base and stride).
 *   h, h_dtype   NULL, or rows of type h_dtype, stride h_stride.  May be y itself (same
 *                base, stride and type).
 *   One of x_out and h is given.  gate and post need y.  scale finite; eps >= 0,
 *   finite.  All sums and products in fp32, x' and h each rounded once (h from the
 *   unrounded x').  An output overlapping any other operand is GDN_ERR_ALIAS; rows
 *   of one stride that lie side by side do not overlap.
 *   1 <= C <= 16384 (GDN_ERR_UNSUPPORTED).  Rows and strides on 16-byte boundaries
 *   with C a multiple of 8 are taken 16 bytes at a time; so are rows that all begin
 *   equally far behind a boundary of eight elements (an odd C, rows side by side, 64
 *   <= C <= 16370) but for their ends, at about half the rate; any other call goes
 *   element by element, at half of that.
 */
GDN_API int gdnb_residual_norm(const void *x, gdna_dtype x_dtype, const void *y, gdna_dtype y_dtype,
                               const void *gate, const float *post, const float *pre, float scale, float eps,
                               void *x_out, void *h, gdna_dtype h_dtype, int64_t rows, int c,
                               int64_t x_stride, int64_t y_stride, int64_t gate_stride,
                               int64_t x_out_stride, int64_t h_stride, void *stream);

/*
 * gdnb_attn_prompt_workspace -- bytes of scratch that gdnb_attn_prompt needs for a
 * shape on any GPU this library runs on (never more for fewer rows or sequences);
 * 0 if the shape is not supported.  Makes no CUDA call.
 */
GDN_API int64_t gdnb_attn_prompt_workspace(int64_t rows, int batch, int nq, int nkv, int d);

/*
 * gdnb_attn_prompt -- causal softmax attention of packed sequences of different
 * lengths: whole prompts, pieces of prompts over what is cached already, and
 * single tokens of decoding requests in one call.
 *   Sequence b's tokens are rows row_start[b] .. row_start[b+1] - 1; its t-th of n
 *   sees keys j < kv_len[b] - (n - 1 - t): kv_len counts the new tokens, whose keys
 *   are in the cache (gdna_page_assign's row_start and kv_len, after
 *   gdna_qk_norm_rope stored the rows).
 *     o = sum_j softmax_j(scale * k_scale * q.k_j) * v_scale * v_j
 *   A row that sees no key gives 0.  With `gate`, o * sigmoid(gate).
 *   q, dtype     [rows] rows of NQ*D, stride q_stride, F32, F16 or BF16.  Query head h
 *                reads key head h / (NQ/NKV).
 *   gate         NULL, or [rows] rows of NQ heads of type dtype, row stride
 *                gate_stride, head stride gate_head_stride.
 *   k_cache, v_cache, cache_dtype (F16, BF16, E4M3), k_scale, v_scale: the cache.
 *   table, max_pages, table_stride: the block table.  Entries past a sequence's
 *                length are not read.  A page number outside [0, pages) reads as a
 *                page of zeros.
 *                table NULL: the keys were never stored in pages.  k_cache and
 *                v_cache are [rows] rows of NKV heads, strides token_stride and
 *                head_stride, and key j of sequence b is row row_start[b] + j;
 *                pages, page_size, max_pages and page_stride are not looked at.
 *                F16 or BF16.
 *   row_start    [batch + 1] int32.  Values are cut to [0, rows], and an end to its
 *                start.  Rows of no sequence are left as they were.  Where starts go
 *                back, so that sequences overlap, each element of a row of several
 *                is of one of their results, and may be of another in the next call.
 *   kv_len       [batch] int32.  Below 0 counts as 0; above max_pages * page_size (or
 *                2^31 - 4096) as that.  NULL with table NULL (the rows' number);
 *                given with it, cut to the rows' number.
 *   scale        finite; > 0 (usually 1/sqrt(D)).
 *   out          [rows] rows of NQ*D, stride out_stride, F16 or BF16, rounded once.
 *   workspace    device scratch of workspace_bytes >= gdnb_attn_prompt_workspace(),
 *                16-byte aligned; any content, and none is kept.  Calls that can
 *                overlap on the GPU need separate ones.
 *   NQ a multiple of NKV, NQ/NKV <= 128, 1 <= D <= 256, batch <= 65536, rows <= 2^31 -
 *   4096 (GDN_ERR_UNSUPPORTED).
 *   Scores, softmax sums and outputs are held in fp32.  The products are of 16-bit
 *   operands, bf16 over a BF16 cache, else fp16: the keys and values exactly, the
 *   queries in one part where that type holds theirs, else in two (an F32 query
 *   keeps 16 bits over a BF16 cache, 22 over the others), and the weights in one
 *   part: to 2^-8 of themselves over a BF16 cache; over the others to 2^-11 of
 *   themselves or 2^-32 of the row's largest, whichever is more.
 *   A value or key that is not finite shows (as NaN or infinity) in the rows that see
 *   it, and in no other; but a key whose score with a row is -inf (an infinite one
 *   whose sign there is the query's opposite) has weight 0 there, and a row of no
 *   other key gives 0.  (An F32 query's two parts may make that score NaN.)
 *   Results do not depend on timing.
 *   Caches (bases and strides) on 16-byte boundaries with pages of a multiple of 8
 *   tokens (E4M3: 4, and heads above 64) are brought in by tensor copies; other pages
 *   by loads of 16 bytes, up to three times slower; heads of no multiple of 16 bytes
 *   and unaligned caches element by element, up to eight times slower.
 *   The kernels' waits for their own copies and products are bounded
 *   (gdn_set_wait_polls; a wait that lasts as long as a sequence's keys by 256 times
 *   the polls); where one runs out, that block's rows are incomplete and
 *   gdn_device_wait_timeouts counts it.
 */
GDN_API int gdnb_attn_prompt(const void *q, gdna_dtype dtype, const void *gate,
                             const void *k_cache, const void *v_cache, gdna_dtype cache_dtype,
                             float k_scale, float v_scale,
                             const int32_t *table, int64_t table_stride,
                             const int32_t *row_start, const int32_t *kv_len, float scale,
                             void *out, gdna_dtype out_dtype, void *workspace, int64_t workspace_bytes,
                             int64_t rows, int batch, int nq, int nkv, int d,
                             int64_t pages, int page_size, int max_pages,
                             int64_t q_stride, int64_t gate_stride, int64_t gate_head_stride, int64_t out_stride,
                             int64_t page_stride, int64_t token_stride, int64_t head_stride, void *stream);

/*
 * gdnb_attn_shared_workspace -- bytes of scratch that gdnb_attn_shared needs for a
 * shape on any GPU this library runs on (never more for fewer requests, groups or
 * tokens); 0 if the shape is not supported.  Makes no CUDA call.
 */
GDN_API int64_t gdnb_attn_shared_workspace(int batch, int groups, int q_len, int nq, int nkv, int d);

/*
 * gdnb_attn_shared -- gdna_attn_decode for requests that begin alike: group g is
 * the requests group_start[g] .. group_start[g+1] - 1, and each of its tokens sees
 * all shared_len[g] keys of the group's prefix, which are read once for all of them,
 * and then its request's own keys as gdna_attn_decode has them: token t of request b
 * (row b*q_len + t) sees own keys j < kv_len[b] - (q_len - 1 - t).  Positions are
 * the caller's: own token j stands at shared_len[g] + j.
 *   group_start  [groups + 1] int32, or NULL: one group of the whole batch (groups 1).
 *                Values are cut to [0, batch], and an end to its start.  Requests of
 *                no group are not written; where starts go back, so that groups
 *                overlap, nothing may be.
 *   shared_table [groups] rows of max_shared_pages page numbers, stride
 *                shared_stride.  shared_len [groups] int32.  Both as table and kv_len
 *                below.
 *   table, max_pages, table_stride, kv_len: the requests' own pages and lengths.
 *   The other arguments, limits and precisions are gdnb_attn_prompt's (own keys of
 *   many requests: gdna_attn_decode's), with batch * q_len <= 2^31 - 4096 and the limits of
 *   gdna_attn_decode.
 */
GDN_API int gdnb_attn_shared(const void *q, gdna_dtype dtype, const void *gate,
                             const void *k_cache, const void *v_cache, gdna_dtype cache_dtype,
                             float k_scale, float v_scale,
                             const int32_t *group_start, int groups,
                             const int32_t *shared_table, int64_t shared_stride, const int32_t *shared_len,
                             const int32_t *table, int64_t table_stride, const int32_t *kv_len, float scale,
                             void *out, gdna_dtype out_dtype, void *workspace, int64_t workspace_bytes,
                             int batch, int q_len, int nq, int nkv, int d,
                             int64_t pages, int page_size, int max_shared_pages, int max_pages,
                             int64_t q_stride, int64_t gate_stride, int64_t gate_head_stride, int64_t out_stride,
                             int64_t page_stride, int64_t token_stride, int64_t head_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDNB_H */
