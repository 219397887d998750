/*
 * gdna.h -- C-ABI of libgdn's attention-layer operators: the softmax-attention
 * layers that a hybrid model has between its gated-delta-rule layers (gdn.h),
 * served from a paged key-value cache.
 *
 * One decode step of such a layer is
 *
 *     gdna_page_assign     once a step: which cache page each new token goes to
 *     gdna_qk_norm_rope    per layer: head norms, rotary positions, cache rows
 *     gdna_attn_decode     per layer: the new tokens' attention over the cache
 *
 * Conventions are gdn.h's: device pointers the caller owns, strides in ELEMENTS,
 * asynchronous on `stream`, nothing allocated, arguments checked on the host
 * before anything is launched, status codes GDN_OK / GDN_ERR_*.  Sizes of zero
 * (batch, rows, q_len) are valid empty calls: no CUDA call is made and nothing
 * is written (but for gdna_page_assign with rows 0 and a batch, whose lengths,
 * starts, head and count are).  Values that live on the device
 * (lengths, page numbers, positions, slots) cannot be checked on the host; the
 * kernels check them, and each entry point says what an invalid one does.  No
 * such value makes a kernel leave its buffers.
 *
 * The cache.  K and V are two arrays of `pages` pages of `page_size` tokens of
 * NKV heads of D values, addressed with the same strides:
 *
 *     element(page, token, head, c) = base + page * page_stride
 *                                   + token * token_stride + head * head_stride + c
 *
 * so tokens-then-heads, heads-then-tokens and K/V interleaved by page all fit.
 * A stored element x stands for x * k_scale (x * v_scale).  A sequence's tokens
 * are found through its row of the block table: token j is token j % page_size
 * of page table[b * table_stride + j / page_size].  A slot is
 * page * page_size + token.
 */
#ifndef GDNA_H
#define GDNA_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types.  GDNA_E4M3 (8 bits: 4 exponent, 3 mantissa, no infinities) is
 * a cache type only. */
typedef enum {
    GDNA_F32 = 0,
    GDNA_F16 = 1,
    GDNA_BF16 = 2,
    GDNA_E4M3 = 3,
    GDNA_DTYPE_MAX_ENUM = 0x7fffffff
} gdna_dtype;

/* How gdna_rope_table stretches positions beyond the trained context. */
typedef enum {
    GDNA_ROPE_PLAIN = 0,      /* angle = p * base^(-2i/rot) */
    GDNA_ROPE_LINEAR = 1,     /* positions divided by `factor` */
    GDNA_ROPE_NTK = 2,        /* base multiplied by factor^(rot/(rot-2)): the fastest pair keeps its
                                 frequency, the slowest is divided by `factor` */
    GDNA_ROPE_YARN = 3,       /* by parts: pairs that turn more than beta_fast times within
                                 `original_len` keep their frequency, those that turn less than
                                 beta_slow times are divided by `factor`, a ramp (linear in the pair
                                 index) between */
    GDNA_ROPE_KIND_MAX_ENUM = 0x7fffffff
} gdna_rope_kind;

/*
 * gdna_rope_table -- the cosines and sines of positions [0, n_pos), on the HOST.
 *   table        HOST pointer, [n_pos] rows of `rot` fp32: rot/2 cosines, then
 *                rot/2 sines.  Computed in 64 bits and rounded once (an fp32
 *                angle at position 2^18 is off by up to 0.016 rad).
 *   rot          even, >= 2: elements of a head that are rotated.
 *   base         > 0, finite.  factor >= 1, finite (ignored by GDNA_ROPE_PLAIN).
 *   original_len, beta_fast, beta_slow
 *                GDNA_ROPE_YARN only: > 0, with beta_fast > beta_slow.
 *   amplitude    > 0, finite: multiplies every entry (1 for none; YaRN's
 *                usual 0.1 ln(factor) + 1 scales q.k by its square).
 *   Errors: GDN_ERR_ARG, GDN_ERR_UNSUPPORTED (unknown kind), GDN_ERR_ALIGN.
 */
GDN_API int gdna_rope_table(float *table, int64_t n_pos, int rot, double base, gdna_rope_kind kind,
                            double factor, double original_len, double beta_fast, double beta_slow,
                            double amplitude);

/*
 * gdna_page_assign -- block tables, slots and positions of a step's new tokens,
 * built on the GPU from the sequences' lengths.
 *   cached       [batch] tokens of each sequence that are in the cache.
 *   fresh        [batch] new tokens of each sequence (0 or more).  Negative
 *                values of either count as 0.
 *   table        [batch] rows of max_pages page numbers, row stride
 *                table_stride: entries of the pages a sequence holds are read,
 *                entries of the pages it takes are written.
 *   free_pages   [n_free] page numbers; free_pages[free_head[0] ..] are free and
 *                are taken in order, sequence by sequence.  (To give pages
 *                back, put them in front of the head and lower it.)
 *   free_head    [1].
 *   kv_len       [batch] written: cached + fresh (cached where not served).
 *   row_start    [batch + 1] written: first token row of each sequence, at most
 *                `rows`; row_start[batch] is the number of rows in use.
 *   slots        [rows] written: the cache slot of each token row, or -1: rows
 *                past the last token (a padded, graph-captured step) and rows of
 *                sequences that are not served.
 *   positions    [rows] written: the token's position in its sequence (0 for
 *                padding rows).
 *   free_head_out [1] written: the head after this call.
 *   unserved     [1] written: how many sequences with new tokens got none of
 *                them placed.
 *   Sequences are served in order.  One is not served where its pages would not
 *   fit its table row, where its rows would not fit `rows`, or where the free
 *   pages have run out; from the first that runs out of pages on, only sequences
 *   that need no page are served.  A sequence that is not served takes no page.
 *   A negative entry of the table or of free_pages gives slot -1.
 *   A batch of 0 is an empty call like any other: no output is written, whatever
 *   `rows`.  A caller that swaps two head buffers each step does not swap them
 *   then, and has no row to store.
 *   No output may overlap another operand (pass two buffers in turn for
 *   free_head).  Results do not depend on timing.
 *   Limits: batch <= 2^20, page_size, max_pages >= 1, rows < 2^31 - 4096
 *   (GDN_ERR_UNSUPPORTED).
 */
GDN_API int gdna_page_assign(const int32_t *cached, const int32_t *fresh, int32_t *table, int64_t table_stride,
                             const int32_t *free_pages, int64_t n_free, const int32_t *free_head,
                             int32_t *kv_len, int32_t *row_start, int64_t *slots, int32_t *positions,
                             int32_t *free_head_out, int32_t *unserved,
                             int batch, int64_t rows, int page_size, int max_pages, void *stream);

/*
 * gdna_qk_norm_rope -- per-head RMS norm of queries and keys, rotary positions
 * and the cache's new rows, in one pass.  Per token row and head x of D values:
 *     y = w * x / sqrt(mean x^2 + eps)                    (y = x if w is NULL)
 *     the first `rot` elements of y in pairs, (a, b) -> (a cos - b sin,
 *     a sin + b cos); pairs (i, i + rot/2), or (2i, 2i + 1) if `interleaved`.
 *   q            [rows] rows of NQ heads: row stride q_stride, head stride
 *                q_head_stride (so a projection that holds a gate beside each
 *                head is read in place).  NULL with NQ = 0 for none.
 *   k, v         [rows] rows of NKV*D, row strides k_stride, v_stride.  v may be
 *                NULL (no V cache rows then; v_cache NULL).  k NULL with NKV = 0
 *                for none.
 *   dtype        type of q, k, v, q_out and k_out: GDNA_F32, F16 or BF16.
 *   qn, kn       [D] fp32 norm weights, or NULL for no norm.
 *   cos_sin      [n_pos] rows of rot fp32 (gdna_rope_table's layout), device.
 *   positions    [rows] int32.  A position outside [0, n_pos) has no angle: the
 *                rotated elements come out NaN.  Both may be NULL with rot = 0.
 *   slots        [rows] int64 cache slots; a row whose slot is outside
 *                [0, pages * page_size) is not stored (padding: -1).
 *   q_out        [rows] rows of NQ*D, stride q_out_stride.
 *   k_out        NULL, or [rows] rows of NKV*D, stride k_out_stride: the
 *                rotated keys beside (or, with k_cache NULL, instead of) the
 *                cache.
 *   k_cache, v_cache  the cache, of type cache_dtype (F16, BF16 or E4M3), or
 *                both NULL.  Stored: the fp32 value divided by k_scale (v_scale)
 *                and rounded to nearest even once; E4M3 saturates at +-448.
 *                Two rows with the same slot: either may be kept.
 *   q_out may be q itself (same base, strides q_stride and q_head_stride = D);
 *   otherwise an output overlapping any operand is GDN_ERR_ALIAS.  Rows of one
 *   stride that lie side by side (q, k and v of one projection) do not overlap,
 *   and k_cache and v_cache may be interleaved in one buffer.
 *   1 <= D <= 256, rot even and <= D, norms and rotations in fp32.  Head sizes
 *   64, 128 and 256 with rot a multiple of 8, on boundaries of four elements, run
 *   a vector kernel; any other call runs a general one, two to three times slower, which
 *   takes at most 2^34 - 8 heads (rows * (NQ + NKV + NKV)) a call
 *   (GDN_ERR_UNSUPPORTED).
 */
GDN_API int gdna_qk_norm_rope(const void *q, const void *k, const void *v, gdna_dtype dtype,
                              const float *qn, const float *kn, float eps,
                              const float *cos_sin, int64_t n_pos, int rot, int interleaved,
                              const int32_t *positions, const int64_t *slots,
                              void *q_out, void *k_out, void *k_cache, void *v_cache, gdna_dtype cache_dtype,
                              float k_scale, float v_scale,
                              int64_t rows, int nq, int nkv, int d, int64_t pages, int page_size,
                              int64_t q_stride, int64_t q_head_stride, int64_t k_stride, int64_t v_stride,
                              int64_t q_out_stride, int64_t k_out_stride,
                              int64_t page_stride, int64_t token_stride, int64_t head_stride, void *stream);

/*
 * gdna_attn_workspace -- bytes of scratch that gdna_attn_decode needs for a
 * shape on any GPU this library runs on (never more for fewer sequences, tokens
 * or heads); 0 if the shape is not supported.  Makes no CUDA call.
 */
GDN_API int64_t gdna_attn_workspace(int batch, int q_len, int nq, int nkv, int d);

/*
 * gdna_attn_decode -- softmax attention of the q_len newest tokens of each
 * sequence (one in a decode step, a few in a verify step) over its cache, the
 * cache's length split over the GPU and joined.
 *   Token t of sequence b (row b*q_len + t) sees keys j < kv_len[b] -
 *   (q_len - 1 - t): kv_len counts the new tokens, whose rows are in the cache.
 *     o = sum_j softmax_j(scale * k_scale * q.k_j) * v_scale * v_j
 *   A row that sees no key gives 0.  With `gate`, o * sigmoid(gate).
 *   q            [batch*q_len] rows of NQ*D, stride q_stride, type dtype.
 *                Query head h reads key head h / (NQ/NKV).
 *   gate         NULL, or [batch*q_len] rows of NQ heads of type dtype, row
 *                stride gate_stride, head stride gate_head_stride.
 *   k_cache, v_cache, cache_dtype (F16, BF16, E4M3), k_scale, v_scale: the cache.
 *   table, max_pages, table_stride: the block table.  Entries past a sequence's
 *                length are not read.  A page number outside [0, pages) reads as
 *                a page of zeros.
 *   kv_len       [batch] int32.  Below 0 counts as 0; above max_pages *
 *                page_size (or 2^31 - 4096) as that.
 *   scale        finite; > 0 (usually 1/sqrt(D)).
 *   out          [batch*q_len] rows of NQ*D, stride out_stride, type out_dtype
 *                (F32, F16 or BF16), rounded once.
 *   lse          NULL, or [batch*q_len][NQ] fp32, contiguous: the natural
 *                logarithm of the softmax's denominator (-inf where no key), to
 *                join with attention over other keys.
 *   workspace    device scratch of workspace_bytes >= gdna_attn_workspace(),
 *                16-byte aligned; any content, and none is kept.  Calls that
 *                can overlap on the GPU need separate ones.
 *   NQ must be a multiple of NKV (GDN_ERR_UNSUPPORTED).  1 <= D <= 256.  Heads of
 *   a multiple of 16 bytes on 16-byte aligned caches (bases and strides) run on
 *   the tensor cores; any other call runs a general kernel, six to fifty times
 *   slower, with the same results up to rounding.  Page sizes that 16 divides are
 *   the fastest, multiples of 8 and of 4 nearly so.
 *   Scores, softmax sums and outputs are held in fp32; queries and weights enter
 *   the products in two or three 16-bit parts where one would show in the output.
 *   On the tensor cores an F32 query over a BF16 cache keeps 16 bits where out is
 *   BF16 and lse NULL, else all 24; a weight over an F16 or E4M3 cache is held to
 *   2^-22 of itself or 2^-40 of its row's largest, whichever is more, over a BF16
 *   cache to 2^-16 of itself (F32 out: 2^-24).
 *   A value or key that is not finite shows in the rows that see it; but a key
 *   whose score with a row is -inf has weight 0 there, and a row of no other key
 *   gives 0.  Results do not depend on timing.
 *   The tensor-core kernels' waits for their own copies are bounded
 *   (gdn_set_wait_polls); where one runs out the rows of that block come out NaN
 *   and gdn_device_wait_timeouts counts it.
 */
GDN_API int gdna_attn_decode(const void *q, gdna_dtype dtype, const void *gate,
                             const void *k_cache, const void *v_cache, gdna_dtype cache_dtype,
                             float k_scale, float v_scale,
                             const int32_t *table, int64_t table_stride, const int32_t *kv_len, float scale,
                             void *out, gdna_dtype out_dtype, float *lse,
                             void *workspace, int64_t workspace_bytes,
                             int batch, int q_len, int nq, int nkv, int d,
                             int64_t pages, int page_size, int max_pages,
                             int64_t q_stride, int64_t gate_stride, int64_t gate_head_stride, int64_t out_stride,
                             int64_t page_stride, int64_t token_stride, int64_t head_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDNA_H */
