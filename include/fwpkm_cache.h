/*
 * fwpkm_cache.h -- C ABI of the paged key-value cache (B200, sm_100a).
 *
 * The fast-weight memory of fwpkm.h holds the distant past of a sequence in a
 * table of fixed size; the attention layers that a model has beside it keep
 * the keys and values of the tokens themselves.  The two calls here write
 * such a cache and read it for one new token of every sequence:
 *
 *   fwpkm_cache_append  new keys and values into the cache's pages, with the
 *                       position rotation of keys and queries on the way
 *   fwpkm_cache_attend  softmax attention of one token of each sequence over
 *                       its cached tokens, split over the cache's length and
 *                       joined
 *
 * Conventions are those of fwpkm.h: pointers to memory the CALLER owns, on
 * the current CUDA device (4-byte aligned where nothing else is said); work
 * enqueued asynchronously on `stream`; status codes, with the message in
 * fwpkm_last_error(); argument checks on the host before anything is enqueued.
 * Neither call allocates, synchronises or keeps anything from one call for the
 * next, so calls on different streams need no order beyond that of their data,
 * and both may be captured into CUDA graphs.
 */
#ifndef FWPKM_CACHE_H_
#define FWPKM_CACHE_H_

#include "fwpkm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of a cache beside FWPKM_F32 and FWPKM_BF16: 8-bit floats with
 * 4 exponent and 3 mantissa bits (finite range +-448), each cached head with
 * its own scale. */
enum { FWPKM_E4M3 = 2 };

/* Position rotation: which two elements of a head turn together. */
enum {
  FWPKM_ROTATE_HALVES = 0, /* elements j and j + rotary/2 */
  FWPKM_ROTATE_PAIRS = 1   /* elements 2j and 2j + 1      */
};

#define FWPKM_CACHE_MAX_DIM 256

/* Bits of *device_errors (set, never cleared, by the kernels). */
#define FWPKM_CACHE_BAD_PAGE 32u   /* a needed table entry is no page of the pool          */
#define FWPKM_CACHE_BAD_LENGTH 64u /* a length is negative, beyond the table, or, in append, */
                                   /* less than the sequence's new tokens                   */

/*
 * The pool of pages.  Token r of page p, cached head h, is the `dim`
 * consecutive elements at p*page_stride + h*head_stride + r*row_stride of
 * `keys` and of `values` (strides in elements, non-negative, each a whole
 * number of 16 bytes; the pointers 16-byte aligned).  A contiguous
 * [pages][kv_heads][page_size][dim] pool and a [pages][page_size][kv_heads]
 * [dim] one are both of this form.
 *   dim       8 .. 256, a multiple of 8; of 16 with FWPKM_E4M3
 *   dtype     FWPKM_F32, FWPKM_BF16 or FWPKM_E4M3
 *   key_scale, value_scale   device fp32 [kv_heads] or NULL (1): an E4M3
 *             element e of head h stands for e * scale[h].  NULL for the
 *             other types.  A key scale that is not finite makes the scores of
 *             its head's visible tokens NaN.
 */
typedef struct {
  void *keys, *values;
  int64_t page_stride, head_stride, row_stride;
  int64_t pages; /* 1 .. 2^31 - 1 */
  int page_size; /* tokens per page, >= 1 */
  int kv_heads;  /* 1 .. 1024 */
  int dim;
  int dtype;
  const float *key_scale, *value_scale;
} fwpkm_cache;

/*
 * The sequences of a call.  Token t of sequence b is row t % page_size of
 * page table[b*table_stride + t / page_size].
 *   B         sequences, 1 .. 2^22 (in attend, B * heads <= 2^22)
 *   table     device int32, table_width entries a row; rows may overlap
 *             (table_stride >= 0, 0: one row for all), and sequences may share
 *             pages that they do not write.  Entries that no token of the call
 *             needs are not looked at (a page given back may be -1).
 *   lengths   device int32 [B]: tokens of sequence b, the new ones included.
 */
typedef struct {
  int B;
  int table_width; /* >= 1 */
  int64_t table_stride;
  const int32_t *table, *lengths;
} fwpkm_cache_batch;

/*
 * fwpkm_cache_append -- write new tokens.
 * Rows starts[b] .. starts[b+1]-1 of k and v are the last tokens of sequence
 * b: with n = starts[b+1] - starts[b], row starts[b] + i has position
 * lengths[b] - n + i.  With starts == NULL there is one row a sequence (rows
 * == B), and a sequence of length 0 has none (its row is left alone).  Rows
 * from starts[B] on (a batch padded to a fixed size) are not touched: neither
 * read into the cache nor written in q_out.
 *   Rotation by position p: elements (a, b) of a pair j, 0 <= j < rotary/2,
 * become (a cos x - b sin x, b cos x + a sin x), x = p * freqs[j] formed in 64
 * bits.  Keys are rotated in 32 bits, rounded to the cache's type (E4M3: after
 * the division by the head's scale, saturating at +-448) and stored; values are
 * stored without the rotation, in the same way; queries, where given, are
 * rotated into q_out.
 *   rows      rows of k, v, q and q_out (0: nothing to do)
 *   in_dtype  type of k, v, q and q_out: FWPKM_F32 or FWPKM_BF16 (FWPKM_F32
 *             with any cache, FWPKM_BF16 with any cache)
 *   k, v      device [rows][kv_heads][dim], row r at element r*k_stride /
 *             r*v_stride (so parts of one projection's output will do); 16-byte
 *             aligned, strides a whole number of 16 bytes
 *   q, q_out  device [rows][heads][dim] in the same form, or both NULL; q_out
 *             may be q itself (same pointer and stride), and must not overlap
 *             any input otherwise.  heads >= 1; ignored without q
 *   starts    device int32 [B+1], non-decreasing from 0, or NULL
 *   rotary    elements of a head that rotate: 0, or a multiple of 16 up to dim
 *   style     FWPKM_ROTATE_*
 *   freqs     device fp32 [rotary/2]: radians per token (NULL with rotary 0)
 *   device_errors  device word or NULL: FWPKM_CACHE_* bits are set in it when
 *             a row has no valid place.  Such a row is not stored (its query is
 *             rotated all the same where its position is not negative).
 * No two rows of a call may have the same place in the pool (two sequences
 * that share the page they write): either one's elements may remain.
 */
fwpkm_status fwpkm_cache_append(const fwpkm_cache *cache, const fwpkm_cache_batch *batch,
                                int rows, int in_dtype, const void *k, int64_t k_stride,
                                const void *v, int64_t v_stride, const void *q, int64_t q_stride,
                                void *q_out, int64_t q_out_stride, int heads,
                                const int32_t *starts, int rotary, int style, const float *freqs,
                                uint32_t *device_errors, void *stream);

/*
 * fwpkm_cache_attend -- attention of one token of each sequence.
 *   s_t = scale * (q . k_t),   lo <= t < lengths[b],
 *   out = sum_t softmax(s)_t v_t,   lse = log sum_t exp(s_t),
 * with lo = max(0, lengths[b] - window), or 0 where window is 0; query head i
 * reads cached head i / (heads / kv_heads).  A sequence without visible tokens
 * gives out = 0 and lse = -infinity, and so does a head whose visible scores are
 * all -infinity; a NaN or +infinity among a head's visible scores makes that
 * sequence's head NaN, and no other.  A NaN or an infinity among the visible
 * values leaves that element of the heads that weigh it not finite (an infinity
 * may come out as NaN), and no other.  What lies in the pool outside the visible
 * tokens does not matter, infinities and NaN included.
 *   Scores, the softmax's maximum and sum, and the sums of values are held in 32
 * bits; the last are rounded to nearest, once for every 8 to 32 tokens.  With 16-
 * and 8-bit pools a weight goes into its products with the values as two parts of
 * the tensor cores' 16-bit types, 16 bits of it for an FWPKM_BF16 pool and 22 for
 * an FWPKM_E4M3 one.  FWPKM_E4M3 pools take the queries in 16-bit floats scaled by
 * a power of two a row, exact but for elements under 2^-14 of the row's largest
 * (off by less than 2^-25 of that).  out is rounded once.  The result does not
 * depend on timing: equal calls give equal bits.
 *   heads     query heads, a multiple of kv_heads, <= 4096
 *   q         device [B][heads][dim], sequence b at element b*q_stride (a whole
 *             number of 16 bytes; 16-byte aligned); FWPKM_F32 for an F32 cache,
 *             FWPKM_BF16 for the others (FWPKM_EUNSUPPORTED otherwise)
 *   scale     finite, below 2e38 in size; usually 1/sqrt(dim).  With 0, a
 *             product that is -infinity still has no weight
 *   window    tokens visible before and including the newest, or 0: all
 *   out       device [B][heads][dim], q's type, 16-byte aligned; like lse, it
 *             overlaps no input (q least of all)
 *   lse       device fp32 [B][heads], or NULL
 *   workspace device memory of at least fwpkm_cache_attend_workspace(...)
 *             bytes, 256-byte aligned, for this call alone until it has run;
 *             its contents do not matter.  A captured graph keeps the one it
 *             was captured with, so graphs that may run at the same time need
 *             workspaces of their own.
 *   device_errors  device word or NULL, as above: a token on a bad page is
 *             left out, and a bad length is taken as the nearest valid one.
 */
fwpkm_status fwpkm_cache_attend(const fwpkm_cache *cache, const fwpkm_cache_batch *batch,
                                int heads, int q_dtype, const void *q, int64_t q_stride,
                                float scale, int window, void *out, float *lse, void *workspace,
                                int64_t workspace_bytes, uint32_t *device_errors, void *stream);

/* Bytes of workspace that fwpkm_cache_attend needs for these sizes (only
 * kv_heads, dim and dtype of the cache are looked at), or a negative
 * fwpkm_status.  Needs no device. */
int64_t fwpkm_cache_attend_workspace(const fwpkm_cache *cache, int B, int heads);

#ifdef __cplusplus
}
#endif
#endif /* FWPKM_CACHE_H_ */
