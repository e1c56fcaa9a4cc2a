/*
 * libpalu — the serving step around a paged key/value cache: queries and keys
 * normalised per head and rotated by position, new tokens appended to pages,
 * and attention of the new tokens over the pages, with a prefix that the
 * whole batch shares read once.
 *
 * Beside the compressed caches of palu.h, kivi.h and svdq.h this is the
 * uncompressed cache of a serving loop (page "add TurboQuant KV cache
 * compression", the pull request's description and review: prompts of
 * different lengths in one batch, a prompt prefix used by many requests,
 * speculative tokens that are rolled back).  A sequence's tokens lie in pages
 * of a pool; the host program hands pages out and keeps, in device memory, a
 * page table and the sequences' lengths.  The calls only read those two, so
 * rolling back rejected tokens, or giving a sequence another page, is a write
 * to them and nothing else, and a captured graph follows them when replayed.
 *
 * Conventions are those of palu.h (status codes, palu_last_error(), caller-
 * owned device memory, asynchronous calls on `stream`, argument errors
 * reported before anything is launched).  What only the device can see sets
 * bits of a device error word, reported by palu_paged_sync():
 * PALU_DEVERR_CAPACITY, PALU_DEVERR_PAGE, PALU_DEVERR_SPAN,
 * PALU_DEVERR_POSITION, PALU_DEVERR_TIMEOUT.  Such a condition never makes a
 * call access memory outside the buffers it was given.
 *
 * Supported: head_dim 128; fp16 or bf16, the same type for queries, keys,
 * values and pages; pages of 16, 32, 64 or 128 tokens; up to 64 query heads
 * per KV head; up to 4096 sequences a call.
 */
#ifndef PALU_PAGED_H
#define PALU_PAGED_H

#include "palu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the calls below. */
enum { PALU_TYPE_F16 = 0, PALU_TYPE_BF16 = 1 };

/* What happens to a head's row x of queries or keys before it is used:
 *   x <- x / sqrt(mean(x^2) + eps) * weight     (where a weight is given)
 *   (x_i, x_j) <- (x_i cos a - x_j sin a, x_j cos a + x_i sin a)
 *                                                (where a table is given)
 * for the rope_dim/2 pairs (i, j) = (n, n + rope_dim/2), or (2n, 2n + 1) when
 * interleaved; channels from rope_dim on are not rotated.  All in fp32, with
 * one rounding to the element type at the end. */
typedef struct {
  const void* q_weight;      /* device [128] of the call's type, 16-byte aligned; NULL: no norm of the queries */
  const void* k_weight;      /* the same for the keys */
  const float* cos_sin;      /* device fp32 [n_positions, rope_dim], 16-byte aligned: a position's rope_dim/2
                                cosines, then its sines; NULL: no rotation */
  int64_t n_positions;
  int32_t rope_dim;          /* a multiple of 16, 16 .. 128 */
  int32_t interleaved;
  float eps;                 /* >= 0 */
  int32_t pad0;
} palu_qk_transform;

/* Normalise and rotate queries and keys, token-major rows of a projection in,
 * head-major tensors out: the layout palu_fit, palu_encode_append,
 * palu_decode_attn and the comparators take.
 *   q, k   device [batch, tokens, heads, 128] with strides (in elements) of
 *          batch, token and head; channels are contiguous, pointers 16-byte
 *          aligned and strides multiples of 8.  Views of one fused projection
 *          are fine.
 *   positions  device int64 [batch, tokens] (read only where there is a
 *          table; may be NULL without one).
 *   q_out  device [batch, q_heads, tokens, 128], k_out the same with
 *          kv_heads; contiguous, 16-byte aligned, overlapping neither the
 *          inputs nor each other.
 *   error  device uint32 (may be NULL): PALU_DEVERR_POSITION is set when a
 *          position lies outside the table; that token's rows become NaN.
 * One kernel launch. */
palu_status palu_qk_norm_rope(const palu_qk_transform* transform, int32_t dtype, int64_t batch, int64_t tokens,
                              int32_t q_heads, int32_t kv_heads, const void* q, const int64_t q_strides[3],
                              const void* k, const int64_t k_strides[3], const int64_t* positions, void* q_out,
                              void* k_out, uint32_t* error, void* stream);

/* A paged cache: plain data, filled by palu_paged_cache_init().  Token t of
 * sequence b lies in row t % page_size of page page_table[b, t / page_size]. */
typedef struct {
  int32_t magic;
  int32_t dtype, kv_heads, page_size;
  int32_t batch, table_width;  /* sequences; page-table entries a sequence */
  int64_t n_pages;
  void *k_pages, *v_pages;
  int64_t k_strides[3], v_strides[3]; /* page, head, token strides in elements */
  const int32_t* page_table;   /* device [batch, table_width] */
  const int64_t* lengths;      /* device [batch] */
  uint32_t* error;             /* device error word */
} palu_paged_cache;

/* Describe a cache on caller-owned device buffers.  Launches nothing.
 *   k_pages, v_pages  device pools, 16-byte aligned; strides [page, head,
 *            token] in elements, positive multiples of 8 (token-major and
 *            head-major pages, and pools that interleave keys and values, are
 *            all given by their strides).
 *   page_table  device int32 [batch, table_width] and lengths device int64
 *            [batch]: the host program's, read by every call on its stream.
 *            A row's entries behind its length are never read (but for
 *            those that an attention call names as shared).
 *   error    device uint32, zeroed by the caller. */
palu_status palu_paged_cache_init(palu_paged_cache* cache, int32_t dtype, int32_t kv_heads, int32_t page_size,
                                  int64_t n_pages, void* k_pages, const int64_t k_strides[3], void* v_pages,
                                  const int64_t v_strides[3], const int32_t* page_table, int64_t batch,
                                  int64_t table_width, const int64_t* lengths, uint32_t* error);

/* Append new tokens: sequence b brings rows offsets[b] .. offsets[b+1]-1 of
 * q, k and v, n_b of them, and lengths[b] already counts them, so they become
 * its tokens lengths[b] - n_b .. lengths[b] - 1.  Keys (and queries) go
 * through the transform; values are copied.  Repeating a call writes the same
 * values to the same places.
 *   offsets  device int32 [batch + 1], from 0 on, non-decreasing; rows at and behind
 *          offsets[batch] (a batch padded for a captured graph) are not
 *          touched.  n_b may be 0.
 *   q      device [tokens, q_heads, 128], strides token and head, or NULL
 *          (then q_out is NULL and q_heads 0); k and v device
 *          [tokens, kv_heads, 128]; alignment as in palu_qk_norm_rope.  None
 *          of them may lie in the rows of the pages that the call writes.
 *   positions  device int64 [tokens], the positions of the rotation; NULL:
 *          each token's place in its sequence.
 *   q_out  device [tokens, q_heads, 128] contiguous, not overlapping q, k or v.
 * Refused on the device, with a bit of the error word (the tokens are not
 * appended and their q_out rows are NaN): a sequence whose length passes
 * table_width * page_size (CAPACITY), is less than n_b, or whose offsets are
 * out of order (SPAN); a page id outside the pool (PAGE); a position outside
 * the table (POSITION).  One kernel launch. */
palu_status palu_paged_append(const palu_paged_cache* cache, const palu_qk_transform* transform, int64_t tokens,
                              const int32_t* offsets, int32_t q_heads, const void* q, const int64_t q_strides[2],
                              const void* k, const int64_t k_strides[2], const void* v, const int64_t v_strides[2],
                              const int64_t* positions, void* q_out, void* stream);

/* Device workspace of palu_paged_attn (16-byte aligned; no initial contents
 * are needed, calls that share one must not overlap on the GPU).  It also
 * serves fewer tokens, a smaller max_new and any other number of shared pages
 * (one sized for shared_pages 0 serves 0 only). */
palu_status palu_paged_attn_workspace_size(const palu_paged_cache* cache, int64_t tokens, int32_t q_heads,
                                           int32_t max_new, int32_t shared_pages, size_t* bytes);

/* Attention of the batch's new tokens over the cache (which already holds
 * their keys and values): the query of sequence b's token at place t attends
 * to the tokens 0 .. t of its sequence.
 *   out = softmax(softmax_scale q K^T) V
 *   q      device [tokens, q_heads, 128], strides token and head; query head
 *          h reads KV head h / (q_heads / kv_heads).  Row r belongs to the
 *          sequence with offsets[b] <= r < offsets[b+1], as in
 *          palu_paged_append; each sequence has at most max_new rows.
 *   shared_pages  leading page-table entries that are the same pages in every
 *          row of the table.  Where that is faster (by the sizes given here)
 *          their keys and values are read once for the whole batch, from row
 *          0 of the table, whatever the length of sequence 0, as far as the
 *          longest sequence with new rows goes.  0: nothing is shared.  The
 *          result does not depend on it beyond rounding.
 *   out    device [tokens, q_heads, 128], contiguous, the cache's type, not
 *          overlapping q; rows at and behind offsets[batch] are not touched.
 *   softmax_scale 0 selects 1/sqrt(128).
 * A row that sees no token (a length of 0, or less than n_b) gets zeros.
 * What the pages hold behind a sequence's length does not matter, NaN and
 * infinities included; the values of its own tokens have to be finite (a
 * token that a query does not see yet has the weight 0, and 0 * NaN is NaN).
 * Weights are rounded to the cache's type once, where a KV head has more than
 * 16 rows (in fp16 those under 2^-20 of a row's largest lose bits, and those
 * under 2^-31 count only in the sum); sums, maxima and accumulators are fp32.
 * Two kernel launches on `stream`, chosen by the sizes given here, not by the
 * lengths; how the SMs are divided follows from the lengths, not from the
 * table's width.  Repeating a call repeats its result bit for bit.
 * A sequence with more than max_new rows or offsets out of order sets
 * PALU_DEVERR_SPAN and its rows are zeros, as are rows before offsets[0] where
 * that is not 0; a length past the table sets PALU_DEVERR_CAPACITY and is cut
 * to it; a page id outside the pool sets PALU_DEVERR_PAGE and page 0 is read
 * for it. */
palu_status palu_paged_attn(const palu_paged_cache* cache, int64_t tokens, const int32_t* offsets, int32_t max_new,
                            int32_t q_heads, const void* q, const int64_t q_strides[2], int32_t shared_pages,
                            float softmax_scale, void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Synchronise `stream`, report and clear the device error word
 * (PALU_ERR_DEVICE with the bits in *device_error if not NULL). */
palu_status palu_paged_sync(const palu_paged_cache* cache, uint32_t* device_error, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PALU_PAGED_H */
