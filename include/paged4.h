/*
 * libpalu — the paged cache of paged.h held in 4 bits: keys and values as
 * 4-bit codes with an fp16 scale and zero for every 32 channels of a token,
 * 160 bytes a token and KV head where fp16 pages take 512.
 *
 * Page "add TurboQuant KV cache compression" (the pull request's description
 * and review) asks for a compressed cache that follows prompts of different
 * lengths, a shared prefix and speculative rollback; the quantizer is that of
 * the blog post "VeloxQuant-MLX 0.8.0 adds KIVI", "What KIVI is", on groups of
 * 32 channels of one token, so that a token is complete when it is appended
 * and can be rolled back: no residual window, no calibration.
 *
 * Page table, lengths, offsets, shared pages, the transform, the error word
 * and the conventions are those of paged.h; tables, lengths and the calls'
 * arguments can be moved between the two caches as they are.
 *
 * Supported: head_dim 128; fp16 or bf16 for queries, keys, values and outputs;
 * pages of 16, 32, 64 or 128 tokens; up to 64 query heads per KV head; up to
 * 4096 sequences a call.
 */
#ifndef PALU_PAGED4_H
#define PALU_PAGED4_H

#include "paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What is held of 32 channels x of one token and KV head, in fp32 without
 * fused operations, ties to even, with min x and max x cut to +-65504:
 *   z = fp16(min x), s = fp16((max x - min x) / 15), the next smaller number
 *   where z + 15 s would pass 65504,
 *   c = min(max(rint((x - z) / s), 0), 15), or 0 where s is 0,
 * and reads back as z + s c.  Channels of which one is not finite all read
 * back as NaN.
 *
 * A page of one KV head is page_size / 16 blocks of PALU_PAGED4_BLOCK bytes,
 * each 16 tokens; block bytes
 *      0 .. 1023  key codes     [token][c 4][group 4] little-endian words: the
 *                               word's nibble n is channel 8 c + 2 n (n < 4) or
 *                               8 c + 2 n - 7 (n >= 4) of the group
 *   1024 .. 1279  key scales    [token][s, z][group 4] fp16
 *   1280 .. 2303  value codes   [half 2][g 8][c 4][m 4] words of the channels
 *                               64 half + 16 m + g (low nibbles) and + 8 (high
 *                               nibbles); byte b is token 2 c + (b >> 1) + 8 (b & 1)
 *   2304 .. 2559  value scales  [s, z][c 4][e 2][group 4][odd 2] fp16, token
 *                               8 e + 2 c + odd
 * which is the order in which the attention's lanes take them. */
#define PALU_PAGED4_BLOCK 2560

/* A 4-bit paged cache: plain data, filled by palu_paged4_cache_init(). */
typedef struct {
  int32_t magic;
  int32_t dtype, kv_heads, page_size;
  int32_t batch, table_width;  /* sequences; page-table entries a sequence */
  int64_t n_pages;
  void* pages;
  int64_t strides[2];          /* page, head strides in bytes */
  const int32_t* page_table;   /* device [batch, table_width] */
  const int64_t* lengths;      /* device [batch] */
  uint32_t* error;             /* device error word */
} palu_paged4_cache;

/* Describe a cache on caller-owned device buffers.  Launches nothing.
 *   pages    device pool, 16-byte aligned: page p of head h at
 *            pages + p * strides[0] + h * strides[1], contiguous there;
 *            strides positive multiples of 16 bytes.  No initial contents are
 *            needed.
 *   dtype    of the queries, keys, values and outputs.
 * The others as in palu_paged_cache_init. */
palu_status palu_paged4_cache_init(palu_paged4_cache* cache, int32_t dtype, int32_t kv_heads, int32_t page_size,
                                   int64_t n_pages, void* pages, const int64_t strides[2], const int32_t* page_table,
                                   int64_t batch, int64_t table_width, const int64_t* lengths, uint32_t* error);

/* Append new tokens, as palu_paged_append does: the codes are those of the
 * rows that it would store (the transformed keys rounded to the cache's type,
 * the values as they are).  Repeating a call writes the same bytes.  Only the
 * new tokens' bytes are written.  None of q, k and v may lie in the pages that
 * the call writes.  Refused on the device as there; a token whose position is
 * outside the table is not appended, the others of its sequence are.  One
 * kernel launch. */
palu_status palu_paged4_append(const palu_paged4_cache* cache, const palu_qk_transform* transform, int64_t tokens,
                               const int32_t* offsets, int32_t q_heads, const void* q, const int64_t q_strides[2],
                               const void* k, const int64_t k_strides[2], const void* v, const int64_t v_strides[2],
                               const int64_t* positions, void* q_out, void* stream);

/* Read tokens back: rows offsets[b] .. offsets[b+1]-1 of the outputs are n_b
 * tokens of sequence b, from place starts[b] on, or its last n_b where starts
 * is NULL, as z + s c rounded once to the cache's type.
 *   starts device int64 [batch] or NULL.
 *   k_out, v_out  device [tokens, kv_heads, 128], contiguous, 16-byte aligned,
 *          not overlapping each other or the pages; rows at and behind
 *          offsets[batch], and before offsets[0], are not touched.
 * A sequence whose offsets are out of order or outside the rows, or whose
 * tokens are not all in 0 .. lengths[b] - 1, sets PALU_DEVERR_SPAN, one whose
 * length passes the table PALU_DEVERR_CAPACITY: nothing is read of either.  A
 * page id outside the pool sets PALU_DEVERR_PAGE; the rows of its tokens are
 * not touched.  One kernel launch. */
palu_status palu_paged4_read(const palu_paged4_cache* cache, int64_t tokens, const int32_t* offsets, const int64_t* starts,
                             void* k_out, void* v_out, void* stream);

/* Device workspace of palu_paged4_attn, as palu_paged_attn_workspace_size. */
palu_status palu_paged4_attn_workspace_size(const palu_paged4_cache* cache, int64_t tokens, int32_t q_heads,
                                            int32_t max_new, int32_t shared_pages, size_t* bytes);

/* Attention of the batch's new tokens over the cache: palu_paged_attn with the
 * keys and values z + s c.  Arguments, rows without a token, shared pages,
 * refusals and repeated results as there.  Bytes behind a sequence's length do
 * not matter.
 * What is rounded follows from the rows that attend to the same keys through a
 * KV head, by the sizes given here: for a sequence's own keys min(max_new, tokens)
 * times q_heads / kv_heads, for shared keys that are read once those of all tokens.
 * Up to 16 of them the codes enter the products as they are, and the scales in
 * fp32 (keys) or with the weights (values): a weight is rounded to fp16 (those
 * under 2^-20 of a row's largest lose bits, those under 2^-31 are lost), and so is
 * its product with the scale, in units that follow the largest scale of each 16
 * tokens and 32 channels (products under 2^-17 of the largest weight's with that
 * scale lose bits, as do scales under 2^-11 of it; scales under 2^-18 have the units
 * of 2^-18).
 * With more rows keys, values and weights are each rounded once to fp16 (weights
 * under 2^-20 of a row's largest lose bits, those under 2^-31 count only in the sum),
 * in bf16 caches too.  Sums, maxima and accumulators are fp32; queries lose nothing
 * but what lies 2^-24 under a row's largest. */
palu_status palu_paged4_attn(const palu_paged4_cache* cache, int64_t tokens, const int32_t* offsets, int32_t max_new,
                             int32_t q_heads, const void* q, const int64_t q_strides[2], int32_t shared_pages,
                             float softmax_scale, void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Synchronise `stream`, report and clear the device error word
 * (PALU_ERR_DEVICE with the bits in *device_error if not NULL). */
palu_status palu_paged4_sync(const palu_paged4_cache* cache, uint32_t* device_error, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PALU_PAGED4_H */
