/*
 * libpalu — pages handed out on the device: the page tables of the paged
 * caches (paged.h, paged4.h) kept by the sequences' lengths, with the offsets,
 * positions and slots of a step's new tokens.
 *
 * Page "add TurboQuant KV cache compression" (the pull request's review:
 * prompts of different lengths, speculative rollback).  palu_draft_verify
 * leaves the lengths on the device; with this call the next step's pages
 * follow from them there, so a loop of planning, appending, attending and
 * verifying needs no word from the host, and a captured graph of it can cross
 * a page's border.
 *
 * Conventions are those of palu.h.
 */
#ifndef PALU_PAGES_H
#define PALU_PAGES_H

#include "palu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A pool of pages: plain data, filled by palu_page_pool_init().  All arrays
 * are the program's, on the device; calls read and write them on their
 * stream. */
typedef struct {
  int32_t magic;
  int32_t page_size, batch, table_width;
  int64_t n_pages;        /* entries of free_pages */
  int32_t* page_table;    /* [batch, table_width]: sequence b's first held[b] entries are its pages */
  int64_t* lengths;       /* [batch] */
  int32_t* held;          /* [batch] */
  int32_t* free_pages;    /* [n_pages]: the first *n_free are the free pages, a stack */
  int32_t* n_free;        /* [1] */
  uint32_t* error;        /* device error word, zeroed by the caller */
} palu_page_pool;

/* Describe a pool.  page_size in 1 .. 65536, batch in 1 .. 4096, table_width
 * in 1 .. 2^30 / page_size, n_pages in 0 .. 2^31 - 1; pointers aligned to
 * their elements, the arrays disjoint.  Launches nothing. */
palu_status palu_page_pool_init(palu_page_pool* pool, int32_t page_size, int64_t batch, int64_t table_width, int64_t n_pages,
                                int32_t* page_table, int64_t* lengths, int32_t* held, int32_t* free_pages, int32_t* n_free,
                                uint32_t* error);

/* One step's plan.  Sequence b brings new_tokens[b] >= 0 tokens:
 *   lengths[b] += new_tokens[b];
 *   need = ceil(lengths[b] / page_size), but not less than the first
 *     shared_pages of the entries that it holds (pages shared with others are
 *     not given back here);
 *   entries need .. held[b]-1 of its row go back: pushed on the free stack in
 *     this order, sequence by sequence;
 *   entries held[b] .. need-1 are taken in this order, sequence by sequence,
 *     each the top of the stack, after all that go back;
 *   held[b] = need.
 * What the entries behind held[b] contain is left as it was.  So lengths that
 * were set back (rejected drafts) return their pages at the next call, and a
 * sequence is ended by a length of 0 (and a new one begun in its place).
 *   offsets   device int32 [batch + 1]: the exclusive sums of new_tokens, as
 *             the caches' calls take them;
 *   positions device int64 [tokens]: row offsets[b] + i is token
 *             lengths[b] - new_tokens[b] + i; -1 at and behind offsets[batch];
 *   slots     device int64 [tokens]: page * page_size + place in the page of
 *             that token; -1 likewise.  positions and slots may be NULL.
 *   new_tokens device int32 [batch], not overlapping what is written.
 * The call is refused as a whole, with a bit of the error word, where the free
 * pages do not suffice or a length would pass the table (PALU_DEVERR_CAPACITY),
 * or a count or length is negative, the counts' sum is above `tokens`, or
 * held or n_free is outside its array (PALU_DEVERR_SPAN): then nothing of the
 * pool changes, offsets are all 0 (the caches' calls touch no rows) and
 * positions and slots all -1.
 * All results are whole numbers and follow from the arguments alone.  One
 * kernel launch.  tokens in 0 .. 2^31 - 1. */
palu_status palu_page_plan(const palu_page_pool* pool, const int32_t* new_tokens, int64_t tokens, int32_t shared_pages,
                           int32_t* offsets, int64_t* positions, int64_t* slots, void* stream);

/* Synchronise `stream`, report and clear the device error word
 * (PALU_ERR_DEVICE with the bits in *device_error if not NULL). */
palu_status palu_page_pool_sync(const palu_page_pool* pool, uint32_t* device_error, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PALU_PAGES_H */
