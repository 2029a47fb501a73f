/*
 * kv_pages.h -- C ABI of the paged cache's bookkeeping on the GPU (libattn.so): block table, slot
 * map and positions of one step from the requests' lengths and the pool of free pages.
 *
 * A pool is a ring of page numbers, device int32[num_pages], and its state, device int32[2] = {first,
 * count}: the free pages are ring[(first + i) % num_pages], i < count. A block table is that of
 * attn.h: position p of sequence s lies in page block_table[s * table_stride + p / page_size].
 *
 * Ownership, threading and errors are those of rope_qk.h. Any contents of the arrays are memory-safe.
 */
#ifndef KV_PAGES_H
#define KV_PAGES_H

#include <stdint.h>

#include "rope_qk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One step: sequence s holds held[s] tokens and gets new_lens[s] more, rows cu_seqlens[s] ..
 * cu_seqlens[s+1] - 1 of the step's T rows (the running sum of new_lens, at most T). The pages that
 * they need beyond the ceil(held[s] / page_size) that it has are taken from the pool in the order
 * of the sequences, and written to the table behind those.
 *
 * A sequence with new tokens is refused, and its row of the table left as it is, where it would
 * need more than max_pages pages or hold 2^31 - 4096 tokens or more (it asks for no page then), where
 * the pages asked for up to it are more than are free, and where its tokens do not all lie in the T
 * rows. One that needs no page is not refused for want of them.
 *  new_lens, held   device int32[num_seqs], read; a negative number counts as 0
 *  T                0 .. 2^30; num_seqs 0 .. 2^24; num_pages 1 .. 2^30; page_size 1 .. 2^30
 *  ring, state      the pool, read: it stays as it is, for the caller to take state_out over or not
 *  block_table      device, only the new entries are written
 *  cu_seqlens       device int32[num_seqs + 1], written
 *  kv_lens          device int32[num_seqs], written: what each sequence holds in this step's calls
 *                   (kv_append, paged_plan), 0 for one that is refused, so that none of its tokens
 *                   has a position there
 *  held_out         device int32[num_seqs], written: what each sequence holds afterwards (held[s] for
 *                   one that is refused)
 *  positions        device int32[T], written: of each row, -1 for rows of no sequence or a refused one
 *  slots            device int64[T], written: page * page_size + position % page_size, as
 *                   kv_append_slots of rope_axes.h takes it; -1 also where the page is negative
 *  state_out        device int32[2], written
 * An output, the table among them, that overlaps an input or another output is refused. One launch. */
int32_t kv_page_step(const int32_t* new_lens, const int32_t* held, int32_t num_seqs, int64_t T,
                     int32_t page_size, int32_t* block_table, int32_t max_pages, int64_t table_stride,
                     const int32_t* ring, int32_t num_pages, const int32_t* state, int32_t* cu_seqlens,
                     int32_t* kv_lens, int32_t* held_out, int32_t* positions, int64_t* slots,
                     int32_t* state_out, void* stream);

/* Gives the pages of sequences back to the pool, in place: of those with gone[s] not 0 the first
 * ceil(held[s] / page_size) (at most max_pages) entries of their rows go behind the ring's last, and
 * held[s] becomes 0. What the ring has no room for is dropped (no page is free twice, so none should).
 * The table stays as it is. One launch of one workgroup.
 *  gone   device uint8[num_seqs] */
int32_t kv_page_release(int32_t* held, const uint8_t* gone, int32_t num_seqs, int32_t page_size,
                        const int32_t* block_table, int32_t max_pages, int64_t table_stride, int32_t* ring,
                        int32_t num_pages, int32_t* state, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KV_PAGES_H */
