/*
 * paged_pages.h — the pages of a paged key/value cache (paged_attn.h) as requests come and go:
 * several answers that share a prompt's pages, pages handed back, and a pool closed up.
 * Compiled into librglru; the same status codes, shapes, streams and rules of ownership as
 * paged_attn.h (of paged_shape: num_seqs, num_pages, page_size and table_width; the rest is
 * ignored).
 *
 * A page may be held by several rows of the block table.  holders (int32 [num_pages]) counts a
 * page's holders beyond the first: zero for a page that is free or in one row, as paged_plan
 * leaves the pages that it takes.  Only whole pages are shared, and tokens are appended behind
 * them, so a page with more than one holder is never written.
 *
 *   paged_fork      rows that begin as copies of other rows: whole pages shared, the last,
 *                   unfinished one as a page of its own, to be copied
 *   paged_copy      copies pages in every cache (layers, keys and values, scales)
 *   paged_release   pages out of rows; those whose last holder lets go return to the ring
 *   paged_compact   the pages in use moved to the front of the pool
 *
 * All four read tables, lengths and lists from device memory and nothing from the host, so they
 * can be captured in a CUDA graph.  Numbers of rows and pages read from there are checked before
 * they address anything: one out of range is passed over.  Results do not depend on timing.
 */
#ifndef PAGED_PAGES_H
#define PAGED_PAGES_H

#include "paged_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Row children[i] becomes a copy of row parents[i], i < num_children (int32 [num_children], at
 * most 8192).  With L = kv_lens[parent] (negative: 0) and s = page_size: kv_lens_out[child] = L;
 * the first floor(L / s) entries of the parent's row are the child's too, one more holder for
 * each page; where L is no multiple of s (and the page is within the table's width) the child's
 * next entry is a page off the ring, children in order, and moves[i] = (the parent's page, the
 * child's), to be copied by paged_copy in each cache.  No page left: the entry is -1.  Else
 * moves[i] = (-1, -1).  Other entries and rows of the outputs keep their value: what the
 * children's rows held before is the caller's to release.  free_state_out = head, count and the
 * number of pages wanted and not had, as in paged_plan.  A child or parent outside the table is
 * passed over (moves[i] = (-1, -1)).
 * block_table_out, kv_lens_out, holders_out and free_state_out may be block_table, kv_lens,
 * holders and free_state.  Where block_table_out is block_table, no row is both a child and a
 * parent; else (a beam's step) any may be.  No row is a child twice. */
rglru_status paged_fork(const paged_shape *shape, int32_t num_children, const int32_t *parents,
                        const int32_t *children, const int32_t *block_table,
                        const int32_t *kv_lens, const int32_t *holders,
                        const int32_t *free_pages, const int32_t *free_state,
                        int32_t *block_table_out, int32_t *kv_lens_out, int32_t *holders_out,
                        int32_t *moves, int32_t *free_state_out, rglru_stream stream);

/* Bytes of the scratch of paged_release and paged_compact: zero before its first use (both leave
 * all of it so, and calls of other shapes may use it where it is large enough), for one stream at a
 * time.  0 for an unsupported shape. */
size_t paged_pages_workspace_bytes(const paged_shape *shape);

/* The entries [first_pages[n], end_pages[n]) of every row n of the block table (int32 [num_seqs],
 * clamped to the table) let go of their pages and become -1 in block_table_out (its other entries
 * keep their value).  With r entries that let go of page p: holders_out[p] = max(0, holders[p] -
 * r), and if r > holders[p] the page is free: free pages are appended to the ring (at (head +
 * count) % num_pages of free_pages) in ascending order.  Entries that are no page (-1) let go of
 * none.  free_state_out = {head, count + pages freed (at most num_pages), 0}.  A request that has
 * ended: [0, ceil(kv_len / page_size)); pages behind a window: [0, floor((kv_len - window + 1) /
 * page_size)), those released before among them.
 * block_table_out, holders_out and free_state_out may be block_table, holders and free_state. */
rglru_status paged_release(const paged_shape *shape, const int32_t *first_pages,
                           const int32_t *end_pages, const int32_t *block_table,
                           const int32_t *holders, int32_t *free_pages,
                           const int32_t *free_state, int32_t *block_table_out,
                           int32_t *holders_out, int32_t *free_state_out, void *workspace,
                           rglru_stream stream);

/* Closes the pool up.  In use are the pages of the entries [0, ceil(kv_lens[n] / page_size)) of
 * every row; every page that is to be kept is in one.  With U of them, the pages in use from
 * number U on, in ascending order, go to the numbers below U that are not in use, in ascending
 * order: moves (int32 [num_pages / 2][2]) lists them as (from, to), for paged_copy, then
 * (-1, -1).  block_table_out is the table with its entries in use renumbered, holders_out the
 * holders by the new numbers (0 for pages not in use), free_pages[i] = U + i for i <
 * num_pages - U, free_state_out = {0, num_pages - U, 0}: the pages from U on may then be given
 * up.  block_table_out and holders_out may be block_table and holders. */
rglru_status paged_compact(const paged_shape *shape, const int32_t *kv_lens,
                           const int32_t *block_table, const int32_t *holders,
                           int32_t *block_table_out, int32_t *holders_out, int32_t *free_pages,
                           int32_t *free_state_out, int32_t *moves, void *workspace,
                           rglru_stream stream);

/* Copies page moves[i][0] to page moves[i][1], i < num_moves (int32 [num_moves][2], at most 2^30),
 * in each of num_caches caches: page p of caches[c] is the page_bytes[c] bytes from
 * caches[c] + p * page_strides[c] on (host arrays; bytes, strides at least page_bytes).  Moves
 * with a page outside [0, num_pages) are passed over.  No page is a destination twice, or a
 * destination and a source (the moves of one paged_fork or paged_compact are so).  Up to 64
 * caches take one launch. */
rglru_status paged_copy(const paged_shape *shape, int32_t num_moves, const int32_t *moves,
                        int32_t num_caches, void *const *caches, const int64_t *page_strides,
                        const int64_t *page_bytes, rglru_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_PAGES_H */
