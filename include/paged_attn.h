/*
 * paged_attn.h — a paged key/value cache and the attention that reads it, on one NVIDIA GB300
 * (sm_103a): the attention layers that hybrid recurrent models alternate with the recurrent
 * layer of librglru.h (windowed, grouped or multi-query heads), in their serving form.
 * Compiled into librglru; the same status codes, dtypes and stream conventions as librglru.h.
 *
 * The cache.  Keys and values live in num_pages pages of page_size token slots each; slot
 * s = page * page_size + offset.  Request n owns the pages of row n of the block table
 * (int32 [num_seqs][table_width]): its token at position p is in page table[n][p / page_size]
 * at offset p % page_size.  One step appends new tokens to some or all requests:
 *
 *   paged_plan       from the request lengths: the offsets of the packed new tokens, the pages
 *                    they need (taken from a ring of free pages), their slots and positions
 *   paged_kv_write   per attention layer: the new keys and values into their slots
 *   paged_attention  per attention layer: the new tokens' queries over the cache
 *
 * All three read lengths and tables from device memory and nothing from the host, so a step
 * can be captured once in a CUDA graph and replayed with other lengths.
 *
 * Conventions for every call:
 *   - Packing: the new tokens of all requests lie one after another in rows of `tokens` tokens;
 *     request n's are [cu_seqlens[n], cu_seqlens[n + 1]).  Rows past cu_seqlens[num_seqs] are
 *     padding.  A request may have no new token.
 *   - Supported: page_size a power of two from 8 to 4096; 1 <= num_seqs <= 8192;
 *     num_pages * page_size < 2^31; num_seqs * table_width < 2^31; tokens <= 2^30; for
 *     paged_kv_write and paged_attention 8 <= D <= 256 with D * sizeof(io) a multiple of 16
 *     bytes, and for paged_attention Hq a multiple of Hkv with Hq / Hkv <= 64; else
 *     RGLRU_ERR_UNSUPPORTED (RGLRU_ERR_INVALID_ARG where a size has no meaning).  Pointers to
 *     q, k, v, o and the caches are 16-byte aligned and their strides positive multiples of 16
 *     bytes; the other arrays are aligned to their element.
 *   - Values read from device memory are never trusted with an address: lengths and offsets
 *     out of range are clamped, a slot outside the cache is skipped, a table entry outside the
 *     cache (or past table_width) reads as zero keys and values.  Such input gives wrong
 *     results, never an out-of-bounds access.
 *   - Ownership: the caller allocates every buffer; the library never allocates or
 *     synchronises.  All work is enqueued on `stream`, launched with programmatic stream
 *     serialisation (set-up may overlap the end of the kernel before it on the stream; memory
 *     is touched only after that kernel has completed).  Argument checks run on the host before
 *     any launch; launch failures return RGLRU_ERR_CUDA.
 */
#ifndef PAGED_ATTN_H
#define PAGED_ATTN_H

#include <stddef.h>
#include <stdint.h>

#include "librglru.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t num_seqs;    /* requests (rows of the block table) */
  int32_t tokens;      /* rows of the packed new tokens */
  int32_t Hq, Hkv, D;  /* query heads, key/value heads, head width (paged_plan ignores them) */
  int32_t num_pages, page_size, table_width;
  rglru_dtype io;      /* storage type of q, k, v, o and of the caches (paged_plan ignores it) */
  int32_t window;      /* keys a token sees, its own included; 0: all before it */
} paged_shape;

/* Strides in elements; the head width D is always contiguous.  paged_kv_write reads the k, v
 * and cache strides, paged_attention the q, o and cache strides. */
typedef struct {
  int64_t q_token, q_head, o_token, o_head;
  int64_t k_token, k_head, v_token, v_head;
  int64_t kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
} paged_strides;

/* Plans one step.  With c = cached_lens[n] tokens in the cache and q = new_lens[n] to append
 * (both int32 [num_seqs], negative values count as 0) and s = page_size:
 *   cu_seqlens [num_seqs + 1] = running sum of q from 0;   kv_lens[n] = c + q;
 *   the request holds ceil(c / s) pages and needs ceil((c + q) / s), at most table_width: the
 *   difference comes off the ring of free pages, requests in order, each request's pages in
 *   order, into block_table[n][ceil(c / s)] onwards (other entries keep their value);
 *   token i of request n, row t = cu_seqlens[n] + i: positions[t] = c + i and
 *   slots[t] = block_table[n][positions[t] / s] * s + positions[t] % s.
 * free_pages is the ring, int32 [num_pages]; free_state = {head, count, -} (int32 [3]): the
 * free pages are free_pages[(head + i) % num_pages], i < count.  free_state_out receives the
 * head and count after the step and the number of pages that were wanted and not had (no free
 * page left, or past table_width); pages not had are written as -1, tokens without a page get
 * slot -1, as do padding rows (their position is 0).  Pages go back to the ring by paged_release
 * (paged_pages.h), or by the caller's own means: at (head + count) % num_pages, with count raised.
 * A table entry whose page lies wholly before every later query's window is not read again, so its
 * page may be returned early.
 * kv_lens may be cached_lens and free_state_out free_state (updated in place); no other
 * arrays may overlap. */
rglru_status paged_plan(const paged_shape *shape, const int32_t *cached_lens,
                        const int32_t *new_lens, const int32_t *free_pages,
                        const int32_t *free_state, int32_t *block_table, int32_t *cu_seqlens,
                        int32_t *kv_lens, int32_t *positions, int64_t *slots,
                        int32_t *free_state_out, rglru_stream stream);

/* Copies row t of k and v ([tokens][Hkv][D] by strides) into slot slots[t] of the caches
 * ([num_pages][page_size][Hkv][D] by strides), t < tokens.  Slots outside
 * [0, num_pages * page_size) are skipped.  Slots must differ from one another (two rows with
 * one slot leave a mixture of both there).  strides NULL: everything contiguous. */
rglru_status paged_kv_write(const paged_shape *shape, const paged_strides *strides,
                            const void *k, const void *v, const int64_t *slots, void *k_cache,
                            void *v_cache, rglru_stream stream);

/* Bytes of paged_attention's scratch (sized for the current device; partial results of rows
 * whose keys are split over several SMs).  It must be zero before its first use
 * (paged_attention leaves what it needs zero as zero) and serve one stream at a time.  0 for
 * an unsupported shape. */
size_t paged_attention_workspace_bytes(const paged_shape *shape);

/* Attention of the new tokens over the cache.  Token i of request n has position
 * p = kv_lens[n] - q_n + i (q_n its number of new tokens: the keys and values of the new
 * tokens themselves are already in the cache) and sees the positions
 *   J = { j : max(0, p - window + 1) <= j <= p }  (window 0: from 0);
 * query head h reads key/value head h / (Hq / Hkv):
 *   s_j = scale q.k_j,  lse = ln sum_J exp(s_j),  o = sum_J exp(s_j - lse) v_j.
 * A token that sees nothing (p < 0: kv_lens[n] < q_n) gets o = 0 and lse = -inf.  Padding rows
 * of o and lse are not written.  o [tokens][Hq][D] by strides in shape.io; lse float32
 * [tokens][Hq], may be NULL; scale > 0 with scale log2(e) finite, and scores are held times
 * log2(e) (so up to 2.3e38).  Whatever the cache holds at positions that no new token sees (past
 * kv_lens, before every window, other requests' pages) has no effect, NaN and infinities
 * included; a NaN or infinity at a position that some new token of a request sees may reach
 * other new tokens of that request.  Scores, softmax and sums are held in float32; with bf16 the
 * weights exp(s_j - max) are rounded to bf16 before they meet v.
 * strides NULL: everything contiguous.  The result does not depend on timing (sums in a fixed
 * order).  A device wait that runs out marks the workspace (rglru_sync_status gives
 * RGLRU_ERR_TIMEOUT); zero it before using it again.  Tests bring that about with
 * rglru_debug_lookback(polls, cta): that CTA of a tensor-core call gets no work and its waits
 * are limited to polls x 100 ns. */
rglru_status paged_attention(const paged_shape *shape, const paged_strides *strides,
                             const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *block_table, const int32_t *cu_seqlens,
                             const int32_t *kv_lens, float scale, void *o, float *lse,
                             void *workspace, rglru_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_ATTN_H */
