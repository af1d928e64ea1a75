/*
 * paged_q4.h — the paged key/value cache (paged_attn.h) held in 4 bits a value: its write, its
 * read, and the attention over it.  Compiled into librglru; the same status codes, shapes,
 * block tables, lengths, streams and rules as paged_attn.h (paged_plan and the calls of
 * paged_pages.h serve both caches).
 *
 * A value is held as a code of 4 bits (E2M1) times a scale of 8 bits (E4M3) that 16 neighbouring
 * channels of a token's head share.  With a = max |x| over the 16:
 *   scale s = the E4M3 number nearest to a / 6 (ties to even), at least 2^-9, at most 448;
 *   code    = the number nearest to x / s among 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives,
 *             ties to the even code (0, 1, 2, 4).
 * So a value is off by at most (1 + 1/16) a / 6 while a lies between 6 * 2^-6 (0.094) and 6 * 448 =
 * 2688; above that it is cut off.  Below, where scales have fewer bits and then end, by at most
 * a / 6 + 2^-10, or 3 * 2^-9 where that is more: a value of a hundredth is held roughly, a group with
 * a <= 2^-11 as zeros.  No factor of a head or tensor is held: a caller whose keys or values are so
 * small multiplies them before the write (and divides paged_q4_attention's scale, or o).
 * Where one of the 16 is not finite the scale is NaN, and all 16 read as NaN.  A value has 6
 * significant bits at most: reading it in bf16 or float32 is exact.
 *
 * Arrays.  Codes: [num_pages][page_size][Hkv][D / 2] bytes, channel 2 i in the low half of byte i;
 * scales: [num_pages][page_size][Hkv][D / 16] bytes; each by strides of pages, tokens and heads.
 * Codes lie on 16 bytes and scales on 4 bytes (base and strides); strides of pages and tokens are
 * below 2^32 bytes.  Head by head (a head's tokens of a page next to one another) is the layout that
 * reads fastest: its copies are of whole lines.
 *
 * Supported: what paged_attention supports, with 16 <= D <= 256 a multiple of 16; else
 * RGLRU_ERR_UNSUPPORTED.  shape.io is the type of q, k, v and o (bf16 or float32).
 */
#ifndef PAGED_Q4_H
#define PAGED_Q4_H

#include "paged_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Strides of q, o, k and v in elements (D contiguous), of codes and scales in bytes.
 * paged_q4_write and paged_q4_read use those of k, v and the caches, paged_q4_attention those of
 * q, o and the caches. */
typedef struct {
  int64_t q_token, q_head, o_token, o_head;
  int64_t k_token, k_head, v_token, v_head;
  int64_t kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
  int64_t ks_page, ks_token, ks_head, vs_page, vs_token, vs_head;
} paged_q4_strides;

/* Row t of k and v ([tokens][Hkv][D] by strides) into slot slots[t] of the caches, t < tokens, as
 * codes and scales.  Slots outside [0, num_pages * page_size) are skipped; slots must differ from
 * one another.  strides NULL: k and v contiguous, the caches head by head
 * ([num_pages][Hkv][page_size] rows, rows of codes padded to 16 bytes, of scales to 4). */
rglru_status paged_q4_write(const paged_shape *shape, const paged_q4_strides *strides,
                            const void *k, const void *v, const int64_t *slots, void *k_codes,
                            void *k_scales, void *v_codes, void *v_scales, rglru_stream stream);

/* The reverse: row t of k and v receives what slot slots[t] of the caches stands for (a copy of a
 * prefix into a wider cache, a check).  Slots may repeat; rows whose slot is outside the cache
 * become zero. */
rglru_status paged_q4_read(const paged_shape *shape, const paged_q4_strides *strides,
                           const int64_t *slots, const void *k_codes, const void *k_scales,
                           const void *v_codes, const void *v_scales, void *k, void *v,
                           rglru_stream stream);

/* Bytes of paged_q4_attention's scratch; as paged_attention_workspace_bytes (zero before its first
 * use, one stream at a time).  0 for an unsupported shape. */
size_t paged_q4_attention_workspace_bytes(const paged_shape *shape);

/* paged_attention over what the caches stand for: the same formulas, rows that see nothing,
 * padding, lengths and table entries out of range, the same rules on what has no effect and on
 * waits that run out.
 * Numerics: keys and values enter the products exactly.  Queries enter as f16, each row times a
 * power of two: exact for bf16 but for elements below 2^-29 of their row's largest; float32 ones as
 * a sum of two (off by 2^-22 of themselves, or 2^-39 of their row's largest where that is more).
 * Weights enter as f16, off by 2^-11 of themselves, or 2^-32 of the row's largest where that is more
 * (2^-36 where requests have up to 16 rows of queries, Hq / Hkv a token, in the mean); float32 ones as
 * a sum of two (2^-22, or 2^-36 of the row's largest).  Scores, softmax and sums are held in float32.
 * The tensor core cuts its sums to 24 bits where others round: with float32 these are sums over up to
 * 256 keys, added up with rounding; with bf16 over all the keys of a request that one SM takes (below
 * 3e-9 of the output a key: 2e-4 for 65536 keys, where bf16's rounding is up to 2e-3). */
rglru_status paged_q4_attention(const paged_shape *shape, const paged_q4_strides *strides,
                                const void *q, const void *k_codes, const void *k_scales,
                                const void *v_codes, const void *v_scales,
                                const int32_t *block_table, const int32_t *cu_seqlens,
                                const int32_t *kv_lens, float scale, void *o, float *lse,
                                void *workspace, rglru_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_Q4_H */
