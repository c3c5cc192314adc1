/*
 * latent_attention.h -- C ABI of the MI355X (gfx950) paged latent cache and of
 * latent attention over it: the step behind the top-k + page-table transform
 * (topk_transform.h), whose slots latent_attention reads, and the step before
 * it that builds the page table.
 *
 * Latent attention keeps, for every token, one latent vector c of
 * LATENT_DIM values and one rotary key r of LATENT_ROPE_DIM values, shared by
 * all heads.  A head's key is [Wk c | r] and its value Wv c.
 *   expanded form: keys and values are multiplied out by the caller's
 *     projection, and attention runs on them head by head;
 *   absorbed form: Wk is folded into the query (q Wk, LATENT_DIM wide) and Wv
 *     into the output projection, so attention runs on c itself: every head
 *     reads the same rows, and nothing is expanded.
 *
 * Cache.  A slot is one token's place: latent row, rotary row and, for 8-bit
 * caches, one scale.  The arrays may be views with a row stride (in
 * elements), so latent and rope may share one buffer.  cache_type:
 *   LATENT_CACHE_BF16  latent rows hold bf16 values; scale is NULL;
 *   LATENT_CACHE_E4M3  latent rows hold fp8 E4M3 codes (OCP: bias 7, no
 *                      infinities, 0x7F / 0xFF are NaN), value = code * scale[slot].
 * rope rows hold bf16 in both.  Row starts must be 16-byte aligned: pointers,
 * and strides of a multiple of 16 bytes.
 *
 * Every pointer is a device pointer on the current device; the caller owns it
 * and the library keeps none past the call.  Calls are asynchronous on
 * `stream`, allocate nothing, keep no state between calls (a workspace is the
 * caller's, so calls on different streams, devices or captured graphs share
 * nothing unless the caller shares it) and may be captured.  bf16 arguments
 * are passed as uint16_t pointers.  What a call writes must not overlap what it
 * reads, but for the page table that is updated in place.  Status codes and topk_last_error() are
 * topk_transform.h's.  Errors of every call: TOPK_ERROR_INVALID_VALUE for a
 * negative size, a required pointer that is NULL, a page size that is not a
 * power of two, a misaligned pointer or stride, sizes that need 2^32 threads or more
 * (2^29 loaded rows; in the absorbed form 2^26 tokens of up to 16 heads, or 2^24
 * tokens times blocks of 64 heads; in the expanded form 2^24 heads times blocks of up
 * to 128 queries); TOPK_ERROR_UNSUPPORTED on a
 * device that is not gfx950; TOPK_ERROR_LAUNCH.  On error nothing was queued.
 *
 * These entry points are additions: they leave topk_abi_version() as it is.
 */
#ifndef LATENT_ATTENTION_H_
#define LATENT_ATTENTION_H_

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "topk_transform.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LATENT_DIM 512
#define LATENT_ROPE_DIM 64
#define LATENT_HEAD_DIM 128 /* expanded form: a head's key without its rotary part, and its value */

#define LATENT_CACHE_BF16 0
#define LATENT_CACHE_E4M3 1

/*
 * paged_append_plan -- pages and slots of the tokens a step appends, from the
 * requests' lengths alone.
 *
 *   kv_lens     (num_requests,) int32: tokens the cache already holds.
 *   new_lens    (num_requests,) int32: tokens this step appends.  Negative
 *               lengths are read as 0.
 *   page_table  (num_requests, pages_per_row) int32, updated in place:
 *               entries [ceil(kv / page_size), ceil((kv + new) / page_size)) of
 *               each row take the next pages of free_pages, request by
 *               request.  Other entries are left as they are, and the ones
 *               below are read (a kept page).
 *   free_pages  (num_free,) int32; free_used (1,) int32 or NULL (= 0): how
 *               many of them earlier steps took.
 *   seq_lens    (num_requests,) int32, written: kv + new (topk_transform's seq_lens).
 *   q_starts    (num_requests + 1,) int32, written: exclusive sums of new_lens.
 *   slot_map, positions   (num_tokens,) int32, written: for token i of request
 *               b, at q_starts[b] + i, its position kv + i and its slot
 *               page_table[b, position / page_size] * page_size + position %
 *               page_size.  Entries past the last token hold -1 in both
 *               (num_tokens may exceed the step's tokens: a captured graph's
 *               buffers); tokens past num_tokens are not written.
 *   free_used_out (1,) int32, written: free_used plus the pages the step
 *               needed.  Must not be free_used itself (it is written while
 *               other workgroups still read that one).  Above num_free it
 *               tells that pages ran out: the entries of those pages hold -1,
 *               and so do their tokens' slots.
 * A token whose page lies beyond pages_per_row, or whose page is negative, or
 * whose slot would not fit int32, gets slot -1 (a page beyond the row is not
 * taken).  Precondition: the sums of new_lens and of kv + new per request
 * stay below 2^31.
 */
topk_status_t paged_append_plan(const int32_t* kv_lens, const int32_t* new_lens, int32_t* page_table,
                                const int32_t* free_pages, const int32_t* free_used, int32_t page_size,
                                int32_t* seq_lens, int32_t* q_starts, int32_t* slot_map, int32_t* positions,
                                int32_t* free_used_out, hipStream_t stream, int32_t num_requests,
                                int64_t pages_per_row, int64_t num_free, int64_t num_tokens);

/*
 * latent_cache_store -- norm, rotation, 8-bit codes and the store, in one pass.
 *
 *   kv          (num_tokens, LATENT_DIM + LATENT_ROPE_DIM) bf16, row stride
 *               kv_stride elements: each token's latent c, then its rotary key r.
 *   norm_weight (LATENT_DIM,) bf16 or NULL.  With it the stored latent is
 *               y = c * rsqrt(mean(c^2) + eps) * norm_weight; without, y = c.
 *   cos_sin     (max_positions, LATENT_ROPE_DIM) fp32 or NULL: the cosines of
 *               the 32 angles of a position, then their sines.  With it the
 *               pair (a, b) of angle i becomes (a cos - b sin, b cos + a sin); interleaved
 *               != 0 pairs elements 2i and 2i + 1, else i and i + 32.
 *   positions   (num_tokens,) int32; read only with cos_sin.
 *   slot_map    (num_tokens,) int32.  Tokens with a slot outside [0, num_slots), or
 *               (with cos_sin) a position outside [0, max_positions), are not
 *               stored.  No two tokens may name one slot (parts of either would be stored).
 * E4M3 caches: scale[slot] = max|y| / 448 (1 where y is all zero), codes =
 * y / scale rounded to nearest even.  A row whose y has a NaN or an infinity
 * reads back as NaN throughout (its scale is NaN).  All arithmetic
 * is fp32; each stored value is rounded once.
 */
topk_status_t latent_cache_store(const uint16_t* kv, int64_t kv_stride, const uint16_t* norm_weight, float eps,
                                 const int32_t* positions, const float* cos_sin, int64_t max_positions,
                                 int32_t interleaved, const int32_t* slot_map, void* latent, int64_t latent_stride,
                                 uint16_t* rope, int64_t rope_stride, float* scale, int32_t cache_type,
                                 hipStream_t stream, int64_t num_tokens, int64_t num_slots);

/*
 * latent_cache_load -- rows of the cache as contiguous bf16, by slot:
 * out_latent (num_rows, LATENT_DIM), out_rope (num_rows, LATENT_ROPE_DIM).
 * A slot outside [0, num_slots) gives a row of zeros.  E4M3 rows are
 * code * scale in fp32, rounded once.
 */
topk_status_t latent_cache_load(const int32_t* slots, const void* latent, int64_t latent_stride, const uint16_t* rope,
                                int64_t rope_stride, const float* scale, int32_t cache_type, uint16_t* out_latent,
                                uint16_t* out_rope, hipStream_t stream, int64_t num_rows, int64_t num_slots);

/*
 * latent_cache_load_paged -- the same, by page table: rows [kv_starts[b],
 * kv_starts[b + 1]) of the output are positions 0, 1, ... of request b (the
 * cached prefix the expanded form needs in front of its projection).
 * kv_starts (num_requests + 1,) int32 ascends from 0.  Rows from
 * kv_starts[num_requests] on are left as they are.  A position whose page is
 * missing (negative, or beyond pages_per_row) gives a row of zeros.
 */
topk_status_t latent_cache_load_paged(const int32_t* page_table, const int32_t* kv_starts, int32_t page_size,
                                      const void* latent, int64_t latent_stride, const uint16_t* rope,
                                      int64_t rope_stride, const float* scale, int32_t cache_type,
                                      uint16_t* out_latent, uint16_t* out_rope, hipStream_t stream,
                                      int32_t num_requests, int64_t pages_per_row, int64_t num_rows,
                                      int64_t num_slots);

/*
 * latent_attention -- absorbed form over selected slots (topk_transform's
 * out_idx as it is).
 *
 *   q        (num_tokens, num_heads, LATENT_DIM + LATENT_ROPE_DIM) bf16 with token and head
 *            strides in elements: each head's absorbed query, then its rotated
 *            rotary query.
 *   indices  (num_tokens, k) int32 slots, in any order.  Slots outside
 *            [0, num_slots) select nothing (topk_transform's -1); a slot
 *            named twice counts twice.
 *   out      (num_tokens, num_heads, LATENT_DIM) bf16, written:
 *            sum_j softmax_j(softmax_scale * (q_c . c_j + q_r . r_j)) c_j.
 *   lse      (num_tokens, num_heads) fp32 or NULL, written: the natural
 *            logarithm of the sum of exponentials.
 * A token that selects nothing gets zeros in out and -inf in lse.  What the
 * cache holds in slots that are not selected is never used, NaN included.  A
 * selected row that makes a head's score NaN (the NaN scale of an E4M3 row
 * among others) or +inf makes that head's out and lse NaN; a score of -inf
 * weighs nothing.
 * Scores, statistics and sums are fp32; the weights are rounded to bf16 for
 * the matrix cores, and the result once at the end.
 * Any score that is finite in fp32 counts as what it is.  Weights are as large as
 * 2^8 until they are divided by their sum at the end, so values beyond 2^120 / keys
 * in magnitude may overflow.
 *
 *   workspace, workspace_bytes: device memory for partial results, at least
 *            what latent_attention_workspace says for (num_tokens, num_heads,
 *            k); read and written by kernels on `stream` until the call
 *            completes there, its contents need not be kept.  NULL if that is 0.
 */
topk_status_t latent_attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, const void* latent,
                               int64_t latent_stride, const uint16_t* rope, int64_t rope_stride, const float* scale,
                               int32_t cache_type, const int32_t* indices, float softmax_scale, uint16_t* out,
                               float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream,
                               int32_t num_tokens, int32_t num_heads, int64_t k, int64_t num_slots);

/*
 * latent_attention_paged -- absorbed form over whole cached sequences.
 * Request b's tokens are rows [q_starts[b], q_starts[b + 1]) of q (q_starts
 * (num_requests + 1,) int32 ascends from 0; num_tokens rows are there).  seq_lens[b] counts the
 * cached positions, the new tokens' own included: the i-th of n new tokens attends
 * positions [0, seq_lens[b] - n + i + 1).  A position whose page is missing
 * (negative, or beyond pages_per_row) is left out.  Rows of q from
 * q_starts[num_requests] on are padding: their out and lse are left as they
 * are.  Other arguments as latent_attention; the workspace is that of (num_tokens,
 * num_heads, pages_per_row * page_size).
 */
topk_status_t latent_attention_paged(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                     const void* latent, int64_t latent_stride, const uint16_t* rope,
                                     int64_t rope_stride, const float* scale, int32_t cache_type,
                                     const int32_t* page_table, const int32_t* seq_lens, const int32_t* q_starts,
                                     int32_t page_size, float softmax_scale, uint16_t* out, float* lse,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream, int32_t num_tokens,
                                     int32_t num_heads, int32_t num_requests, int64_t pages_per_row,
                                     int64_t num_slots);

/* Bytes of workspace for up to num_tokens tokens of num_heads heads that attend
 * up to `keys` keys each (on the current device): it grows with both, so that of a
 * step's largest call serves the smaller ones. */
topk_status_t latent_attention_workspace(int32_t num_tokens, int32_t num_heads, int64_t keys, size_t* bytes);

/*
 * latent_attention_expanded -- expanded form over ragged batches (prompts,
 * with or without a cached prefix).
 *
 *   q        (num_tokens, num_heads, LATENT_HEAD_DIM + LATENT_ROPE_DIM) bf16,
 *            token and head strides in elements.
 *   kv_up    (num_kv, num_heads, 2 * LATENT_HEAD_DIM) bf16, token and head
 *            strides: each head's key (without the rotary part), then its
 *            value.  Token strides (rope's too) are below 2^24 elements.
 *   rope     (num_kv, LATENT_ROPE_DIM) bf16, row stride: the rotary keys,
 *            shared by the heads.
 *   q_starts, kv_starts   (num_requests + 1,) int32, ascending from 0:
 *            request b has query rows [q_starts[b], q_starts[b + 1]) and key
 *            rows [kv_starts[b], kv_starts[b + 1]).
 *   causal   != 0: the i-th of nq queries attends keys [0, nk - nq + i + 1) of
 *            its request's nk; 0: all of them.
 *   out      (num_tokens, num_heads, LATENT_HEAD_DIM) bf16; lse (num_tokens,
 *            num_heads) fp32 or NULL: as latent_attention.
 * A query with no key gets zeros and -inf, one with a score that is NaN or
 * +inf gets NaN in both.  Rows of q from
 * q_starts[num_requests] on are left as they are in out and lse; key rows from
 * kv_starts[num_requests] on are not read.  The workspace is
 * latent_attention_expanded_workspace's, otherwise as latent_attention's.
 */
topk_status_t latent_attention_expanded(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                        const uint16_t* kv_up, int64_t kv_token_stride, int64_t kv_head_stride,
                                        const uint16_t* rope, int64_t rope_stride, const int32_t* q_starts,
                                        const int32_t* kv_starts, float softmax_scale, int32_t causal, uint16_t* out,
                                        float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream,
                                        int32_t num_tokens, int64_t num_kv, int32_t num_heads, int32_t num_requests);

/* Bytes of workspace of a call with these sizes or smaller ones (on the current device). */
topk_status_t latent_attention_expanded_workspace(int32_t num_tokens, int32_t num_heads, int64_t num_kv,
                                                  int32_t num_requests, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* LATENT_ATTENTION_H_ */
