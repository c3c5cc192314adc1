/*
 * indexer_paged.h -- C ABI of the indexer's paged key cache on the MI355X
 * (gfx950): the step before the scoring and selection of indexer_topk.h and
 * topk_transform.h.  A step of a model appends its tokens' index keys
 * (indexer_cache_store), brings their queries in the form the scores take
 * (indexer_queries), scores them against the cached keys where they are
 * (indexer_logits_paged, whose rows topk_transform selects from), or lays a
 * long prompt's cached keys in a row for indexer_topk's scan
 * (indexer_cache_load_paged).
 *
 * Cache.  A slot is one token's place, the same as in the latent cache
 * (latent_attention.h): paged_append_plan's slot_map and page_table serve both.
 * keys (num_slots, 128) uint8: fp8 E4M3 codes (OCP: bias 7, no infinities, 0x7F /
 * 0xFF are NaN), row stride key_stride bytes, rows on 16-byte boundaries;
 * key_scale (num_slots,) fp32: value = code * key_scale[slot].
 *
 * A row of INDEXER_HEAD_DIM values x is brought in 8 bits like this:
 *   rotation (with cos_sin): the first INDEXER_ROPE_DIM values are 32 pairs;
 *     the pair (a, b) of angle i becomes (a cos - b sin, b cos + a sin), interleaved
 *     != 0 pairing elements 2i and 2i + 1, else i and i + 32;
 *   mixing (with hadamard != 0): y[i] = sum_j (-1)^popcount(i & j) x[j] / sqrt(128),
 *     which leaves products of a query and a key as they are and spreads what is
 *     large in one of their elements over all;
 *   scale = max|y| / 448, but 2^-126 at least (1 where y is all zero), codes = y / scale, a quotient in
 *     fp32 (with mixing, of numerator and denominator without their factor 1 / sqrt(128)), rounded to
 *     nearest even.  A row with a NaN or an infinity has a NaN scale, and so has one whose sums in the
 *     rotation or the mixing leave fp32 (values beyond 2^120).
 * cos_sin (max_positions, 64) fp32: the cosines of the 32 angles of a position, then
 * their sines; 16-byte aligned.  All arithmetic is fp32; each stored value is rounded once.
 *
 * Every pointer is a device pointer on the current device; the caller owns it
 * and the library keeps none past the call.  Calls are asynchronous on
 * `stream`, allocate nothing, need no workspace, keep no state between calls
 * and may be captured.  bf16 arguments are passed as uint16_t pointers.  What a call writes must not
 * overlap what it reads.  Status codes and topk_last_error() are
 * topk_transform.h's.  Errors of every call: TOPK_ERROR_INVALID_VALUE for a negative
 * size, a required pointer that is NULL, a page size that is not a power of
 * two, a misaligned pointer or stride, sizes that a launch cannot count (stated
 * at the call); TOPK_ERROR_UNSUPPORTED on a device that is not gfx950;
 * TOPK_ERROR_LAUNCH.  On error nothing was queued.
 *
 * These entry points are additions: they leave topk_abi_version() as it is.
 */
#ifndef INDEXER_PAGED_H_
#define INDEXER_PAGED_H_

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "indexer_topk.h"
#include "topk_transform.h"

#ifdef __cplusplus
extern "C" {
#endif

#define INDEXER_ROPE_DIM 64

#define INDEXER_BF16 0
#define INDEXER_FP32 1

/*
 * indexer_cache_store -- layer norm, rotation, mixing, 8-bit codes and the
 * store of a step's index keys, in one pass.
 *
 *   k           (num_tokens, 128) bf16, row stride k_stride elements.
 *   norm_weight, norm_bias   (128,) of norm_type (INDEXER_BF16 or INDEXER_FP32),
 *               16-byte aligned, or both NULL.  With them x = (k - mean(k)) / sqrt(mean((k -
 *               mean(k))^2) + eps) * norm_weight + norm_bias; without, x = k.
 *   positions   (num_tokens,) int32; read only with cos_sin (NULL: no rotation).
 *   slot_map    (num_tokens,) int32.  Tokens with a slot outside [0, num_slots), or
 *               (with cos_sin) a position outside [0, max_positions), are not
 *               stored.  No two tokens may name one slot (parts of either would be stored).
 * Up to 2^31 - 1 tokens.
 */
topk_status_t indexer_cache_store(const uint16_t* k, int64_t k_stride, const void* norm_weight, const void* norm_bias,
                                  int32_t norm_type, float eps, const int32_t* positions, const float* cos_sin,
                                  int64_t max_positions, int32_t interleaved, int32_t hadamard,
                                  const int32_t* slot_map, uint8_t* keys, int64_t key_stride, float* key_scale,
                                  hipStream_t stream, int64_t num_tokens, int64_t num_slots);

/*
 * indexer_queries -- a step's queries and head weights as indexer_logits,
 * indexer_topk and indexer_logits_paged take them.
 *
 *   q           (num_tokens, 32, 128) bf16, token and head strides in elements.
 *   weights     (num_tokens, 32) of weight_type, row stride in elements.
 *   out_q       (num_tokens, 32, 128) uint8, written: each head's codes.
 *   out_weights (num_tokens, 32) fp32, written: weights * weight_scale * the
 *               head's scale, so that the scores of the codes under these are those
 *               of the values under weights * weight_scale.
 * With cos_sin, tokens with a position outside [0, max_positions) are padding:
 * their rows of out_q and out_weights are left as they are.  Up to 2^26 tokens.
 */
topk_status_t indexer_queries(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, const void* weights,
                              int64_t weight_stride, int32_t weight_type, float weight_scale, const int32_t* positions,
                              const float* cos_sin, int64_t max_positions, int32_t interleaved, int32_t hadamard,
                              uint8_t* out_q, float* out_weights, hipStream_t stream, int64_t num_tokens);

/*
 * indexer_cache_load_paged -- the cached keys of whole requests in a row, as
 * indexer_logits and indexer_topk take them: rows [kv_starts[b], kv_starts[b +
 * 1]) of out_keys (num_rows, 128) and out_scale (num_rows,) are positions 0, 1,
 * ... of request b.  kv_starts (num_requests + 1,) int32 ascends from 0.  Rows
 * from kv_starts[num_requests] on are left as they are.  A position whose page
 * is missing (negative, or beyond pages_per_row, or its slot beyond num_slots) gives codes
 * and a scale of zero.  Up to 2^31 - 1 rows.
 */
topk_status_t indexer_cache_load_paged(const int32_t* page_table, const int32_t* kv_starts, int32_t page_size,
                                       const uint8_t* keys, int64_t key_stride, const float* key_scale,
                                       uint8_t* out_keys, float* out_scale, hipStream_t stream, int32_t num_requests,
                                       int64_t pages_per_row, int64_t num_rows, int64_t num_slots);

/*
 * indexer_logits_paged -- scores of a step's new tokens against their
 * requests' cached keys (indexer_topk.h's formula and its error bound; NaN codes
 * are outside the contract).
 *
 *   q          (num_tokens, 32, 128) uint8 codes, row-major, 16-byte aligned.
 *   weights    (num_tokens, 32) fp32, 16-byte aligned.
 *   page_table (num_requests, pages_per_row) int32; seq_lens (num_requests,)
 *              int32: cached positions, the new tokens' own included; q_starts
 *              (num_requests + 1,) int32, ascending from 0: request b's tokens are
 *              rows [q_starts[b], q_starts[b + 1]).
 *   logits     (num_tokens, width) fp32, written: for the i-th of request b's n
 *              tokens, the scores of positions [0, L), L = seq_lens[b] - n + i + 1
 *              clamped to [0, min(width, pages_per_row * page_size)]; other entries are
 *              left as they are.  A position whose page is missing (negative, or its
 *              slot beyond num_slots) scores -inf.
 *   lens       (num_tokens,) int32 or NULL, written: L (topk_transform's seq_lens).
 * Rows from q_starts[num_requests] on are padding: their logits are left as
 * they are, and their lens are 0.  For topk_transform, a request's row of the page table
 * stands for each of its tokens.
 * num_tokens * (width / 64 + 1) must stay below 2^31, and width below 2^29.
 * Results do not depend on what else is in a call, but its time does: how many tokens a key is read for at once
 * follows num_tokens / num_requests (requests without new tokens and padding among them), so a long chunk and many
 * requests of one token, or of none, are faster in calls of their own.
 */
topk_status_t indexer_logits_paged(const uint8_t* q, const float* weights, const uint8_t* keys, int64_t key_stride,
                                   const float* key_scale, const int32_t* page_table, const int32_t* seq_lens,
                                   const int32_t* q_starts, int32_t page_size, float* logits, int32_t* lens,
                                   hipStream_t stream, int32_t num_tokens, int32_t num_requests,
                                   int64_t pages_per_row, int64_t width, int64_t num_slots);

#ifdef __cplusplus
}
#endif

#endif /* INDEXER_PAGED_H_ */
