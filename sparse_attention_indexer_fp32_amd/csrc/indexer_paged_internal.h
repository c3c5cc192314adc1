// Internal interface between the C-ABI layer of the indexer's paged cache
// (indexer_paged_api.cpp) and its kernels.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace indexer {

// Rotation, mixing: the same for keys and queries.
struct TurnArgs {
  const int32_t* positions;
  const float* cos_sin;      // or nullptr
  int64_t max_positions;
  int32_t interleaved;
  int32_t hadamard;
};

struct StoreArgs {
  TurnArgs turn;
  const uint16_t* k;
  int64_t k_stride;          // elements
  const void* norm_weight;   // or nullptr
  const void* norm_bias;
  int32_t norm_fp32;
  float eps;
  const int32_t* slot_map;
  uint8_t* keys;
  int64_t key_stride;        // bytes
  float* key_scale;
  int64_t num_tokens;
  int64_t num_slots;
};
hipError_t launch_key_store(const StoreArgs& a, hipStream_t stream);

struct QueryArgs {
  TurnArgs turn;
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;   // elements
  const void* weights;
  int64_t weight_stride;     // elements
  int32_t weight_fp32;
  float weight_scale;
  uint8_t* out_q;
  float* out_weights;
  int64_t num_tokens;
};
hipError_t launch_queries(const QueryArgs& a, hipStream_t stream);

// The paged key cache as the readers see it.
struct PagedKeys {
  const uint8_t* keys;
  int64_t key_stride;        // bytes
  const float* scale;
  const int32_t* page_table;
  int64_t pages_per_row;
  int64_t num_slots;
  int32_t log2_page;
  int32_t num_requests;
};

struct KeyLoadArgs {
  PagedKeys cache;
  const int32_t* kv_starts;
  uint8_t* out_keys;
  float* out_scale;
  int64_t num_rows;
};
hipError_t launch_key_load(const KeyLoadArgs& a, hipStream_t stream);

struct PagedLogitsArgs {
  PagedKeys cache;
  const uint8_t* q;
  const float* weights;
  const int32_t* seq_lens;
  const int32_t* q_starts;
  float* logits;
  int32_t* lens;             // or nullptr
  int64_t width;
  int64_t most_keys;         // min(width, pages_per_row * page size)
  int32_t num_tokens;
};
hipError_t launch_paged_logits(const PagedLogitsArgs& a, int cus, hipStream_t stream);

}  // namespace indexer
