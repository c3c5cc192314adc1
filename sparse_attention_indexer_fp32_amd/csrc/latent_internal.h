// Internal interface between the latent cache's and latent attention's C-ABI
// layer (latent_api.cpp) and their kernels.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "latent_attention.h"

namespace latent {

constexpr int kLatent = LATENT_DIM;
constexpr int kRope = LATENT_ROPE_DIM;
constexpr int kQuery = kLatent + kRope;
constexpr int kHead = LATENT_HEAD_DIM;

// Threads of a launch along x: the hardware counts them in 32 bits, and what is
// beyond is cut off without an error.
constexpr int64_t kMaxThreads = UINT32_MAX;

// A paged cache as the kernels see it; strides in bytes.
struct Cache {
  const char* latent;
  const char* rope;
  const float* scale;        // E4M3 only
  int64_t latent_stride;
  int64_t rope_stride;
  int64_t num_slots;
};

struct PlanArgs {
  const int32_t* kv_lens;
  const int32_t* new_lens;
  int32_t* page_table;
  const int32_t* free_pages;
  const int32_t* free_used;  // or nullptr
  int32_t* seq_lens;
  int32_t* q_starts;
  int32_t* slot_map;
  int32_t* positions;
  int32_t* free_used_out;
  int64_t pages_per_row;
  int64_t num_free;
  int64_t num_tokens;
  int32_t num_requests;
  int32_t log2_page;
};
hipError_t launch_append_plan(const PlanArgs& a, hipStream_t stream);

struct StoreArgs {
  const uint16_t* kv;
  int64_t kv_stride;         // elements
  const uint16_t* norm_weight;   // or nullptr
  const int32_t* positions;
  const float* cos_sin;      // or nullptr
  int64_t max_positions;
  const int32_t* slot_map;
  char* latent;
  char* rope;
  float* scale;
  int64_t latent_stride;     // bytes
  int64_t rope_stride;
  int64_t num_tokens;
  int64_t num_slots;
  float eps;
  int32_t interleaved;
};
hipError_t launch_cache_store(const StoreArgs& a, bool e4m3, hipStream_t stream);

struct LoadArgs {
  Cache cache;
  const int32_t* slots;      // by slot, or nullptr
  const int32_t* page_table; // by page table
  const int32_t* kv_starts;
  int64_t pages_per_row;
  uint16_t* out_latent;
  uint16_t* out_rope;
  int64_t num_rows;
  int32_t num_requests;
  int32_t log2_page;
};
int64_t load_threads(int64_t num_rows);
hipError_t launch_cache_load(const LoadArgs& a, bool e4m3, hipStream_t stream);

// Absorbed form.  Tokens' keys are cut in tiles of kTileKeys.  Split: `wgs`
// workgroups share all tokens' tiles evenly, so one may end a token, hold
// whole ones and begin another; parts of a token go to the workspace and are
// joined by a second launch.  Not split: one workgroup per token.
constexpr int kTileKeys = 32;
constexpr int kShareTiles = 4;       // tiles a workgroup of a split launch takes at least
constexpr int kPlanTokens = 1024;    // tokens a split launch over whole sequences takes at most

struct AttendArgs {
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;   // elements
  Cache cache;
  const int32_t* indices;    // (num_tokens, k): selected slots, or nullptr
  int64_t k;
  const int32_t* page_table; // whole sequences
  const int32_t* seq_lens;
  const int32_t* q_starts;
  int64_t pages_per_row;
  int32_t num_requests;
  int32_t log2_page;
  float scale_log2;          // softmax scale * log2(e)
  uint16_t* out;
  float* lse;                // or nullptr
  int32_t num_tokens;
  int32_t num_heads;
  int32_t wgs;               // split: workgroups per head block; 0: not split
  // workspace of a split launch (split_layout)
  float* part_out;
  float2* part_ml;
  int32_t* part_rec;
};

// By head count: waves that share a ring of tiles, and heads they take; and the
// workspace of a split launch.
int attend_waves(int num_heads);
int attend_heads(int num_heads);
struct SplitLayout {
  size_t out_bytes, ml_bytes, rec_bytes;
  size_t total() const { return out_bytes + ml_bytes + rec_bytes; }
};
SplitLayout split_layout(int num_tokens, int num_heads, int wgs);
int64_t attend_threads(int num_tokens, int num_heads);     // the most of any launch of the call
hipError_t launch_attend(const AttendArgs& a, bool e4m3, hipStream_t stream);

// Absorbed form over whole sequences that share prefixes.  A unit is 64
// neighbouring rows of (token, head) pairs of one group against its shared
// prefix, or of one request against its own keys.  `wgs` workgroups share all
// units' tiles evenly; every unit's parts go to the workspace and are joined by a
// second launch.  Tokens are taken `shared_tokens` at a time.
constexpr int kUnitWaves = 4;
constexpr int kUnitRows = 16 * kUnitWaves;
constexpr int kSharedTiles = 6;      // tiles a workgroup takes at least, the cost of a unit among them
struct SharedArgs {
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;   // elements
  Cache cache;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* q_starts;
  const int32_t* group_starts;
  const int32_t* shared_lens;
  int64_t pages_per_row;
  int32_t num_requests;
  int32_t num_groups;
  int32_t log2_page;
  float scale_log2;          // softmax scale * log2(e)
  uint16_t* out;
  float* lse;                // or nullptr
  int32_t first_token;       // of this launch
  int32_t num_tokens;        // of this launch
  int32_t num_heads;
  int32_t wgs;
  int32_t pieces;            // of 16 rows, that units of one kind may have
  // workspace (shared_layout)
  float* part_out;
  float2* part_ml;
  int4* part_rec;            // two a row: its places in the parts of the group's unit, and of the request's
};
int shared_tokens(int num_tokens, int num_heads, int64_t keys);
int shared_pieces(int num_tokens, int num_heads);
SplitLayout shared_layout(int num_tokens, int num_heads, int wgs);
hipError_t launch_shared(const SharedArgs& a, bool e4m3, hipStream_t stream);

// Expanded form.  A unit is a block of 128 queries of one head.  Split: `wgs`
// workgroups share all units' tiles of 64 keys evenly, as above.
constexpr int kPlanRequests = 512;       // requests a split launch takes at most
constexpr int kPrefillShareTiles = 8;    // tiles a workgroup of a split launch takes at least
struct PrefillArgs {
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;   // elements
  const uint16_t* kv;
  int64_t kv_token_stride, kv_head_stride; // elements
  const uint16_t* rope;
  int64_t rope_stride;                     // elements
  const int32_t* q_starts;
  const int32_t* kv_starts;
  float scale_log2;
  int32_t causal;
  uint16_t* out;
  float* lse;                // or nullptr
  int32_t num_tokens;
  int64_t num_kv;
  int32_t num_heads;
  int32_t num_requests;
  int32_t wgs;               // split: workgroups; 0: one per unit
  float* part_out;           // workspace of a split launch (prefill_split_layout)
  float2* part_ml;
  int32_t* part_rec;
};
int64_t prefill_blocks(int num_tokens, int num_requests);   // of one head, at most
SplitLayout prefill_split_layout(int num_tokens, int num_heads, int num_requests, int wgs);
int64_t prefill_threads(int num_tokens, int num_heads, int num_requests);
hipError_t launch_prefill(const PrefillArgs& a, hipStream_t stream);

}  // namespace latent
