// C-ABI layer of the indexer's paged key cache: argument and device checks,
// launches.  Nothing is allocated or kept here but the number of CUs of each
// device seen.

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdio>
#include <cstring>

#include "indexer_paged.h"
#include "indexer_paged_internal.h"
#include "topk_internal.h"

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_cus[kMaxDevices];   // CUs of each device, -1 when it is not gfx950, 0 before it is asked

topk_status_t fail(topk_status_t st, const char* msg) {
  topk::set_last_error(msg);
  return st;
}

topk_status_t invalid(const char* msg) { return fail(TOPK_ERROR_INVALID_VALUE, msg); }

topk_status_t launched(hipError_t e, const char* what) {
  if (e == hipSuccess) {
    topk::set_last_launch(what);
    return TOPK_SUCCESS;
  }
  char buf[256];
  std::snprintf(buf, sizeof(buf), "%s launch: %s", what, hipGetErrorString(e));
  return fail(TOPK_ERROR_LAUNCH, buf);
}

// CUs of the current device; TOPK_ERROR_UNSUPPORTED when it is not gfx950.
topk_status_t device_cus(int* cus) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return fail(TOPK_ERROR_LAUNCH, "hipGetDevice failed");
  if (dev < 0 || dev >= kMaxDevices) return fail(TOPK_ERROR_UNSUPPORTED, "device number too large");
  int n = g_cus[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
      return fail(TOPK_ERROR_LAUNCH, "hipGetDeviceProperties failed");
    n = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? prop.multiProcessorCount : -1;
    g_cus[dev].store(n, std::memory_order_relaxed);
  }
  if (n < 0) return fail(TOPK_ERROR_UNSUPPORTED, "device is not gfx950");
  *cus = n;
  return TOPK_SUCCESS;
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int log2_of(int32_t page_size) {
  if (page_size < 1 || (page_size & (page_size - 1)) != 0) return -1;
  return __builtin_ctz((unsigned)page_size);
}

topk_status_t check_keys(const uint8_t* keys, int64_t key_stride, const float* key_scale, int64_t num_slots) {
  if (num_slots < 0 || num_slots > (int64_t)INT32_MAX) return invalid("num_slots must be in [0, 2^31)");
  if (num_slots > 0 && (!keys || !key_scale)) return invalid("keys and key_scale must be non-null when num_slots > 0");
  if (key_stride < INDEXER_HEAD_DIM || key_stride > (int64_t)1 << 31)
    return invalid("cache rows overlap or are too far apart: key_stride must be in [128, 2^31]");
  if (!aligned(keys) || key_stride % 16 != 0) return invalid("cache rows must start on 16-byte boundaries");
  return TOPK_SUCCESS;
}

topk_status_t check_turn(const int32_t* positions, const float* cos_sin, int64_t max_positions, int32_t interleaved,
                         int32_t hadamard, indexer::TurnArgs* t) {
  if (cos_sin && (!positions || max_positions < 0)) return invalid("cos_sin needs positions and max_positions >= 0");
  if (cos_sin && !aligned(cos_sin)) return invalid("cos_sin must start on a 16-byte boundary");
  t->positions = positions;
  t->cos_sin = cos_sin;
  t->max_positions = max_positions;
  t->interleaved = interleaved;
  t->hadamard = hadamard;
  return TOPK_SUCCESS;
}

// A paged cache of a reading call, and its page table.
topk_status_t check_paged(const uint8_t* keys, int64_t key_stride, const float* key_scale, int64_t num_slots,
                          const int32_t* page_table, int32_t page_size, int32_t num_requests, int64_t pages_per_row,
                          indexer::PagedKeys* c) {
  const topk_status_t st = check_keys(keys, key_stride, key_scale, num_slots);
  if (st != TOPK_SUCCESS) return st;
  c->log2_page = log2_of(page_size);
  if (c->log2_page < 0) return invalid("page_size must be a power of two");
  if (num_requests < 0 || pages_per_row < 0 || pages_per_row > (int64_t)INT32_MAX)
    return invalid("num_requests must be >= 0 and pages_per_row in [0, 2^31)");
  if (num_requests > 0 && pages_per_row > 0 && !page_table) return invalid("page_table must be non-null");
  c->keys = keys;
  c->key_stride = key_stride;
  c->scale = key_scale;
  c->page_table = page_table;
  c->pages_per_row = pages_per_row;
  c->num_slots = num_slots;
  c->num_requests = num_requests;
  return TOPK_SUCCESS;
}

}  // namespace

extern "C" {

topk_status_t indexer_cache_store(const uint16_t* k, int64_t k_stride, const void* norm_weight, const void* norm_bias,
                                  int32_t norm_type, float eps, const int32_t* positions, const float* cos_sin,
                                  int64_t max_positions, int32_t interleaved, int32_t hadamard,
                                  const int32_t* slot_map, uint8_t* keys, int64_t key_stride, float* key_scale,
                                  hipStream_t stream, int64_t num_tokens, int64_t num_slots) {
  topk::set_last_error("");
  topk_status_t st = check_keys(keys, key_stride, key_scale, num_slots);
  if (st != TOPK_SUCCESS) return st;
  indexer::StoreArgs a{};
  st = check_turn(positions, cos_sin, max_positions, interleaved, hadamard, &a.turn);
  if (st != TOPK_SUCCESS) return st;
  if (num_tokens < 0 || num_tokens > (int64_t)INT32_MAX) return invalid("num_tokens must be in [0, 2^31)");
  if (norm_type != INDEXER_BF16 && norm_type != INDEXER_FP32) return invalid("norm_type must be INDEXER_BF16 or INDEXER_FP32");
  if (!norm_weight != !norm_bias) return invalid("norm_weight and norm_bias go together");
  if (!aligned(norm_weight) || !aligned(norm_bias)) return invalid("norm_weight and norm_bias must start on 16-byte boundaries");
  if (num_tokens == 0) return TOPK_SUCCESS;
  if (!k || !slot_map) return invalid("k and slot_map must be non-null");
  if (k_stride < INDEXER_HEAD_DIM || k_stride % 8 != 0 || !aligned(k))
    return invalid("k's rows must not overlap and must start on 16-byte boundaries");
  int cus = 0;
  st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  a.k = k;
  a.k_stride = k_stride;
  a.norm_weight = norm_weight;
  a.norm_bias = norm_bias;
  a.norm_fp32 = norm_type == INDEXER_FP32;
  a.eps = eps;
  a.slot_map = slot_map;
  a.keys = keys;
  a.key_stride = key_stride;
  a.key_scale = key_scale;
  a.num_tokens = num_tokens;
  a.num_slots = num_slots;
  return launched(indexer::launch_key_store(a, stream), "indexer-cache-store");
}

topk_status_t indexer_queries(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, const void* weights,
                              int64_t weight_stride, int32_t weight_type, float weight_scale, const int32_t* positions,
                              const float* cos_sin, int64_t max_positions, int32_t interleaved, int32_t hadamard,
                              uint8_t* out_q, float* out_weights, hipStream_t stream, int64_t num_tokens) {
  topk::set_last_error("");
  indexer::QueryArgs a{};
  topk_status_t st = check_turn(positions, cos_sin, max_positions, interleaved, hadamard, &a.turn);
  if (st != TOPK_SUCCESS) return st;
  if (num_tokens < 0 || num_tokens > (int64_t)1 << 26) return invalid("num_tokens must be in [0, 2^26]");
  if (weight_type != INDEXER_BF16 && weight_type != INDEXER_FP32) return invalid("weight_type must be INDEXER_BF16 or INDEXER_FP32");
  if (num_tokens == 0) return TOPK_SUCCESS;
  if (!q || !weights || !out_q || !out_weights) return invalid("q, weights, out_q and out_weights must be non-null");
  if (q_token_stride < 0 || weight_stride < 0 || q_head_stride < INDEXER_HEAD_DIM)
    return invalid("q's heads overlap, or a stride is negative");
  if (!aligned(q) || !aligned(out_q) || q_token_stride % 8 != 0 || q_head_stride % 8 != 0)
    return invalid("q's rows and out_q must start on 16-byte boundaries");
  int cus = 0;
  st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  a.q = q;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.weights = weights;
  a.weight_stride = weight_stride;
  a.weight_fp32 = weight_type == INDEXER_FP32;
  a.weight_scale = weight_scale;
  a.out_q = out_q;
  a.out_weights = out_weights;
  a.num_tokens = num_tokens;
  return launched(indexer::launch_queries(a, stream), "indexer-queries");
}

topk_status_t indexer_cache_load_paged(const int32_t* page_table, const int32_t* kv_starts, int32_t page_size,
                                       const uint8_t* keys, int64_t key_stride, const float* key_scale,
                                       uint8_t* out_keys, float* out_scale, hipStream_t stream, int32_t num_requests,
                                       int64_t pages_per_row, int64_t num_rows, int64_t num_slots) {
  topk::set_last_error("");
  indexer::KeyLoadArgs a{};
  topk_status_t st = check_paged(keys, key_stride, key_scale, num_slots, page_table, page_size, num_requests, pages_per_row, &a.cache);
  if (st != TOPK_SUCCESS) return st;
  if (num_rows < 0 || num_rows > (int64_t)INT32_MAX) return invalid("num_rows must be in [0, 2^31)");
  if (num_rows == 0 || num_requests == 0) return TOPK_SUCCESS;
  if (!kv_starts || !out_keys || !out_scale) return invalid("kv_starts, out_keys and out_scale must be non-null");
  if (!aligned(out_keys)) return invalid("out_keys must start on a 16-byte boundary");
  int cus = 0;
  st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  a.kv_starts = kv_starts;
  a.out_keys = out_keys;
  a.out_scale = out_scale;
  a.num_rows = num_rows;
  return launched(indexer::launch_key_load(a, stream), "indexer-cache-load paged");
}

topk_status_t indexer_logits_paged(const uint8_t* q, const float* weights, const uint8_t* keys, int64_t key_stride,
                                   const float* key_scale, const int32_t* page_table, const int32_t* seq_lens,
                                   const int32_t* q_starts, int32_t page_size, float* logits, int32_t* lens,
                                   hipStream_t stream, int32_t num_tokens, int32_t num_requests,
                                   int64_t pages_per_row, int64_t width, int64_t num_slots) {
  topk::set_last_error("");
  indexer::PagedLogitsArgs a{};
  topk_status_t st = check_paged(keys, key_stride, key_scale, num_slots, page_table, page_size, num_requests, pages_per_row, &a.cache);
  if (st != TOPK_SUCCESS) return st;
  if (num_tokens < 0) return invalid("num_tokens must be >= 0");
  if (width < 0 || width >= (int64_t)1 << 29) return invalid("width must be in [0, 2^29)");
  if (num_tokens == 0) return TOPK_SUCCESS;
  if (!q || !weights || !q_starts) return invalid("q, weights and q_starts must be non-null");
  if (num_requests > 0 && !seq_lens) return invalid("seq_lens must be non-null");
  if (!aligned(q) || !aligned(weights)) return invalid("q and weights must start on 16-byte boundaries");
  if (!logits && width > 0) return invalid("logits must be non-null");
  if ((width / 64 + 1) * num_tokens > (int64_t)INT32_MAX) return invalid("more tokens and positions than the tiles of a launch are counted in");
  int cus = 0;
  st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  const int64_t cached = pages_per_row * (int64_t)page_size;
  a.q = q;
  a.weights = weights;
  a.seq_lens = seq_lens;
  a.q_starts = q_starts;
  a.logits = logits;
  a.lens = lens;
  a.width = width;
  a.most_keys = width < cached ? width : cached;
  a.num_tokens = num_tokens;
  return launched(indexer::launch_paged_logits(a, cus, stream), "indexer-logits paged");
}

}  // extern "C"
