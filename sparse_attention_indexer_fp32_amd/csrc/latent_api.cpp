// C-ABI layer of the paged latent cache and of latent attention: argument and
// device checks, launch shapes.  Nothing is allocated or kept here but the
// number of CUs of each device seen.

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdio>
#include <cstring>

#include "latent_attention.h"
#include "latent_internal.h"
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

// The cache's arrays; strides in elements in, bytes out.
topk_status_t check_cache(const void* latent, int64_t latent_stride, const uint16_t* rope, int64_t rope_stride,
                          const float* scale, int32_t cache_type, int64_t num_slots, latent::Cache* c) {
  if (cache_type != LATENT_CACHE_BF16 && cache_type != LATENT_CACHE_E4M3)
    return invalid("cache_type must be LATENT_CACHE_BF16 or LATENT_CACHE_E4M3");
  const bool e4m3 = cache_type == LATENT_CACHE_E4M3;
  if (num_slots < 0 || num_slots > (int64_t)INT32_MAX) return invalid("num_slots must be in [0, 2^31)");
  if (num_slots > 0 && (!latent || !rope)) return invalid("latent and rope must be non-null when num_slots > 0");
  if (e4m3 && num_slots > 0 && !scale) return invalid("an E4M3 cache needs its scales");
  if (!e4m3 && scale) return invalid("a bf16 cache has no scales");
  const int64_t lb = latent_stride * (e4m3 ? 1 : 2), rb = rope_stride * 2;
  if (latent_stride < LATENT_DIM || rope_stride < LATENT_ROPE_DIM)
    return invalid("cache rows overlap: latent_stride >= 512 and rope_stride >= 64 are needed");
  if (latent_stride > (int64_t)1 << 31 || rope_stride > (int64_t)1 << 31) return invalid("cache row stride too large");
  if (!aligned(latent) || !aligned(rope) || lb % 16 != 0 || rb % 16 != 0)
    return invalid("cache rows must start on 16-byte boundaries");
  c->latent = static_cast<const char*>(latent);
  c->rope = reinterpret_cast<const char*>(rope);
  c->scale = scale;
  c->latent_stride = lb;
  c->rope_stride = rb;
  c->num_slots = num_slots;
  return TOPK_SUCCESS;
}

// Largest row stride (elements) of the expanded form's keys: byte offsets within a tile of 64 rows take 32 bits.
constexpr int64_t kMaxTileStride = (1 << 24) - 8;

// The kernels' scale: in log2 units, and not quite 0, which would make 0 * -inf
// of a masked score (2^-149, the least there is, leaves every finite score below 2^-21).
float scale_log2(float softmax_scale) {
  return softmax_scale == 0.f ? 0x1p-149f : softmax_scale * 1.44269504088896340736f;
}

// Tiles of a token that attends `keys` keys, and one more: an upper bound for what the kernel counts.
int64_t bound_tiles(int64_t keys) { return keys / latent::kTileKeys + (keys % latent::kTileKeys != 0) + 1; }

// The most workgroups that share so many tokens' tiles: it grows with both.  One takes
// a CU's LDS, and kShareTiles tiles or more: one token of 64 tiles x 128 heads
// took 27.8 us at one tile to a workgroup, 22.3 at two and 21.9 at four; 4 tokens
// x 64 heads 31.6, 26.6 and 25.3.
int most_wgs(int cus, int32_t num_tokens, int64_t blocks, int64_t tiles) {
  const int64_t wgs = cus / blocks, share = latent::kShareTiles;
  const int64_t most = tiles > share * cus ? wgs : num_tokens * tiles / share;
  return most < 1 || wgs < 1 ? 1 : (int)(wgs < most ? wgs : most);
}

int64_t head_blocks(int32_t num_heads) {
  const int heads = latent::attend_heads(num_heads);
  return ((int64_t)num_heads + heads - 1) / heads;
}

// Workgroups that share the tiles of a launch of absorbed attention, or 0 for one
// workgroup per token.  Not split, two workgroups run on a CU at a time, and the
// last round of them may leave most CUs idle: split is what leaves more than a
// third idle (64 heads, 2048 selected bf16 slots, us split and not: 300 tokens
// 143 and 150, 400 tokens 195 and 158, 512 tokens 196 and 178; 700 tokens of 8-bit
// slots 366 and 333).  With 32 heads split launches are the faster ones where rounds
// are not full (700 tokens 237 and 286) and with 8-bit slots (512 tokens 184 and
// 222, 2048 tokens 689 and 817), and as fast otherwise (512 tokens 173 and 172,
// 2048 tokens 669 and 656), so all of them are; with 16 heads they are not
// (1024 tokens 336 and 331, 8-bit 361 and 330).
int split_wgs(int cus, int32_t num_tokens, int32_t num_heads, int64_t keys, bool paged, int32_t num_requests) {
  if (paged && (num_tokens > latent::kPlanTokens || num_requests > 65535)) return 0;
  const int64_t blocks = head_blocks(num_heads), tiles = bound_tiles(keys);
  if (tiles > (int64_t)INT32_MAX / num_tokens) return 0;         // the plan counts tiles in 32 bits
  const int64_t items = num_tokens * blocks, round = 2 * (int64_t)cus;
  const int64_t rounds = (items + round - 1) / round;
  if (latent::attend_waves(num_heads) != 2 && 3 * items >= 2 * rounds * round) return 0;
  return most_wgs(cus, num_tokens, blocks, tiles);
}

// The same for the expanded form: workgroups that share all units' tiles, or 0
// for one workgroup per unit (at most two run on a CU at a time).  Split pays
// where units leave a quarter of the card idle and are long, 32 tiles of 64
// keys on average (us split and not, new tokens x heads behind cached
// ones: 100 x 8 behind 60000 92 and 1335; 2048 x 16 behind 2048 99 and 112; 128
// x 64 behind 2000 57 and 66, behind 1000 54 and 43; 1500 x 32 behind 6000 266
// and 266, 2048 x 32 behind 8000 427 and 390: shares of a head read
// different keys at a time, blocks of a head the same ones out of L2).
constexpr int64_t kSplitKeys = 32 * 64;
int prefill_wgs(int cus, int32_t num_tokens, int32_t num_heads, int64_t num_kv, int32_t num_requests) {
  const int64_t units = latent::prefill_blocks(num_tokens, num_requests) * num_heads, round = 2 * (int64_t)cus;
  const bool pays = 4 * units < 3 * round && num_kv >= kSplitKeys * num_requests;
  return num_requests <= latent::kPlanRequests && pays ? (int)round : 0;
}

topk_status_t check_queries(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, const uint16_t* out,
                            int32_t num_tokens, int32_t num_heads, int width) {
  if (num_tokens < 0 || num_heads < 0) return invalid("num_tokens and num_heads must be >= 0");
  if (num_tokens == 0 || num_heads == 0) return TOPK_SUCCESS;
  if (!q || !out) return invalid("q and out must be non-null");
  if (q_token_stride < 0 || q_head_stride < 0 || (num_heads > 1 && q_head_stride < width))
    return invalid("q's heads overlap, or a stride is negative");
  if (!aligned(q) || !aligned(out) || q_token_stride % 8 != 0 || q_head_stride % 8 != 0)
    return invalid("q's rows and out must start on 16-byte boundaries");
  return TOPK_SUCCESS;
}

// The launch of an absorbed call whose arguments hold; a's workspace from the caller's.
topk_status_t attend(latent::AttendArgs& a, int64_t keys, bool e4m3, void* workspace, size_t workspace_bytes,
                     hipStream_t stream) {
  if (latent::attend_threads(a.num_tokens, a.num_heads) > latent::kMaxThreads)
    return invalid("more tokens and heads than a launch has threads for");
  int cus = 0;
  const topk_status_t st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  a.wgs = split_wgs(cus, a.num_tokens, a.num_heads, keys, !a.indices, a.num_requests);
  if (a.wgs > 0) {
    const latent::SplitLayout s = latent::split_layout(a.num_tokens, a.num_heads, a.wgs);
    if (!workspace || workspace_bytes < s.total()) return invalid("the workspace is smaller than latent_attention_workspace says");
    if (!aligned(workspace)) return invalid("the workspace must start on a 16-byte boundary");
    char* p = static_cast<char*>(workspace);
    a.part_out = reinterpret_cast<float*>(p);
    a.part_ml = reinterpret_cast<float2*>(p + s.out_bytes);
    a.part_rec = reinterpret_cast<int32_t*>(p + s.out_bytes + s.ml_bytes);
  }
  char buf[160];
  std::snprintf(buf, sizeof(buf), "latent-attention %s %s waves=%d wgs=%d", a.indices ? "selected" : "paged",
                e4m3 ? "e4m3" : "bf16", latent::attend_waves(a.num_heads), a.wgs);
  return launched(latent::launch_attend(a, e4m3, stream), buf);
}

}  // namespace

extern "C" {

topk_status_t paged_append_plan(const int32_t* kv_lens, const int32_t* new_lens, int32_t* page_table,
                                const int32_t* free_pages, const int32_t* free_used, int32_t page_size,
                                int32_t* seq_lens, int32_t* q_starts, int32_t* slot_map, int32_t* positions,
                                int32_t* free_used_out, hipStream_t stream, int32_t num_requests,
                                int64_t pages_per_row, int64_t num_free, int64_t num_tokens) {
  topk::set_last_error("");
  const int log2_page = log2_of(page_size);
  if (log2_page < 0) return invalid("page_size must be a power of two");
  if (num_requests < 0 || pages_per_row < 0 || num_free < 0 || num_tokens < 0)
    return invalid("num_requests, pages_per_row, num_free and num_tokens must be >= 0");
  if (num_free > (int64_t)INT32_MAX || num_tokens > (int64_t)INT32_MAX || pages_per_row > (int64_t)INT32_MAX)
    return invalid("num_free, num_tokens and pages_per_row must fit in int32");
  if (!q_starts || !free_used_out) return invalid("q_starts and free_used_out must be non-null");
  if (free_used == free_used_out) return invalid("free_used_out must not be free_used");
  if (num_requests > 0 && (!kv_lens || !new_lens || !seq_lens)) return invalid("kv_lens, new_lens and seq_lens must be non-null");
  if (num_requests > 0 && (seq_lens == kv_lens || seq_lens == new_lens))
    return invalid("seq_lens must not be kv_lens or new_lens: other workgroups still read those");
  if (num_requests > 0 && pages_per_row > 0 && !page_table) return invalid("page_table must be non-null");
  if (num_free > 0 && !free_pages) return invalid("free_pages must be non-null");
  if (num_tokens > 0 && (!slot_map || !positions)) return invalid("slot_map and positions must be non-null");
  int cus = 0;
  const topk_status_t st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  latent::PlanArgs a{};
  a.kv_lens = kv_lens;
  a.new_lens = new_lens;
  a.page_table = page_table;
  a.free_pages = free_pages;
  a.free_used = free_used;
  a.seq_lens = seq_lens;
  a.q_starts = q_starts;
  a.slot_map = slot_map;
  a.positions = positions;
  a.free_used_out = free_used_out;
  a.pages_per_row = pages_per_row;
  a.num_free = num_free;
  a.num_tokens = num_tokens;
  a.num_requests = num_requests;
  a.log2_page = log2_page;
  return launched(latent::launch_append_plan(a, stream), "paged-append-plan");
}

topk_status_t latent_cache_store(const uint16_t* kv, int64_t kv_stride, const uint16_t* norm_weight, float eps,
                                 const int32_t* positions, const float* cos_sin, int64_t max_positions,
                                 int32_t interleaved, const int32_t* slot_map, void* latent, int64_t latent_stride,
                                 uint16_t* rope, int64_t rope_stride, float* scale, int32_t cache_type,
                                 hipStream_t stream, int64_t num_tokens, int64_t num_slots) {
  topk::set_last_error("");
  latent::Cache c{};
  topk_status_t st = check_cache(latent, latent_stride, rope, rope_stride, scale, cache_type, num_slots, &c);
  if (st != TOPK_SUCCESS) return st;
  if (num_tokens < 0 || num_tokens > (int64_t)INT32_MAX) return invalid("num_tokens must be in [0, 2^31)");
  if (num_tokens == 0) return TOPK_SUCCESS;
  if (!kv || !slot_map) return invalid("kv and slot_map must be non-null");
  if (kv_stride < LATENT_DIM + LATENT_ROPE_DIM || kv_stride % 8 != 0 || !aligned(kv))
    return invalid("kv's rows must not overlap and must start on 16-byte boundaries");
  if (norm_weight && !aligned(norm_weight)) return invalid("norm_weight must start on a 16-byte boundary");
  if (cos_sin && (!positions || max_positions < 0)) return invalid("cos_sin needs positions and max_positions >= 0");
  int cus = 0;
  st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  latent::StoreArgs a{};
  a.kv = kv;
  a.kv_stride = kv_stride;
  a.norm_weight = norm_weight;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.max_positions = max_positions;
  a.slot_map = slot_map;
  a.latent = static_cast<char*>(latent);
  a.rope = reinterpret_cast<char*>(rope);
  a.scale = scale;
  a.latent_stride = c.latent_stride;
  a.rope_stride = c.rope_stride;
  a.num_tokens = num_tokens;
  a.num_slots = num_slots;
  a.eps = eps;
  a.interleaved = interleaved;
  return launched(latent::launch_cache_store(a, cache_type == LATENT_CACHE_E4M3, stream), "latent-cache-store");
}

topk_status_t latent_cache_load(const int32_t* slots, const void* latent, int64_t latent_stride, const uint16_t* rope,
                                int64_t rope_stride, const float* scale, int32_t cache_type, uint16_t* out_latent,
                                uint16_t* out_rope, hipStream_t stream, int64_t num_rows, int64_t num_slots) {
  topk::set_last_error("");
  latent::LoadArgs a{};
  topk_status_t st = check_cache(latent, latent_stride, rope, rope_stride, scale, cache_type, num_slots, &a.cache);
  if (st != TOPK_SUCCESS) return st;
  if (num_rows < 0 || num_rows > (int64_t)INT32_MAX) return invalid("num_rows must be in [0, 2^31)");
  if (latent::load_threads(num_rows) > latent::kMaxThreads) return invalid("more rows than a launch has threads for");
  if (num_rows == 0) return TOPK_SUCCESS;
  if (!slots || !out_latent || !out_rope) return invalid("slots, out_latent and out_rope must be non-null");
  if (!aligned(out_latent) || !aligned(out_rope)) return invalid("out_latent and out_rope must start on 16-byte boundaries");
  int cus = 0;
  st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  a.slots = slots;
  a.out_latent = out_latent;
  a.out_rope = out_rope;
  a.num_rows = num_rows;
  return launched(latent::launch_cache_load(a, cache_type == LATENT_CACHE_E4M3, stream), "latent-cache-load");
}

topk_status_t latent_cache_load_paged(const int32_t* page_table, const int32_t* kv_starts, int32_t page_size,
                                      const void* latent, int64_t latent_stride, const uint16_t* rope,
                                      int64_t rope_stride, const float* scale, int32_t cache_type,
                                      uint16_t* out_latent, uint16_t* out_rope, hipStream_t stream,
                                      int32_t num_requests, int64_t pages_per_row, int64_t num_rows,
                                      int64_t num_slots) {
  topk::set_last_error("");
  latent::LoadArgs a{};
  topk_status_t st = check_cache(latent, latent_stride, rope, rope_stride, scale, cache_type, num_slots, &a.cache);
  if (st != TOPK_SUCCESS) return st;
  a.log2_page = log2_of(page_size);
  if (a.log2_page < 0) return invalid("page_size must be a power of two");
  if (num_rows < 0 || num_rows > (int64_t)INT32_MAX) return invalid("num_rows must be in [0, 2^31)");
  if (latent::load_threads(num_rows) > latent::kMaxThreads) return invalid("more rows than a launch has threads for");
  if (num_requests < 0 || pages_per_row < 0) return invalid("num_requests and pages_per_row must be >= 0");
  if (num_rows == 0 || num_requests == 0) return TOPK_SUCCESS;
  if (!kv_starts || !out_latent || !out_rope) return invalid("kv_starts, out_latent and out_rope must be non-null");
  if (pages_per_row > 0 && !page_table) return invalid("page_table must be non-null");
  if (!aligned(out_latent) || !aligned(out_rope)) return invalid("out_latent and out_rope must start on 16-byte boundaries");
  int cus = 0;
  st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  a.page_table = page_table;
  a.kv_starts = kv_starts;
  a.pages_per_row = pages_per_row;
  a.out_latent = out_latent;
  a.out_rope = out_rope;
  a.num_rows = num_rows;
  a.num_requests = num_requests;
  return launched(latent::launch_cache_load(a, cache_type == LATENT_CACHE_E4M3, stream), "latent-cache-load paged");
}

topk_status_t latent_attention_workspace(int32_t num_tokens, int32_t num_heads, int64_t keys, size_t* bytes) {
  topk::set_last_error("");
  if (!bytes) return invalid("bytes must be non-null");
  if (num_tokens < 0 || num_heads < 0 || keys < 0) return invalid("num_tokens, num_heads and keys must be >= 0");
  *bytes = 0;
  if (num_tokens == 0 || num_heads == 0) return TOPK_SUCCESS;
  int cus = 0;
  const topk_status_t st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  // Also of fewer tokens and keys, which may be split where these are not.
  const int wgs = most_wgs(cus, num_tokens, head_blocks(num_heads), bound_tiles(keys));
  *bytes = latent::split_layout(num_tokens, num_heads, wgs).total();
  return TOPK_SUCCESS;
}

topk_status_t latent_attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, const void* latent,
                               int64_t latent_stride, const uint16_t* rope, int64_t rope_stride, const float* scale,
                               int32_t cache_type, const int32_t* indices, float softmax_scale, uint16_t* out,
                               float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream,
                               int32_t num_tokens, int32_t num_heads, int64_t k, int64_t num_slots) {
  topk::set_last_error("");
  latent::AttendArgs a{};
  topk_status_t st = check_cache(latent, latent_stride, rope, rope_stride, scale, cache_type, num_slots, &a.cache);
  if (st != TOPK_SUCCESS) return st;
  st = check_queries(q, q_token_stride, q_head_stride, out, num_tokens, num_heads, LATENT_DIM + LATENT_ROPE_DIM);
  if (st != TOPK_SUCCESS) return st;
  if (k < 0 || k > (int64_t)INT32_MAX) return invalid("k must be in [0, 2^31)");
  if (num_tokens == 0 || num_heads == 0) return TOPK_SUCCESS;
  if (k > 0 && !indices) return invalid("indices must be non-null");
  a.q = q;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  // with k = 0 nothing is read through it, but it tells the two forms apart
  a.indices = indices ? indices : reinterpret_cast<const int32_t*>(q);
  a.k = k;
  a.scale_log2 = scale_log2(softmax_scale);
  a.out = out;
  a.lse = lse;
  a.num_tokens = num_tokens;
  a.num_heads = num_heads;
  return attend(a, k, cache_type == LATENT_CACHE_E4M3, workspace, workspace_bytes, stream);
}

topk_status_t latent_attention_paged(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                     const void* latent, int64_t latent_stride, const uint16_t* rope,
                                     int64_t rope_stride, const float* scale, int32_t cache_type,
                                     const int32_t* page_table, const int32_t* seq_lens, const int32_t* q_starts,
                                     int32_t page_size, float softmax_scale, uint16_t* out, float* lse,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream, int32_t num_tokens,
                                     int32_t num_heads, int32_t num_requests, int64_t pages_per_row,
                                     int64_t num_slots) {
  topk::set_last_error("");
  latent::AttendArgs a{};
  topk_status_t st = check_cache(latent, latent_stride, rope, rope_stride, scale, cache_type, num_slots, &a.cache);
  if (st != TOPK_SUCCESS) return st;
  st = check_queries(q, q_token_stride, q_head_stride, out, num_tokens, num_heads, LATENT_DIM + LATENT_ROPE_DIM);
  if (st != TOPK_SUCCESS) return st;
  a.log2_page = log2_of(page_size);
  if (a.log2_page < 0) return invalid("page_size must be a power of two");
  if (num_requests < 0 || pages_per_row < 0 || pages_per_row > (int64_t)INT32_MAX)
    return invalid("num_requests must be >= 0 and pages_per_row in [0, 2^31)");
  if (num_tokens == 0 || num_heads == 0 || num_requests == 0) return TOPK_SUCCESS;
  if (!seq_lens || !q_starts || (pages_per_row > 0 && !page_table))
    return invalid("page_table, seq_lens and q_starts must be non-null");
  a.q = q;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.q_starts = q_starts;
  a.pages_per_row = pages_per_row;
  a.num_requests = num_requests;
  a.scale_log2 = scale_log2(softmax_scale);
  a.out = out;
  a.lse = lse;
  a.num_tokens = num_tokens;
  a.num_heads = num_heads;
  return attend(a, pages_per_row * (int64_t)page_size, cache_type == LATENT_CACHE_E4M3, workspace, workspace_bytes,
                stream);
}

topk_status_t latent_attention_expanded_workspace(int32_t num_tokens, int32_t num_heads, int64_t num_kv,
                                                  int32_t num_requests, size_t* bytes) {
  topk::set_last_error("");
  if (!bytes) return invalid("bytes must be non-null");
  if (num_tokens < 0 || num_heads < 0 || num_kv < 0 || num_requests < 0)
    return invalid("num_tokens, num_heads, num_kv and num_requests must be >= 0");
  *bytes = 0;
  if (num_tokens == 0 || num_heads == 0 || num_requests == 0) return TOPK_SUCCESS;
  int cus = 0;
  const topk_status_t st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  // Also of smaller calls, which may be split where this one is not.
  if (num_kv >= kSplitKeys) *bytes = latent::prefill_split_layout(num_tokens, num_heads, num_requests, 2 * cus).total();
  return TOPK_SUCCESS;
}

topk_status_t latent_attention_expanded(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                        const uint16_t* kv_up, int64_t kv_token_stride, int64_t kv_head_stride,
                                        const uint16_t* rope, int64_t rope_stride, const int32_t* q_starts,
                                        const int32_t* kv_starts, float softmax_scale, int32_t causal, uint16_t* out,
                                        float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream,
                                        int32_t num_tokens, int64_t num_kv, int32_t num_heads, int32_t num_requests) {
  topk::set_last_error("");
  topk_status_t st =
      check_queries(q, q_token_stride, q_head_stride, out, num_tokens, num_heads, LATENT_HEAD_DIM + LATENT_ROPE_DIM);
  if (st != TOPK_SUCCESS) return st;
  if (num_kv < 0 || num_kv > (int64_t)INT32_MAX) return invalid("num_kv must be in [0, 2^31)");
  if (num_requests < 0) return invalid("num_requests must be >= 0");
  if (num_tokens == 0 || num_heads == 0 || num_requests == 0) return TOPK_SUCCESS;
  if (!q_starts || !kv_starts) return invalid("q_starts and kv_starts must be non-null");
  if (num_kv > 0 && (!kv_up || !rope)) return invalid("kv_up and rope must be non-null when num_kv > 0");
  if (num_heads > 65535) return invalid("num_heads must be at most 65535");
  if (latent::prefill_threads(num_tokens, num_heads, num_requests) > latent::kMaxThreads)
    return invalid("more tokens, requests and heads than a launch has threads for");
  if (kv_token_stride < 0 || kv_head_stride < 0 || (num_heads > 1 && kv_head_stride < 2 * LATENT_HEAD_DIM) ||
      rope_stride < LATENT_ROPE_DIM)
    return invalid("kv_up's heads or rope's rows overlap, or a stride is negative");
  if (kv_token_stride > kMaxTileStride || rope_stride > kMaxTileStride)
    return invalid("kv_up's and rope's rows must be less than 2^24 elements apart");
  if (!aligned(kv_up) || !aligned(rope) || kv_token_stride % 8 != 0 || kv_head_stride % 8 != 0 || rope_stride % 8 != 0)
    return invalid("kv_up's and rope's rows must start on 16-byte boundaries");
  int cus = 0;
  st = device_cus(&cus);
  if (st != TOPK_SUCCESS) return st;
  latent::PrefillArgs a{};
  a.q = q;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.kv = kv_up;
  a.kv_token_stride = kv_token_stride;
  a.kv_head_stride = kv_head_stride;
  a.rope = rope;
  a.rope_stride = rope_stride;
  a.q_starts = q_starts;
  a.kv_starts = kv_starts;
  a.scale_log2 = scale_log2(softmax_scale);
  a.causal = causal;
  a.out = out;
  a.lse = lse;
  a.num_tokens = num_tokens;
  a.num_kv = num_kv;
  a.num_heads = num_heads;
  a.num_requests = num_requests;
  a.wgs = prefill_wgs(cus, num_tokens, num_heads, num_kv, num_requests);
  if (a.wgs > 0) {
    const latent::SplitLayout s = latent::prefill_split_layout(num_tokens, num_heads, num_requests, a.wgs);
    if (!workspace || workspace_bytes < s.total())
      return invalid("the workspace is smaller than latent_attention_expanded_workspace says");
    if (!aligned(workspace)) return invalid("the workspace must start on a 16-byte boundary");
    char* p = static_cast<char*>(workspace);
    a.part_out = reinterpret_cast<float*>(p);
    a.part_ml = reinterpret_cast<float2*>(p + s.out_bytes);
    a.part_rec = reinterpret_cast<int32_t*>(p + s.out_bytes + s.ml_bytes);
  }
  char buf[96];
  std::snprintf(buf, sizeof(buf), "latent-attention expanded wgs=%d", a.wgs);
  return launched(latent::launch_prefill(a, stream), buf);
}

}  // extern "C"
