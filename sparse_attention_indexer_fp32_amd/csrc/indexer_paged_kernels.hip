// Scores of new tokens against their requests' paged index keys on gfx950:
//
//   score[t, j] = s[j] sum_h w[t, h] relu(q[t, h, :] . k[j, :])
//
// for the positions j that token t sees, H = 32 heads of D = 128, in bf16 on the matrix
// cores from fp8 codes (exact), summed in fp32: the same values as the scores over
// contiguous keys.  Two kernels, by the tokens that a request has on average:
//   * few: a key is used by one wave, which streams keys and holds one token's
//     queries, or two tokens'; HBM bounds it;
//   * many: a workgroup holds eight tokens' queries, and stages keys in LDS for all
//     of them; the matrix cores bound it.
// In both the workgroups share all requests' tiles evenly.
//
// Measured (MI355X), 64-position pages: one token of each of 64 requests behind 4096 to 65536 keys
// 56-60 us, 5.1-5.4 TB/s (a loop that only reads the same bytes: 44-50); one token behind 2^20 keys 26
// us, 5.4 TB/s; 1024 tokens behind 65536 keys 447-496 us, 1110-1230 TFLOP/s, which is what a large
// library matrix product reaches less 10-20 %.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "indexer_device.h"
#include "indexer_paged_internal.h"
#include "latent_device.h"
#include "share_plan.h"

namespace indexer {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kWaveKeys = 32;

__device__ __attribute__((aligned(16))) const uint8_t kNoKey[kDim] = {};

// A request's tokens and keys.
struct Request {
  int32_t q0, q1;        // its rows of q
  int32_t end;           // the same, before it was cut to the rows there are
  int32_t len;           // cached positions
  int32_t keys;          // those that are scored for some row
};
__device__ __forceinline__ Request request_of(const PagedLogitsArgs& a, int b) {
  Request r;
  r.q0 = a.q_starts[b];
  r.end = a.q_starts[b + 1];
  r.q1 = r.end < a.num_tokens ? r.end : a.num_tokens;
  r.len = a.seq_lens[b];
  r.keys = r.len < 0 ? 0 : ((int64_t)r.len < a.most_keys ? r.len : (int32_t)a.most_keys);
  return r;
}
__device__ __forceinline__ int32_t row_len(const PagedLogitsArgs& a, const Request& r, int t) {
  const int64_t n = (int64_t)r.len - (r.end - t) + 1;
  return (int32_t)(n < 0 ? 0 : (n < a.most_keys ? n : a.most_keys));
}

// A request's tiles of KEYS keys: one at least, so that somebody writes its rows' lens.
template <int KEYS>
__device__ __forceinline__ uint32_t tiles_of(const Request& r) {
  return r.keys > 0 ? (uint32_t)(r.keys + KEYS - 1) / KEYS : 1;
}
template <int ROWS, int KEYS>
__device__ __forceinline__ uint32_t weight_of(const PagedLogitsArgs& a, int b) {
  const Request r = request_of(a, b);
  if (r.q0 < 0 || r.q1 <= r.q0) return 0;
  return (uint32_t)((r.q1 - r.q0 + ROWS - 1) / ROWS) * tiles_of<KEYS>(r);
}

// Rows behind the last request see nothing.
__device__ __forceinline__ void clear_lens(const PagedLogitsArgs& a) {
  if (!a.lens) return;
  const int last = a.q_starts[a.cache.num_requests];
  for (int64_t t = (last < 0 ? 0 : last) + (int64_t)blockIdx.x * kThreads + threadIdx.x; t < a.num_tokens; t += (int64_t)gridDim.x * kThreads)
    a.lens[t] = 0;
}

// The slot of position j, whose page is `page`, or -1.
__device__ __forceinline__ int32_t slot_of(const PagedKeys& c, int32_t j, int32_t page) {
  const int64_t slot = ((int64_t)page << c.log2_page) + (j & ((1 << c.log2_page) - 1));
  return page >= 0 && slot < c.num_slots ? (int32_t)slot : -1;
}

// A row of the scores as a buffer: what is stored beyond its `len` is dropped, so stores
// need no branch, which would part them from the arithmetic around them.  (Its size in bytes, and every
// offset below kDropped, fit 31 bits: rows are shorter than 2^29.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t score_row(const PagedLogitsArgs& a, int64_t t, int32_t len) {
  return __builtin_amdgcn_make_buffer_rsrc(a.logits + t * a.width, 0, len * 4, 0x00027000);
}
constexpr uint32_t kDropped = 0xFFFFFFFCu;

// ---- few tokens a request ---------------------------------------------------------------------

// A workgroup's waves take 32 keys each of a tile of 128.  Keys go straight to LDS, in a ring of the
// wave's own, kDepth tiles ahead and without a barrier: eight keys an instruction, whole rows.  (Loaded
// to registers as the matrix instruction takes them, 16 of a row's bytes an instruction, 64 requests of
// 34816 keys took 71 us against 60.)  WHOLE: every tile of 32 keys lies in one page, and so in one
// piece of memory that the cache either holds or does not: one scalar address for all of its loads
// (with an address a key 63 us).
constexpr int kDepth = 2;
constexpr int kFewTile = kWaves * kWaveKeys;
constexpr int kKeyBytes = kWaveKeys * kDim;
constexpr int kWordBytes = kWaveKeys * 4;
constexpr int kStageBytes = kKeyBytes + 3 * kWordBytes;             // keys, scales; biases, pages (not WHOLE)
constexpr int kRingBytes = kDepth * kStageBytes;

constexpr int64_t kMaxWholeStride = 1 << 26;    // a tile's offsets take 32 bits

// A key's 16-byte chunk c lies at chunk c ^ (key / 2 % 8) of its row: the 16 keys that are read
// together, two rows to 256 bytes, then fall in different banks.
__device__ __forceinline__ int key_swizzle(int key) { return (key >> 1) & 7; }

template <int R, bool WHOLE>
__global__ __launch_bounds__(kThreads, R == 1 ? 4 : 2) void few_logits_kernel(PagedLogitsArgs a, uint32_t most) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const PagedKeys& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, hb = lane >> 5;
  const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds + wave * kRingBytes;
  SharePlan& plan = *reinterpret_cast<SharePlan*>(lds);
  auto weight = [&](int b) { return weight_of<R, kFewTile>(a, b); };
  plan_shares<kThreads>(weight, c.num_requests, blockIdx.x, most, 1, plan);
  uint32_t lo = __builtin_amdgcn_readfirstlane(plan.begin), start = __builtin_amdgcn_readfirstlane(plan.start);
  const uint32_t hi = __builtin_amdgcn_readfirstlane(plan.end);
  int b = __builtin_amdgcn_readfirstlane(plan.entity);
  __syncthreads();                        // the plan lay where the keys go
  clear_lens(a);
  // offsets of a lane's loads within a tile of consecutive keys: key 8 k + lane / 8, its chunk of 16 bytes
  uint32_t offset[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int key = 8 * k + (lane >> 3);
    offset[k] = (uint32_t)key * (uint32_t)c.key_stride + (((lane & 7) ^ key_swizzle(key)) << 4);
  }

  while (lo < hi) {
    const Request r = request_of(a, b);
    const uint32_t tiles = tiles_of<kFewTile>(r), blocks = (uint32_t)((r.q1 - r.q0 + R - 1) / R);
    const uint32_t block = (lo - start) / tiles, begin = start + block * tiles;
    const uint32_t first = lo - begin, last = hi - begin < tiles ? hi - begin : tiles;
    const int t0 = r.q0 + (int)block * R;
    __amdgpu_buffer_rsrc_t out[R];
    int32_t most_len = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool live = t0 + i < r.q1;
      const int t = live ? t0 + i : t0;
      const int32_t len = live ? row_len(a, r, t) : 0;
      most_len = len > most_len ? len : most_len;
      out[i] = score_row(a, t, len);
      if (a.lens && first == 0 && tid == 0 && live) a.lens[t] = len;
    }
    const uint32_t used = (uint32_t)(most_len + kFewTile - 1) / kFewTile, stop = last < used ? last : used;
    const int32_t from = (int32_t)first * kFewTile + wave * kWaveKeys;
    // this wave's tiles: 32 keys of each, but for a last one that ends before them
    const int count = from < most_len ? ((int)(stop - first) - 1) + ((int32_t)(stop - 1) * kFewTile + wave * kWaveKeys < most_len) : 0;
    if (first < stop && count > 0) {
      const int32_t* pages = c.page_table + (int64_t)b * c.pages_per_row;
      auto position = [&](int i) { return from + i * kFewTile + n; };
      // WHOLE: the page of a tile (past the last tile, of that one)
      auto tile_page = [&](int i) {
        typedef const __attribute__((address_space(4))) int32_t* scalar_ptr;
        return ((scalar_ptr)pages)[(from + (i < count ? i : count - 1) * kFewTile) >> c.log2_page];
      };
      // otherwise: the pages of its keys
      auto load_pages = [&](int i, uint32_t stage) {
        int32_t j = position(i < count ? i : count - 1);
        j = j < most_len ? j : most_len - 1;
        latent::queue_words_to_lds(pages + (j >> c.log2_page), stage + kKeyBytes + 2 * kWordBytes);
      };
      // WHOLE: the tile's first slot, or -1
      auto tile_slot = [&](int i, int32_t page) {
        return slot_of(c, from + (i < count ? i : count - 1) * kFewTile, page);
      };
      auto load_keys = [&](int i, int32_t page, uint32_t stage) {
        if constexpr (WHOLE) {
          const int32_t slot = tile_slot(i, page), at = slot < 0 || i >= count ? 0 : slot;
          const uint8_t* keys = c.keys + (int64_t)at * c.key_stride;
#pragma unroll
          for (int k = 0; k < 4; ++k) latent::stream_to_lds(keys, offset[k], stage + 1024 * k);
          latent::queue_words_to_lds(c.scale + at + n, stage + kKeyBytes);
        } else {
          const int32_t own = latent::read_lds<int32_t>(stage + kKeyBytes + 2 * kWordBytes + n * 4);
          const int32_t j = position(i), slot = i < count && j < most_len ? slot_of(c, j, own) : -1;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = 8 * k + (lane >> 3);
            const int32_t s = __builtin_amdgcn_ds_bpermute(key * 4, slot);
            const uint8_t* row = s >= 0 ? c.keys + (int64_t)s * c.key_stride : kNoKey;
            latent::stream_row_to_lds(row + (((lane & 7) ^ key_swizzle(key)) << 4), stage + 1024 * k);
          }
          latent::queue_words_to_lds(slot >= 0 ? c.scale + slot : reinterpret_cast<const float*>(kNoKey), stage + kKeyBytes);
          typedef __attribute__((address_space(3))) float* lds_ptr;
          if (lane < 32) *(lds_ptr)(stage + kKeyBytes + kWordBytes + n * 4) = slot >= 0 ? 0.f : -INFINITY;
        }
      };
      int32_t page[kDepth + 1];           // WHOLE: of the tiles whose keys are on their way, and of the next one
#pragma unroll
      for (int d = 0; d <= kDepth; ++d) page[d] = WHOLE ? tile_page(d) : 0;
      if (!WHOLE) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) load_pages(d, ring + d * kStageBytes);
      }
      RowOperand rows[R];
#pragma unroll
      for (int i = 0; i < R; ++i) load_row(a.q, a.weights, t0 + i < r.q1 ? t0 + i : t0, true, lane, rows[i]);
      // from here on only the ring's loads are in flight: the queries are there too
      latent::wait_loads<0>();
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) asm volatile("" : "+v"(rows[i].w[k]));
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const uint32_t stage = ring + d * kStageBytes;
        load_keys(d, page[d], stage);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (!WHOLE) load_pages(d + kDepth, stage);
        // (stores, dropped, so that every tile is behind as many operations as any other)
#pragma unroll
        for (int k = 0; k < R; ++k) __builtin_amdgcn_raw_buffer_store_b32(0, out[k], kDropped, 0, 0);
      }
      uint32_t stage = ring;
      for (int i = 0; i < count; ++i) {
        // Behind tile i's loads: its stores, and kDepth - 1 tiles' loads and stores.  The pages of
        // tile i + kDepth (not WHOLE), loaded behind tile i's keys, have to be there as well.
        constexpr int kLoads = WHOLE ? 5 : 6;
        latent::wait_loads<(kDepth - 1) * (kLoads + R) + R>();
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
          v[k] = __builtin_bit_cast(uint4, latent::read_lds<u32x4>(stage + n * kDim + (((hb * 4 + k) ^ key_swizzle(n)) << 4)));
        }
        const float scale = latent::read_lds<float>(stage + kKeyBytes + n * 4);
        const float bias = WHOLE ? (tile_slot(i, page[0]) < 0 ? -INFINITY : 0.f)
                                 : latent::read_lds<float>(stage + kKeyBytes + kWordBytes + n * 4);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");        // read: the stage is free
        load_keys(i + kDepth, page[kDepth], stage);
        if (WHOLE) {
#pragma unroll
          for (int d = 0; d < kDepth; ++d) page[d] = page[d + 1];
          page[kDepth] = tile_page(i + 1 + kDepth);
        } else {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          load_pages(i + 2 * kDepth, stage);
        }
        bf16x8 key[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          key[2 * k] = widen8(v[k].x, v[k].y);
          key[2 * k + 1] = widen8(v[k].z, v[k].w);
        }
        const uint32_t at = hb == 0 ? (uint32_t)position(i) * 4 : kDropped;
#pragma unroll
        for (int k = 0; k < R; ++k) {
          f32x16 acc = {};
#pragma unroll
          for (int s = 0; s < 8; ++s) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(rows[k].a[s], key[s], acc, 0, 0, 0);
          // (a key that is not there is scaled by 0, or by a number where its place holds one)
          const float score = bias < 0.f ? -INFINITY : finish_score(rows[k], acc, scale, lane);
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(score), out[k], at, 0, 0);
        }
        stage = stage + kStageBytes < ring + kRingBytes ? stage + kStageBytes : ring;
      }
      latent::wait_loads<0>();            // nothing is on its way to the ring any more
    }
    lo = begin + last;
    if (block + 1 == blocks && lo == begin + tiles) {
      start += blocks * tiles;
      if (lo < hi) b = __builtin_amdgcn_readfirstlane(next_entity(weight, b + 1, c.num_requests));
    }
  }
}

// ---- many tokens a request --------------------------------------------------------------------

// A wave holds the queries of two tokens.  64 keys at a time are loaded by all threads
// (two stages ahead, in registers), widened to bf16 into LDS (two buffers) and read by
// every wave.  The relu, the head weights and the sum over heads take as many vector instructions as the
// matrix cores have time for: those of a tile of 32 keys are laid between the
// matrix instructions of the next, so that a wave keeps both busy by itself.
constexpr int kManyRows = 2;              // of a wave
constexpr int kManyBlock = kWaves * kManyRows;
constexpr int kManyTile = 64;
constexpr int kBufferBytes = kManyTile * kDim * 2;

// LDS byte offset of 16-byte chunk c (0..15) of position n's bf16 row.
__device__ __forceinline__ int tile_offset(int n, int c) { return n * (kDim * 2) + ((c ^ (n & 15)) << 4); }

// A score, or -inf where the key is not there, whatever the product of nothing came to.  (A choice by bits, one
// instruction: a comparison became a branch around the arithmetic.)
__device__ __forceinline__ uint32_t score_bits(float score, uint32_t there) {
  return (__float_as_uint(score) & there) | (0xFF800000u & ~there);
}

__global__ __launch_bounds__(kThreads, 2) void many_logits_kernel(PagedLogitsArgs a, uint32_t most) {
  __shared__ SharePlan plan;
  __shared__ __attribute__((aligned(16))) char buffers[2 * kBufferBytes];
  __shared__ uint2 scale_there[2][kManyTile];      // a key's scale, and all ones in the bits or none: is it there?
  const PagedKeys& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, hb = lane >> 5;
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)buffers;
  // neighbouring shares on one XCD, whose L2 then holds the keys that they have in common
  const uint32_t per = gridDim.x / 8, share = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  auto weight = [&](int b) { return weight_of<kManyBlock, kManyTile>(a, b); };
  plan_shares<kThreads>(weight, c.num_requests, share, most, 1, plan);
  uint32_t lo = __builtin_amdgcn_readfirstlane(plan.begin), start = __builtin_amdgcn_readfirstlane(plan.start);
  const uint32_t hi = __builtin_amdgcn_readfirstlane(plan.end);
  int b = __builtin_amdgcn_readfirstlane(plan.entity);
  clear_lens(a);

  while (lo < hi) {
    const Request r = request_of(a, b);
    const uint32_t tiles = tiles_of<kManyTile>(r), blocks = (uint32_t)((r.q1 - r.q0 + kManyBlock - 1) / kManyBlock);
    const uint32_t block = (lo - start) / tiles, begin = start + block * tiles;
    const uint32_t first = lo - begin, last = hi - begin < tiles ? hi - begin : tiles;
    const int t0 = r.q0 + (int)block * kManyBlock + wave * kManyRows;
    RowOperand rows[kManyRows];
    __amdgpu_buffer_rsrc_t out[kManyRows];
#pragma unroll
    for (int i = 0; i < kManyRows; ++i) {
      const bool live = t0 + i < r.q1;
      const int t = live ? t0 + i : r.q1 - 1;
      load_row(a.q, a.weights, t, true, lane, rows[i]);
      const int32_t len = live ? row_len(a, r, t) : 0;
      out[i] = score_row(a, t, len);
      if (a.lens && first == 0 && lane == 0 && live) a.lens[t] = len;
    }
    // the longest row of the workgroup's, and of the wave's own
    const int end_row = r.q0 + (int)(block + 1) * kManyBlock < r.q1 ? r.q0 + (int)(block + 1) * kManyBlock : r.q1;
    const int32_t most_len = row_len(a, r, end_row - 1);
    const bool live_wave = t0 < r.q1;
    const uint32_t used = (uint32_t)(most_len + kManyTile - 1) / kManyTile, stop = last < used ? last : used;
    if (first < stop) {
      const int32_t* pages = c.page_table + (int64_t)b * c.pages_per_row;
      // a thread loads 32 bytes of a key
      const int sn = tid >> 2, sc = tid & 3;
      struct Loaded {
        uint4 r0, r1;
        float scale;
        uint32_t there;
      };
      auto key_position = [&](uint32_t tile) {
        const int32_t j = (int32_t)((tile < stop ? tile : stop - 1) * kManyTile) + sn;
        return j < most_len ? j : most_len - 1;
      };
      auto page_of = [&](uint32_t tile) { return pages[key_position(tile) >> c.log2_page]; };
      auto fetch = [&](Loaded& v, uint32_t tile, int32_t page) {
        const int32_t slot = slot_of(c, key_position(tile), page);
        const uint4* src = reinterpret_cast<const uint4*>((slot >= 0 ? c.keys + (int64_t)slot * c.key_stride : kNoKey) + sc * 32);
        v.r0 = src[0];
        v.r1 = src[1];
        v.scale = *(slot >= 0 ? c.scale + slot : reinterpret_cast<const float*>(kNoKey));
        v.there = slot >= 0 ? 0xFFFFFFFFu : 0u;
      };
      auto stage = [&](const Loaded& v, int buf) {
        char* t = buffers + buf * kBufferBytes;
        *reinterpret_cast<bf16x8*>(t + tile_offset(sn, 4 * sc)) = widen8(v.r0.x, v.r0.y);
        *reinterpret_cast<bf16x8*>(t + tile_offset(sn, 4 * sc + 1)) = widen8(v.r0.z, v.r0.w);
        *reinterpret_cast<bf16x8*>(t + tile_offset(sn, 4 * sc + 2)) = widen8(v.r1.x, v.r1.y);
        *reinterpret_cast<bf16x8*>(t + tile_offset(sn, 4 * sc + 3)) = widen8(v.r1.z, v.r1.w);
        if (sc == 0) scale_there[buf][sn] = make_uint2(__float_as_uint(v.scale), v.there);
      };
      f32x16 acc[2][kManyRows] = {};      // of the tile being multiplied, and of the one before
      uint2 st = make_uint2(0, 0);        // of the one before: the lane's key's scale, whether it is there, and where its score goes
      uint32_t at = kDropped;
      auto multiply = [&](int buf, int half, uint32_t position, bool finish) {
        f32x16(&now)[kManyRows] = acc[half];
        f32x16(&before)[kManyRows] = acc[half ^ 1];
        const int nb = half * kWaveKeys + n;
        bf16x8 key[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) key[s] = latent::read_lds<bf16x8>(base + buf * kBufferBytes + tile_offset(nb, hb * 8 + s));
#pragma unroll
        for (int i = 0; i < kManyRows; ++i) now[i] = f32x16{};
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int i = 0; i < kManyRows; ++i) now[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(rows[i].a[s], key[s], now[i], 0, 0, 0);
        if (finish) {
#pragma unroll
          for (int i = 0; i < kManyRows; ++i) {
            __builtin_amdgcn_raw_buffer_store_b32(score_bits(finish_score(rows[i], before[i], __uint_as_float(st.x), lane), st.y), out[i], at, 0, 0);
          }
        }
        st = scale_there[buf][nb];
        at = hb == 0 ? position * 4 : kDropped;
      };
      Loaded l0, l1;
      fetch(l0, first, page_of(first));
      fetch(l1, first + 1, page_of(first + 1));
      int32_t p = page_of(first + 2);
      __syncthreads();                    // the last block's reads are done
      stage(l0, 0);
      fetch(l0, first + 2, p);
      p = page_of(first + 3);
      __syncthreads();
      for (uint32_t i = first; i < stop; i += 2) {
        if (live_wave) {
          multiply(0, 0, i * kManyTile + n, true);
          multiply(0, 1, i * kManyTile + kWaveKeys + n, true);
        }
        stage(l1, 1);
        fetch(l1, i + 3, p);
        p = page_of(i + 4);
        __syncthreads();
        if (live_wave && i + 1 < stop) {
          multiply(1, 0, (i + 1) * kManyTile + n, true);
          multiply(1, 1, (i + 1) * kManyTile + kWaveKeys + n, true);
        }
        stage(l0, 0);
        fetch(l0, i + 4, p);
        p = page_of(i + 5);
        __syncthreads();
      }
      // the last tile's scores
#pragma unroll
      for (int i = 0; i < kManyRows; ++i) {
        __builtin_amdgcn_raw_buffer_store_b32(score_bits(finish_score(rows[i], acc[1][i], __uint_as_float(st.x), lane), st.y), out[i], at, 0, 0);
      }
    }
    lo = begin + last;
    if (block + 1 == blocks && lo == begin + tiles) {
      start += blocks * tiles;
      if (lo < hi) b = __builtin_amdgcn_readfirstlane(next_entity(weight, b + 1, c.num_requests));
    }
  }
}

template <int R>
void launch_few(const PagedLogitsArgs& a, unsigned wgs, hipStream_t stream) {
  const bool whole = (1 << a.cache.log2_page) % kWaveKeys == 0 && a.cache.num_slots > 0 && a.cache.num_slots % kWaveKeys == 0 &&
                     a.cache.key_stride <= kMaxWholeStride;
  constexpr int kLds = kWaves * kRingBytes;
  if (whole)
    hipLaunchKernelGGL((few_logits_kernel<R, true>), dim3(wgs), dim3(kThreads), kLds, stream, a, wgs);
  else
    hipLaunchKernelGGL((few_logits_kernel<R, false>), dim3(wgs), dim3(kThreads), kLds, stream, a, wgs);
}

}  // namespace

hipError_t launch_paged_logits(const PagedLogitsArgs& a, int cus, hipStream_t stream) {
  // By the tokens of a request, on average: one, two, more.  64 requests behind 34816 keys, in us:
  //   tokens of a request            1      2      3      4      8
  //   few, a token at a time        58     90    162    189    406
  //   few, two tokens at a time     64     63    120    122    241
  //   many                          95     92    114    114    150
  // (with three tokens the last two are within a sixth of each other elsewhere: 16 such requests 28 and 34, one
  // behind a million keys 57 and 60, 200 behind 1000 to 20000 118 and 114)
  // The average is all that the host knows.  Where it misleads: 512 tokens of one request and one of each of 63
  // others 252 us (137 and 54 in calls of their own); 64 tokens of one beside 63 requests without any 33 (alone 29), 1000
  // behind 16384 keys beside 999 short ones without any 231 (alone 124); 512 and one each of 511, behind 4096 keys, 78
  // (77 in two calls).
  const int64_t tokens = a.num_tokens, requests = a.cache.num_requests;
  const int form = tokens <= requests ? 1 : (tokens <= 2 * requests ? 2 : 3);
  const int64_t tiles = tokens * (a.most_keys / (form < 3 ? kFewTile : kManyTile) + 1), most = (form == 1 ? 4 : 2) * (int64_t)cus;
  const unsigned wgs = (unsigned)((tiles < most ? tiles : most) + 7) / 8 * 8;
  if (form == 1)
    launch_few<1>(a, wgs, stream);
  else if (form == 2)
    launch_few<2>(a, wgs, stream);
  else
    hipLaunchKernelGGL(many_logits_kernel, dim3(wgs), dim3(kThreads), 0, stream, a, wgs);
  return hipGetLastError();
}

}  // namespace indexer
