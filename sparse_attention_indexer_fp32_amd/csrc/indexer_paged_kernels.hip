// Scores of new tokens against their requests' paged index keys on gfx950:
//
//   score[t, j] = s[j] sum_h w[t, h] relu(q[t, h, :] . k[j, :])
//
// for the positions j that token t sees, H = 32 heads of D = 128, in bf16 on the matrix
// cores from fp8 codes (exact), summed in fp32: the same values as the scores over
// contiguous keys.
//
// A wave holds the queries of kRows tokens of a request in registers and takes 32 keys at a
// time straight from the cache, 64 bytes a lane (half a key), two tiles ahead: with
// few tokens a request every key is used by one wave, and nothing is gained by
// way of LDS.  A workgroup's four waves take 128 neighbouring keys, a tile; the
// workgroups share all requests' tiles evenly.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "indexer_device.h"
#include "indexer_paged_internal.h"
#include "share_plan.h"

namespace indexer {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kWaveKeys = 32;
constexpr int kTileKeys = kWaves * kWaveKeys;

__device__ __attribute__((aligned(16))) const uint8_t kNoKey[kDim] = {};

// A request's tokens and keys.
struct Request {
  int32_t q0, q1;        // its rows of q
  int32_t end;           // the same, before it was cut to the rows there are
  int64_t len;           // cached positions
  int64_t keys;          // those that are scored for some row
};
__device__ __forceinline__ Request request_of(const PagedLogitsArgs& a, int b) {
  Request r;
  r.q0 = a.q_starts[b];
  r.end = a.q_starts[b + 1];
  r.q1 = r.end < a.num_tokens ? r.end : a.num_tokens;
  r.len = a.seq_lens[b];
  r.keys = r.len < 0 ? 0 : (r.len < a.most_keys ? r.len : a.most_keys);
  return r;
}
__device__ __forceinline__ int64_t row_len(const PagedLogitsArgs& a, const Request& r, int t) {
  const int64_t n = r.len - (r.end - t) + 1;
  return n < 0 ? 0 : (n < a.most_keys ? n : a.most_keys);
}

template <int R>
__device__ __forceinline__ uint32_t tiles_of(const Request& r) {
  return r.keys > 0 ? (uint32_t)((r.keys + kTileKeys - 1) / kTileKeys) : 1;   // one at least: somebody writes lens
}
template <int R>
__device__ __forceinline__ uint32_t weight_of(const PagedLogitsArgs& a, int b) {
  const Request r = request_of(a, b);
  if (r.q0 < 0 || r.q1 <= r.q0) return 0;
  return (uint32_t)((r.q1 - r.q0 + R - 1) / R) * tiles_of<R>(r);
}

// A lane's half of a key as it was loaded.
struct KeyRegs {
  uint4 v[4];
  float scale;
};

template <int R>
__global__ __launch_bounds__(kThreads, R == 1 ? 4 : 2) void paged_logits_kernel(PagedLogitsArgs a, uint32_t most) {
  __shared__ SharePlan plan;
  const PagedKeys& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, hb = lane >> 5;
  // neighbouring shares on one XCD, whose L2 then holds the keys that they have in common
  const uint32_t per = (gridDim.x + 7) / 8, share = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  auto weight = [&](int b) { return weight_of<R>(a, b); };
  plan_shares<kThreads>(weight, c.num_requests, (blockIdx.x >> 3) < per ? share : most, most, 1, plan);
  uint32_t lo = __builtin_amdgcn_readfirstlane(plan.begin), hi = __builtin_amdgcn_readfirstlane(plan.end);
  uint32_t start = __builtin_amdgcn_readfirstlane(plan.start);
  int b = __builtin_amdgcn_readfirstlane(plan.entity);

  // rows behind the last request
  if (a.lens) {
    const int last = a.q_starts[c.num_requests];
    for (int64_t t = (last < 0 ? 0 : last) + (int64_t)blockIdx.x * kThreads + tid; t < a.num_tokens; t += (int64_t)gridDim.x * kThreads)
      a.lens[t] = 0;
  }

  while (lo < hi) {
    const Request r = request_of(a, b);
    const uint32_t tiles = tiles_of<R>(r), blocks = (uint32_t)((r.q1 - r.q0 + R - 1) / R);
    const uint32_t block = (lo - start) / tiles, begin = start + block * tiles;
    const uint32_t first = lo - begin, last = hi - begin < tiles ? hi - begin : tiles;
    const int t0 = r.q0 + (int)block * R;
    RowOperand rows[R];
    int64_t len[R];
    int64_t most_len = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool live = t0 + i < r.q1;
      load_row(a.q, a.weights, live ? t0 + i : t0, true, lane, rows[i]);
      len[i] = live ? row_len(a, r, t0 + i) : 0;
      most_len = len[i] > most_len ? len[i] : most_len;
      if (a.lens && first == 0 && tid == 0 && live) a.lens[t0 + i] = (int32_t)len[i];
    }
    const int32_t* pages = c.page_table + (int64_t)b * c.pages_per_row;
    const int64_t page_mask = ((int64_t)1 << c.log2_page) - 1;
    auto position = [&](uint32_t tile) { return (int64_t)tile * kTileKeys + wave * kWaveKeys + n; };
    // the page of this lane's key (of the last one's, past them)
    auto page_of = [&](uint32_t tile) {
      int64_t j = position(tile);
      j = j < most_len ? j : most_len - 1;
      return pages[j >> c.log2_page];
    };
    auto slot_of = [&](uint32_t tile, int32_t page) {
      int64_t j = position(tile);
      j = j < most_len ? j : most_len - 1;
      const int64_t slot = ((int64_t)page << c.log2_page) + (j & page_mask);
      return page >= 0 && slot < c.num_slots ? (int32_t)slot : -1;
    };
    auto fetch = [&](int32_t slot, KeyRegs& k) {
      const uint8_t* row = slot >= 0 ? c.keys + (int64_t)slot * c.key_stride : kNoKey;
      const uint4* src = reinterpret_cast<const uint4*>(row + hb * 64);
#pragma unroll
      for (int i = 0; i < 4; ++i) k.v[i] = src[i];
      k.scale = *(slot >= 0 ? c.scale + slot : reinterpret_cast<const float*>(kNoKey));
    };
    auto compute = [&](uint32_t tile, const KeyRegs& k, int32_t slot) {
      bf16x8 key[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        key[2 * i] = widen8(k.v[i].x, k.v[i].y);
        key[2 * i + 1] = widen8(k.v[i].z, k.v[i].w);
      }
      const int64_t j = position(tile);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        f32x16 acc = {};
#pragma unroll
        for (int s = 0; s < 8; ++s) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(rows[i].a[s], key[s], acc, 0, 0, 0);
        float score = finish_score(rows[i], acc, k.scale, lane);
        if (slot < 0) score = -INFINITY;
        if (hb == 0 && j < len[i]) a.logits[(int64_t)(t0 + i) * a.width + j] = score;
      }
    };
    // keys of the rows' own range only: the last block's rows see more than the first's
    const uint32_t used = (uint32_t)((most_len + kTileKeys - 1) / kTileKeys), stop = last < used ? last : used;
    if (first < stop) {
      KeyRegs k0, k1;
      int32_t s0, s1, p;
      s0 = slot_of(first, page_of(first));
      fetch(s0, k0);
      const uint32_t top = stop - 1;
      s1 = slot_of(first + 1 < top ? first + 1 : top, page_of(first + 1 < top ? first + 1 : top));
      fetch(s1, k1);
      p = page_of(first + 2 < top ? first + 2 : top);
      for (uint32_t i = first; i < stop; i += 2) {
        compute(i, k0, s0);
        const uint32_t n2 = i + 2 < top ? i + 2 : top, n3 = i + 3 < top ? i + 3 : top, n4 = i + 4 < top ? i + 4 : top;
        s0 = slot_of(n2, p);
        fetch(s0, k0);
        p = page_of(n3);
        if (i + 1 < stop) compute(i + 1, k1, s1);
        s1 = slot_of(n3, p);
        fetch(s1, k1);
        p = page_of(n4);
      }
    }
    lo = begin + last;
    if (block + 1 == blocks && lo == begin + tiles) {
      start += blocks * tiles;
      if (lo < hi) b = next_entity(weight, b + 1, c.num_requests);
    }
  }
}

}  // namespace

hipError_t launch_paged_logits(const PagedLogitsArgs& a, int cus, hipStream_t stream) {
  // one token a request and less: one row a wave
  const bool single = a.num_tokens <= a.cache.num_requests;
  const int64_t tiles = (int64_t)a.num_tokens * (a.most_keys / kTileKeys + 1);
  const int64_t most = (int64_t)cus * (single ? 4 : 2);
  const unsigned wgs = (unsigned)((tiles < most ? tiles : most) + 7) / 8 * 8;
  if (single)
    hipLaunchKernelGGL(paged_logits_kernel<1>, dim3(wgs), dim3(kThreads), 0, stream, a, wgs);
  else
    hipLaunchKernelGGL(paged_logits_kernel<2>, dim3(wgs), dim3(kThreads), 0, stream, a, wgs);
  return hipGetLastError();
}

}  // namespace indexer
