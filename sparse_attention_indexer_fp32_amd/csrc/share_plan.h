// Even shares of ragged work, worked out by every workgroup of a launch for itself:
// entities (requests, or groups of them) in order, each so many tiles of work,
// and workgroup number `share` takes the tiles [begin, end) of them all.  No launch
// of its own, nothing kept between calls, and no more entities than memory holds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct SharePlan {
  uint32_t total;        // tiles of all entities
  uint32_t begin, end;   // this share's
  uint32_t start;        // tiles before the entity that holds tile `begin`
  int32_t entity;        // and its number
  uint32_t wave[16];
};

// Shares of a launch: as many as there are, but `least` tiles each.  The first
// `more` take each + 1, the others `each`, in order.
struct Shares {
  uint32_t count, each, more;
  __device__ __forceinline__ Shares(uint32_t total, uint32_t most, uint32_t least) {
    const uint32_t n = total / least;
    count = n < 1 ? 1 : n < most ? n : most;
    each = total / count;
    more = total - each * count;
  }
  __device__ __forceinline__ uint32_t begin(uint32_t share) const { return share * each + (share < more ? share : more); }
  // the share that holds a tile
  __device__ __forceinline__ uint32_t owner(uint32_t tile) const {
    const uint32_t longer = more * (each + 1);
    return tile < longer ? tile / (each + 1) : more + (tile - longer) / each;
  }
};

// weight(e): tiles of entity e; their sum is below 2^32.  Called by all threads of a
// workgroup of THREADS; returns with `plan` filled (and a barrier passed), begin == end for
// a share that has none.
template <int THREADS, typename Weight>
__device__ __forceinline__ void plan_shares(Weight weight, int entities, uint32_t share, uint32_t most, uint32_t least,
                                            SharePlan& plan) {
  constexpr int kWaves = THREADS / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t first = tid < entities ? weight(tid) : 0;
  uint32_t sum = first;
  for (int e = tid + THREADS; e < entities; e += THREADS) sum += weight(e);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) plan.wave[wave] = sum;
  __syncthreads();
  uint32_t total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) total += plan.wave[w];
  const Shares shares(total, most, least);
  const bool any = total > 0 && share < shares.count;
  const uint32_t begin = any ? shares.begin(share) : 0, end = any ? shares.begin(share + 1) : 0;
  if (tid == 0) {
    plan.total = total;
    plan.begin = begin;
    plan.end = end;
    plan.start = 0;
    plan.entity = 0;
  }
  uint32_t before = 0;
  for (int base = 0; begin < end && before <= begin && base < entities; base += THREADS) {
    __syncthreads();
    const int e = base + tid;
    const uint32_t own = base == 0 ? first : (e < entities ? weight(e) : 0);
    uint32_t incl = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 63) plan.wave[wave] = incl;
    __syncthreads();
    uint32_t all = 0, at = before + incl - own;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) at += plan.wave[w];
      all += plan.wave[w];
    }
    if (at <= begin && begin < at + own) {
      plan.start = at;
      plan.entity = e;
    }
    before += all;
  }
  __syncthreads();
}

// The first entity from `e` on that has tiles (wave-uniform; there is one): 64 at a time.
template <typename Weight>
__device__ __forceinline__ int next_entity(Weight weight, int e, int entities) {
  const int lane = threadIdx.x & 63;
  for (; e < entities; e += 64) {
    const uint64_t any = __ballot(e + lane < entities && weight(e + lane) > 0);
    if (any) return e + (int)__builtin_ctzll(any);
  }
  return entities;
}
