// What the absorbed attention kernels share: the layout of a ring of tiles in LDS,
// the loads that fill it, and the two products of a tile.  attend_kernels.hip
// describes the tiling.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "latent_device.h"
#include "latent_internal.h"

namespace latent {
namespace {

constexpr int kHeads = 16;                   // heads of a wave
constexpr int kLatentSteps = kLatent / 32;   // 16 steps of the first product
constexpr int kRopeSteps = kRope / 32;       // and 2 of the rotary part
constexpr int kColBlocks = kLatent / 16;     // 32 blocks of O^T
constexpr int kReadsAhead = 4;               // LDS reads in flight before a matrix instruction
constexpr int kRowBytes = kLatent * 2;       // a bf16 row in LDS
constexpr int kRopeBytes = kRope * 2;
constexpr int kTileLatent = kTileKeys * kRowBytes;
constexpr int kTileCodes = kTileKeys * kLatent;
constexpr int kTileRope = kTileKeys * kRopeBytes;

__device__ __attribute__((aligned(16))) const char kZeroRow[kRowBytes] = {};

// A workgroup's LDS: a ring of stages (one tile's rows as they are loaded), the
// keys' scales (E4M3) and the tiles' list entries, with one bf16 tile or two of codes on
// their way while one is computed.  Two rings fit a CU:
//   * two workgroups of one ring, when every token has its own (they drift
//     apart, so one computes while the other waits);
//   * one workgroup with two rings, whose waves take alternate tiles of the same
//     part and are joined in LDS at its end, when tokens are split: half the parts to
//     write out and read back (64 tokens x 64 heads over 2048 8-bit slots: 8
//     parts of 128 KB a token became 4).
// (One workgroup of 128 heads and one ring keeps 8 waves in step: with the
// kernel as it then was, 1024 tokens x 128 heads x 2048 slots took 778 us so, and
// 748 as two workgroups of 64.)
template <int NW, int RINGS, bool E4M3>
struct Lds {
  static constexpr int kLatentBytes = E4M3 ? kTileCodes : kTileLatent;
  static constexpr int kStageBytes = kLatentBytes + kTileRope;
  static constexpr int kAhead = E4M3 ? 2 : 1;                                 // tiles on their way
  static constexpr int kStages = kAhead + 1;
  static constexpr int kScales = kStages * kStageBytes;                       // a wave's own: 32 a stage
  static constexpr int kEntries = kScales + (E4M3 ? NW * kStages * 128 : 0);  // a wave's own: two tiles
  static constexpr int kRingBytes = (kEntries + NW * 2 * 128 + 255) / 256 * 256;
  // joining: the second ring's waves' accumulators, then their maxima and sums
  static constexpr int kJoinBytes = RINGS > 1 ? NW * (kHeads * kLatent * 4 + 512) : 0;
  static constexpr int kBytes = RINGS * kRingBytes > kJoinBytes ? RINGS * kRingBytes : kJoinBytes;
  static_assert(2 / RINGS * kBytes <= 160 * 1024, "two rings to a CU");
  // loads of rows a wave queues per tile
  static constexpr int kLoads = (E4M3 ? kTileKeys / 2 : kTileKeys) / NW + 4 / NW;
};

// What a wave keeps of its 16 heads along a row of keys.
struct HeadState {
  bf16x8 q[kLatentSteps + kRopeSteps];
  f32x4 o[kColBlocks];
  float m;      // reference maximum (log2 units)
  float l;      // this lane's part of the sum
};

// The same as swizzle() for rows of codes: 8-byte reads of one chunk of 16
// consecutive rows, and transposed reads whose 16 lanes cover one chunk of rows
// 4 g + 0..3 and 16 + 4 g + 0..3.
__device__ __forceinline__ int code_swizzle(int row) {
  return (row & 3) | ((row ^ (row >> 2)) & 4) | (row & 8);
}

// A slot's row; zeros for a slot below 0.  (Selected, not branched on: a tile takes 32 of them.)
__device__ __forceinline__ const char* row_at(const char* base, int64_t stride, int slot) {
  return (slot < 0 ? kZeroRow : base) + (int64_t)(slot < 0 ? 0 : slot) * stride;
}

// Lane `from`'s address, in every lane.
__device__ __forceinline__ const char* row_of(const char* rows, int from) {
  const uint64_t v = (uint64_t)(uintptr_t)rows;
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, from), hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), from);
  return reinterpret_cast<const char*>((uintptr_t)((uint64_t)hi << 32 | lo));
}

// Queues the loads of a tile's rows into the stage at LDS address `lds`;
// `slots`: lane i (mod 32) holds key i's.  Every lane forms the address of its own
// key's row, and a load takes it from there by two lane reads: formed one row
// after the other, the addresses took as long to queue as the tile to compute
// where one wave loads all rows.
template <int NW, bool E4M3>
__device__ __forceinline__ void load_tile(const Cache& c, int slots, uint32_t lds, int wave) {
  const int lane = lane_here();
  const char* rows = row_at(c.latent, c.latent_stride, slots);
  if (E4M3) {
    constexpr int kEach = kTileKeys / 2 / NW;   // two rows an instruction
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int pair = wave * kEach + i;
      const char* r0 = row_of(rows, 2 * pair);
      const char* r1 = row_of(rows, 2 * pair + 1);
      const int sw = lane < 32 ? code_swizzle(2 * pair) : code_swizzle(2 * pair + 1);
      queue_to_lds((lane < 32 ? r0 : r1) + ((lane & 31) ^ sw) * 16, lds + pair * 2 * kLatent);
    }
  } else {
    constexpr int kEach = kTileKeys / NW;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int key = wave * kEach + i;
      queue_to_lds(row_of(rows, key) + (lane ^ swizzle(key)) * 16, lds + key * kRowBytes);
    }
  }
  lds += E4M3 ? kTileCodes : kTileLatent;
  constexpr int kRopeEach = 4 / NW;             // eight rows an instruction
#pragma unroll
  for (int i = 0; i < kRopeEach; ++i) {
    const int group = wave * kRopeEach + i;
    const int s = __builtin_amdgcn_ds_bpermute((group * 8 + (lane >> 3)) * 4, slots);
    const char* row = row_at(c.rope, c.rope_stride, s);
    queue_to_lds(row + ((lane ^ ((group * 8 + (lane >> 3)) >> 1)) & 7) * 16, lds + group * 8 * kRopeBytes);
  }
}

// A lane's LDS offsets within a tile.  The other offsets differ from these in
// bits that the swizzle only flips (bf16: a step's chunks in bits 6 and 7, a
// column block's in bits 5 to 7; codes: bits 5 to 7, and 4 to 7).  They are
// formed where they are read: as registers of their own they would push Q and
// O^T out.
struct TileReads {
  int key;      // row lane % 16, the first step's values
  int rope;
  int value;    // transposed reads of the lane group's rows, column block 0
};

template <bool E4M3>
__device__ __forceinline__ TileReads tile_reads(int lane) {
  const int i = lane & 15, g = lane >> 4;
  TileReads t;
  t.rope = i * kRopeBytes + (((g ^ (i >> 1)) & 7) << 4);
  if (E4M3) {
    const int key = 4 * g + ((i >> 1) & 3) + 16 * (i >> 3);
    t.key = i * kLatent + (((g >> 1) ^ code_swizzle(i)) << 4) + (g & 1) * 8;
    t.value = key * kLatent + (code_swizzle(key) << 4) + (i & 1) * 8;
  } else {
    const int key = 4 * g + (i >> 2);
    t.key = i * kRowBytes + ((g ^ swizzle(i)) << 4);
    t.value = key * kRowBytes + ((((i & 3) >> 1) ^ swizzle(key)) << 4) + (i & 1) * 8;
  }
  return t;
}

// Scores of a tile at LDS address lat: s[b][r] is the lane's head's with key
// 16 b + 4 (lane / 16) + r.  scales (E4M3): each key's scale.  (Stages begin at
// multiples of 256 bytes, so their address may be added before the xor.)
template <bool E4M3>
__device__ __forceinline__ void score_tile(const HeadState& st, f32x4 (&s)[2], uint32_t lat, uint32_t scales,
                                           const TileReads& at, int lane) {
  s[0] = f32x4{};
  s[1] = f32x4{};
  const uint32_t key = (uint32_t)here(at.key + (int)lat);
  if constexpr (E4M3) {
    // rows 16 on swizzle with bit 2 flipped
    run_ahead<2 * kLatentSteps, kReadsAhead>(
        [&](int n) {
          const int k = n >> 1, b = n & 1;
          return read_lds<u32x2>((key ^ (uint32_t)(((k & 7) << 5) ^ (b << 6))) + 16 * b * kLatent + (k >> 3) * 256);
        },
        [&](int n, bf16x8 rows) { s[n & 1] = mfma16(rows, st.q[n >> 1], s[n & 1]); });
    const int g = lane >> 4;
#pragma unroll
    for (int b = 0; b < 2; ++b) s[b] *= read_lds<f32x4>(scales + 64 * b + 16 * g);
  } else {
    run_ahead<2 * kLatentSteps, kReadsAhead>(
        [&](int n) {
          const int k = n >> 1, b = n & 1;
          return read_lds<bf16x8>((key ^ (uint32_t)((k & 3) << 6)) + 16 * b * kRowBytes + (k >> 2) * 256);
        },
        [&](int n, bf16x8 rows) { s[n & 1] = mfma16(rows, st.q[n >> 1], s[n & 1]); });
  }
  const uint32_t rope = (uint32_t)at.rope + lat + (E4M3 ? kTileCodes : kTileLatent);
  run_ahead<2 * kRopeSteps, 2 * kRopeSteps>(
      [&](int n) { return read_lds<bf16x8>((rope ^ (uint32_t)((n >> 1) << 6)) + 16 * (n & 1) * kRopeBytes); },
      [&](int n, bf16x8 rows) { s[n & 1] = mfma16(rows, st.q[kLatentSteps + (n >> 1)], s[n & 1]); });
}

// The softmax step of a tile whose scores are s: the weights, in the order of the
// second product's keys.  mask: the keys that count for this lane's head (of the lane's
// own half of the keys, as the tile has them).  With CLEAN, keys that do not count for
// some heads count for others, and their scales may be NaN.
template <bool E4M3, bool CLEAN = false>
__device__ __forceinline__ bf16x8 weights_of_tile(HeadState& st, f32x4 (&s)[2], uint32_t scales, uint32_t mask,
                                                  float scale_log2, int lane) {
  const int g = lane >> 4;
  const uint32_t own = mask >> (4 * g);
  if (mask != 0xFFFFFFFFu) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!((own >> (16 * b + r)) & 1)) s[b][r] = -INFINITY;
  }
  float top = s[0][0];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) top = fmaxf(top, s[b][r]);
  top = max_of_4(top) * scale_log2;
  if (__any(top > st.m + kLazy || fabsf(st.m) > kFar)) {
    const float m = fmaxf(st.m, top);
    const float f = __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= f;
#pragma unroll
    for (int cb = 0; cb < kColBlocks; ++cb) st.o[cb] *= f;
    if (__any(fabsf(m) > kFar)) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[b][r] *= scale_log2;
      scale_log2 = 1.0f;
    }
  }
  // Weights in bf16 (the matrix cores' type): an unbiased rounding of at most 2^-8 on
  // each (over codes of the weight times the key's scale, as one), as large as the rounding of the
  // result itself: against 64 bits results are off by 0.0017 to 0.0022 (relative, in the mean square), with fp32
  // weights by 0.0017.  Two bf16 terms a weight would double the second product.  The sum keeps them in fp32.
  bf16x8 p;
  float sum = 0.f;                        // a tile at a time: few additions to a large number
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    f32x4 w;
#pragma unroll
    for (int r = 0; r < 4; ++r) w[r] = __builtin_amdgcn_exp2f(fmaf(s[b][r], scale_log2, -st.m));
    sum += (w[0] + w[1]) + (w[2] + w[3]);
    if (E4M3) w *= read_lds<f32x4>(scales + 64 * b + 16 * g);
    if (E4M3 && CLEAN) {
#pragma unroll
      for (int r = 0; r < 4; ++r) w[r] = (own >> (16 * b + r)) & 1 ? w[r] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) p[4 * b + r] = (__bf16)w[r];
  }
  st.l += sum;
  return p;
}

// The second product's rows of a tile, a block of 16 latent values after the other: use(block, rows).
template <bool E4M3, typename Use>
__device__ __forceinline__ void for_values(uint32_t lat, const TileReads& at, Use use) {
  const uint32_t value = (uint32_t)here(at.value + (int)lat);
  if constexpr (E4M3) {
    run_ahead<kColBlocks, kReadsAhead>(
        [&](int cb) { return read_tr8((value ^ (uint32_t)((cb & 15) << 4)) + (cb >> 4) * 256); }, use);
  } else {
    run_ahead<kColBlocks, kReadsAhead>(
        [&](int cb) {
          const uint32_t v = (value ^ (uint32_t)((cb & 7) << 5)) + (cb >> 3) * 256;
          return join8(read_tr(v), read_tr(v + 16 * kRowBytes));
        },
        use);
  }
}

// The softmax step and the second product of a tile whose scores are s.
// mask: the tile's selected keys.
template <bool E4M3>
__device__ __forceinline__ void weigh_tile(HeadState& st, f32x4 (&s)[2], uint32_t lat, uint32_t scales,
                                           uint32_t mask, float scale_log2, const TileReads& at, int lane) {
  const bf16x8 p = weights_of_tile<E4M3>(st, s, scales, mask, scale_log2, lane);
  for_values<E4M3>(lat, at, [&](int cb, bf16x8 cols) { st.o[cb] = mfma16(cols, p, st.o[cb]); });
}

}  // namespace
}  // namespace latent
