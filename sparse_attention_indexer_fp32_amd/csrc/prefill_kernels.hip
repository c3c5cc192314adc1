// Latent attention, expanded form, on gfx950: causal attention over ragged
// batches whose heads have keys of 128 values of their own and 64 rotary
// values that all heads share, and values of 128.
//
//   z[i, j] = scale * (q_i[:128] . k_j + q_i[128:] . r_j),  j <= nk - nq + i
//   out_i   = sum_j softmax_j(z[i]) v_j
//
// One pass over the keys with a running reference maximum and sum per query.
//
// Tiling.  A workgroup of 4 waves takes 128 queries of one head, a wave 32 of
// them; keys come in tiles of 64.  Both products are taken transposed
// (S^T = K Q^T, O^T = V^T P^T), so that a lane keeps one query throughout: its
// column of scores, their maximum and sum, its column of O^T.  A lane's
// scores are exactly the elements of P^T that it feeds to the second product, when
// the keys of a step are taken in the order the accumulator holds them, so
// weights never leave their registers.  Q and O^T stay in registers; K is read
// from LDS 16 bytes a lane, V by transposed reads.  A tile's rows (each key's
// 512 bytes of key and value, and its rotary key) are loaded straight into LDS
// while the previous tile is computed.
//
// A unit is 128 queries of one head, and a workgroup takes one, the longest
// first; where units are few and long, workgroups share all units' tiles evenly
// instead, and parts of a unit are joined by a second launch.
//
// Measured (MI355X): a prompt of 8192 tokens x 32 heads 684-760 us over several
// cards, 900-1005 TFLOP/s, where a large library matrix product reaches 1255-1365:
// the matrix cores are busy 49 % of the time, and the softmax's vector
// instructions (160 to 40 matrix ones a tile, 32 of them exponentials) take the
// other half; LDS 26 %.  Six chunks of 1 to 1500 tokens behind 0 to 5000 cached
// ones x 20 heads 223-268 us, up to 745 TFLOP/s: bound by the longest units, 6500
// keys at 2.4 us a tile with two workgroups on a CU.  (The output written from the
// accumulators, 8 bytes a lane, and lane offsets that did not fit the registers
// cost 743 us instead of 716; head after head instead of block after block 738
// instead of 691.)

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "latent_device.h"
#include "latent_internal.h"

namespace latent {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;           // queries of a workgroup
constexpr int kKeys = 64;                    // keys of a tile
constexpr int kUpBytes = 2 * kHead * 2;      // a key row: key, then value
constexpr int kRopeBytes = kRope * 2;
constexpr int kHeadSteps = kHead / 16;       // 8 steps of the first product
constexpr int kRopeSteps = kRope / 16;       // and 4 of the rotary part
constexpr int kColBlocks = kHead / 32;       // 4 blocks of O^T
constexpr int kReadsAhead = 4;               // LDS reads in flight before a matrix instruction

struct Stage {
  char up[kKeys * kUpBytes];
  char rope[kKeys * kRopeBytes];
};

struct Block {
  int64_t q0, nq;            // the request's queries, and keys
  int64_t k0, nk;
  int64_t first;             // first query of the block in its request
};

// Request r's queries and keys, within the arrays; no queries if it starts in front of them.
__device__ __forceinline__ void request_rows(const PrefillArgs& a, int64_t r, Block& blk) {
  blk.q0 = a.q_starts[r];
  const int64_t q1 = a.q_starts[r + 1];
  blk.nq = blk.q0 >= 0 ? (q1 < a.num_tokens ? q1 : a.num_tokens) - blk.q0 : 0;
  blk.k0 = a.kv_starts[r];
  int64_t k1 = a.kv_starts[r + 1];
  k1 = k1 < a.num_kv ? k1 : a.num_kv;
  blk.nk = k1 > blk.k0 && blk.k0 >= 0 ? k1 - blk.k0 : 0;
}

__device__ __forceinline__ int64_t blocks_of(int64_t queries) { return queries > 0 ? (queries + kRows - 1) / kRows : 0; }

// Keys that query `row` of a request attends.
__device__ __forceinline__ int64_t keys_of(const PrefillArgs& a, const Block& blk, int64_t row) {
  const int64_t n = a.causal ? blk.nk - blk.nq + 1 + row : blk.nk;
  return n < 0 ? (int64_t)0 : (n < blk.nk ? n : blk.nk);
}
__device__ __forceinline__ int64_t last_row(const Block& blk) {
  return (blk.first + kRows < blk.nq ? blk.first + kRows : blk.nq) - 1;
}
// A block's tiles; one even when it has no key, so that somebody writes its rows.
__device__ __forceinline__ int64_t block_tiles(const PrefillArgs& a, const Block& blk) {
  const int64_t n = (keys_of(a, blk, last_row(blk)) + kKeys - 1) / kKeys;
  return n > 0 ? n : 1;
}

// The tiles of a request's first n blocks.  Causal: a whole block's last query
// attends kRows keys more than the block before, so block j has c + 2 j tiles
// (one, where that is below 1).
__device__ __forceinline__ int64_t tiles_before(const PrefillArgs& a, const Block& blk, int64_t n) {
  const int64_t most = (blk.nk + kKeys - 1) / kKeys, all = most > 0 ? most : 1;
  if (!a.causal) return n * all;
  constexpr int kStep = kRows / kKeys;
  static_assert(kRows % kKeys == 0, "a block adds whole tiles");
  const int64_t whole = n * kRows <= blk.nq ? n : n - 1;       // (the last may be partial: it has all keys)
  const int64_t c = (blk.nk - blk.nq + kRows + kKeys - 1 + (blk.nq / kKeys + 1) * kKeys) / kKeys - (blk.nq / kKeys + 1);
  int64_t ones = c < 1 ? (1 - c + kStep - 1) / kStep : 0;
  ones = ones < whole ? ones : whole;
  return ones + (whole - ones) * c + (whole * (whole - 1) - ones * (ones - 1)) / 2 * kStep + (n - whole) * all;
}

// Block `index` of the requests' blocks of kRows queries; false past the last.
// Wave-uniform, 64 requests at a time.
__device__ __forceinline__ bool find_block(const PrefillArgs& a, int64_t index, int lane, Block& blk) {
  int64_t before = 0;
  for (int64_t base = 0; base < a.num_requests; base += 64) {
    const int64_t b = base + lane;
    int n = 0;
    if (b < a.num_requests) {
      request_rows(a, b, blk);
      n = (int)blocks_of(blk.nq);
    }
    int incl = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    const uint64_t hit = __ballot(before + incl > index);
    if (hit) {
      const int src = (int)__builtin_ctzll(hit);
      request_rows(a, base + src, blk);
      blk.first = (index - before - __builtin_amdgcn_readlane(incl - n, src)) * kRows;
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// Block `index` of at most 64 requests' blocks, the longest first: a block's
// level is its last query's keys in steps of kRows, so d blocks before a
// request's last one it is d lower (blocks with no key count as level 1).  The
// lanes try 64 levels at a time for the lowest one that has at most `index`
// blocks above it.  Wave-uniform.
__device__ __forceinline__ bool find_longest(const PrefillArgs& a, int64_t index, int lane, Block& blk) {
  const int requests = (int)a.num_requests;
  int n = 0, top = 0;
  if (lane < requests) {
    request_rows(a, lane, blk);
    n = (int)blocks_of(blk.nq);
    top = n > 0 ? (int)((blk.nk + kRows - 1) / kRows) : 0;
  }
  // blocks of a request above a level
  auto above = [&](int levels, int count, int level) {
    const int some = a.causal ? (levels - level < count ? levels - level : count) : count;
    return level < 1 ? count : (levels > level ? some : 0);
  };
  int low = 0, high = 1, all = 0;
  for (int r = 0; r < requests; ++r) {
    const int levels = __builtin_amdgcn_readlane(top, r);
    all += __builtin_amdgcn_readlane(n, r);
    high = levels > high ? levels : high;
  }
  if (index >= all) return false;
  while (high - low > 1) {                 // more than `index` blocks above low, at most that above high
    const int step = (high - low + 63) / 64, level = low + (lane + 1) * step;
    int count = 0;
    for (int r = 0; r < requests; ++r)
      count += above(__builtin_amdgcn_readlane(top, r), __builtin_amdgcn_readlane(n, r), level);
    const int hit = (int)__builtin_ctzll(__ballot(count <= index || level >= high));
    const int found = low + (hit + 1) * step;
    low = found - step;
    high = found < high ? found : high;
  }
  // of the blocks at this level
  const int higher = above(top, n, high), here_n = above(top, n, high - 1) - higher;
  int before = 0;
  for (int r = 0; r < requests; ++r) {
    const int higher_r = __builtin_amdgcn_readlane(higher, r), n_r = __builtin_amdgcn_readlane(here_n, r);
    before += higher_r + (r < lane ? n_r : 0);
  }
  const int nth = (int)index - before;
  const int src = (int)__builtin_ctzll(__ballot(nth >= 0 && nth < here_n));
  request_rows(a, src, blk);
  blk.first = (int64_t)(__builtin_amdgcn_readlane(n, src) - 1 - __builtin_amdgcn_readlane(higher, src) -
                        __builtin_amdgcn_readlane(nth, src)) * kRows;
  return true;
}

// A value that is the same in every lane, as the compiler cannot see.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Of a split launch's workgroups, those that take part.
__device__ __forceinline__ int64_t shares_of(const PrefillArgs& a, int64_t tiles) {
  const int64_t most = tiles / kPrefillShareTiles;
  return most < 1 ? (tiles > 0 ? 1 : 0) : most < a.wgs ? most : (int64_t)a.wgs;
}

// A split launch's plan: the tiles of one head before each request, and the blocks.
struct SplitPlan {
  int64_t tiles[kPlanRequests + 1];
  int32_t blocks[kPlanRequests + 1];
  int64_t wave_tiles[kWaves];
  int32_t wave_blocks[kWaves];
};

__device__ void plan_split(const PrefillArgs& a, SplitPlan& plan, int tid) {
  constexpr int kEach = kPlanRequests / (64 * kWaves);       // neighbouring requests a lane sums up
  const int lane = tid & 63, wave = tid >> 6;
  int64_t tiles[kEach], sum = 0;
  int32_t blocks[kEach], count = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t r = (int64_t)tid * kEach + i;
    tiles[i] = sum;
    blocks[i] = count;
    if (r >= a.num_requests) continue;
    Block blk;
    request_rows(a, r, blk);
    sum += tiles_before(a, blk, blocks_of(blk.nq));
    count += (int32_t)blocks_of(blk.nq);
  }
  int64_t tiles_to = sum;
  int32_t blocks_to = count;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t t = __shfl_up(tiles_to, d);
    const int32_t b = __shfl_up(blocks_to, d);
    if (lane >= d) {
      tiles_to += t;
      blocks_to += b;
    }
  }
  if (lane == 63) {
    plan.wave_tiles[wave] = tiles_to;
    plan.wave_blocks[wave] = blocks_to;
  }
  lds_barrier();
  for (int w = 0; w < wave; ++w) {
    tiles_to += plan.wave_tiles[w];
    blocks_to += plan.wave_blocks[w];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    plan.tiles[tid * kEach + i] = tiles_to - sum + tiles[i];
    plan.blocks[tid * kEach + i] = blocks_to - count + blocks[i];
  }
  if (tid == 64 * kWaves - 1) {
    plan.tiles[kPlanRequests] = tiles_to;
    plan.blocks[kPlanRequests] = blocks_to;
  }
  lds_barrier();
}

// Where a lane's loads of a tile come from: byte offsets from the tile's first
// rows, the same for every whole tile.
struct TileLoads {
  uint32_t up[kKeys / 2 / kWaves];     // two rows an instruction
  uint32_t rope[kKeys / 8 / kWaves];   // eight rotary keys an instruction
};

// Rows at or past `rows` are replaced by the last row before: whatever it
// holds, its weight is masked.
__device__ __forceinline__ TileLoads tile_loads(const PrefillArgs& a, int rows, int lane, int wave) {
  TileLoads t;
#pragma unroll
  for (int i = 0; i < kKeys / 2 / kWaves; ++i) {
    const int key = 2 * (wave * (kKeys / 2 / kWaves) + i) + (lane >> 5);
    const int row = key < rows ? key : rows - 1;
    t.up[i] = (uint32_t)row * (uint32_t)(a.kv_token_stride * 2) + (uint32_t)(((lane & 31) ^ swizzle(key)) * 16);
  }
#pragma unroll
  for (int i = 0; i < kKeys / 8 / kWaves; ++i) {
    const int key = 8 * (wave * (kKeys / 8 / kWaves) + i) + (lane >> 3);
    const int row = key < rows ? key : rows - 1;
    t.rope[i] = (uint32_t)row * (uint32_t)(a.rope_stride * 2) + (uint32_t)(((lane ^ (key >> 1)) & 7) * 16);
  }
  return t;
}

// Queues the loads of the tile whose first rows are at up and rope.
__device__ __forceinline__ void load_tile(const char* up, const char* rope, const TileLoads& t, Stage& st, int wave) {
#pragma unroll
  for (int i = 0; i < kKeys / 2 / kWaves; ++i)
    load_to_lds(up + t.up[i], st.up + (wave * (kKeys / 2 / kWaves) + i) * 2 * kUpBytes);
#pragma unroll
  for (int i = 0; i < kKeys / 8 / kWaves; ++i)
    load_to_lds(rope + t.rope[i], st.rope + (wave * (kKeys / 8 / kWaves) + i) * 8 * kRopeBytes);
}

struct RowState {
  bf16x8 q[kHeadSteps + kRopeSteps];
  f32x16 o[kColBlocks];
  float m;      // reference maximum (log2 units)
  float l;      // this lane's part of the sum
};

// A lane's LDS offsets within a tile.  The other offsets differ from these in
// bits that the swizzle only flips (chunk 2 k + hb in bits 5 to 7, column block
// in bits 6 and 7), and are formed where they are read.
struct TileReads {
  int key;      // row lane % 32, chunk hb
  int rope;
  int value;    // transposed reads of rows 4 hb + 0..3, column block 0
};

__device__ __forceinline__ TileReads tile_reads(int lane) {
  const int i = lane & 31, hb = lane >> 5, j = lane & 15, quarter = (lane >> 4) & 1;
  const int key = 4 * hb + (j >> 2);
  TileReads t;
  t.key = i * kUpBytes + ((hb ^ swizzle(i)) << 4);
  t.rope = i * kRopeBytes + (((hb ^ (i >> 1)) & 7) << 4);
  t.value = key * kUpBytes + kUpBytes / 2 + (((2 * quarter + ((j & 3) >> 1)) ^ swizzle(key)) << 4) + (j & 1) * 8;
  return t;
}

// Whether a tile's values hold an infinity or a NaN (the same answer in every lane).
__device__ __forceinline__ bool values_not_finite(const Stage& t, int lane) {
  bool bad = false;
#pragma unroll 4
  for (int at = lane; at < kKeys * 16; at += 64) {
    const uint4 v = *reinterpret_cast<const uint4*>(t.up + (at >> 4) * kUpBytes + kUpBytes / 2 + (at & 15) * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      bad = bad || (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
  }
  return __any(bad);
}

// The second product of a masked tile whose values are not all finite: a
// matrix product would bring 0 * inf = NaN into rows that do not attend the
// key, so each key is added where it is attended only.
__device__ __forceinline__ void add_values_one_by_one(f32x16 (&o)[kColBlocks], const f32x16 (&w)[2],
                                                                const Stage& t, int limit, int lane) {
  const int hb = lane >> 5;
#pragma unroll 1
  for (int key = 0; key < kKeys; ++key) {
    // the weight of this lane's query for the key sits in one half-wave
    float own = 0.f;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (32 * kb + acc_row(r, hb) == key) own = w[kb][r];
    const float p = own + other_half(own, lane);
    if (key >= limit) continue;
    const int row = here(hb);
#pragma unroll
    for (int cb = 0; cb < kColBlocks; ++cb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int col = cb * 32 + acc_row(r, row);
        const char* at = t.up + key * kUpBytes + kUpBytes / 2 + (((col >> 3) ^ swizzle(key)) << 4) + (col & 7) * 2;
        o[cb][r] = fmaf((float)(__bf16)p, (float)*reinterpret_cast<const __bf16*>(at), o[cb][r]);
      }
  }
}

// One tile for a wave's 32 queries.  MASKED: the lane's query attends the
// tile's keys below `limit` only.
template <bool MASKED>
__device__ __forceinline__ void attend_tile(RowState& st, const Stage& t, const TileReads& at, int limit,
                                            float scale_log2, int lane) {
  const int hb = lane >> 5;
  const uint32_t stage = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)t.up;
  f32x16 s[2] = {f32x16{}, f32x16{}};
  {
    const uint32_t key = (uint32_t)here(at.key), rope = (uint32_t)here(at.rope);
    run_ahead<2 * (kHeadSteps + kRopeSteps), kReadsAhead>(
        [&](int n) {
          const int k = n >> 1, kb = n & 1;
          return read_lds<bf16x8>(stage + (k < kHeadSteps ? (key ^ (uint32_t)(k << 5)) + 32 * kb * kUpBytes
                                                          : (rope ^ (uint32_t)((k - kHeadSteps) << 5)) + kKeys * kUpBytes +
                                                                32 * kb * kRopeBytes));
        },
        [&](int n, bf16x8 rows) { s[n & 1] = mfma(rows, st.q[n >> 1], s[n & 1]); });
  }
  float top = -INFINITY;
  const int own_limit = limit - 4 * hb;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if (MASKED && 32 * kb + acc_row(r, 0) >= own_limit) s[kb][r] = -INFINITY;
      top = fmaxf(top, s[kb][r]);
    }
  top = fmaxf(top, other_half(top, lane)) * scale_log2;
  if (__any(top > st.m + kLazy || fabsf(st.m) > kFar)) {
    const float m = fmaxf(st.m, top);
    const float f = __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= f;
#pragma unroll
    for (int cb = 0; cb < kColBlocks; ++cb)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[cb][r] *= f;
    if (__any(fabsf(m) > kFar)) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[kb][r] *= scale_log2;
      scale_log2 = 1.0f;
    }
  }
  // Weights in bf16 (the matrix cores' type): an unbiased rounding of at most 2^-8 on
  // each, as large as the rounding of the result itself.  The sum keeps them in
  // fp32, a tile at a time: added to the running sum one by one, a long row's many
  // small weights would each be rounded against it (131072 equal ones 3e-4 off).
  bf16x8 p[4];
  float sum[2] = {};
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float w = __builtin_amdgcn_exp2f(fmaf(s[kb][r], scale_log2, -st.m));
      sum[kb] += w;
      if (MASKED) s[kb][r] = w;
      p[2 * kb + ((r >> 2) & 1)][((r >> 3) << 2) + (r & 3)] = (__bf16)w;   // a step: rows 0..3 and 16..19 of each half
    }
  st.l += sum[0] + sum[1];
  if (MASKED && values_not_finite(t, lane_here())) {
    add_values_one_by_one(st.o, s, t, limit, lane_here());
    return;
  }
  const uint32_t value = (uint32_t)here(at.value);
  run_ahead<4 * kColBlocks, kReadsAhead>(
      [&](int n) {
        // step k: rows 32 (k / 2) + 8 (k % 2) + 4 hb + 0..3 and those 16 on; rows 8 on swizzle with bits 0 and 1 flipped
        const int k = n / kColBlocks, cb = n % kColBlocks;
        const uint32_t v = stage + (value ^ (uint32_t)((cb << 6) ^ (k & 1) * 48)) + (32 * (k >> 1) + 8 * (k & 1)) * kUpBytes;
        return join8(read_tr(v), read_tr(v + 16 * kUpBytes));
      },
      [&](int n, bf16x8 cols) { st.o[n % kColBlocks] = mfma(cols, p[n / kColBlocks], st.o[n % kColBlocks]); });
}

// A wave's 32 rows of the output, out_i = o_i / l, by way of LDS (`own`: 8 KB
// of the wave's): a lane holds 8-byte pieces of one row, and writes 16 bytes of
// whole rows (each 16-byte chunk is flipped with its row, against bank conflicts).
__device__ __forceinline__ void write_rows(const PrefillArgs& a, const Block& blk, int64_t wave_row, int64_t head,
                                           const f32x16 (&o)[kColBlocks], float m, float l, char* own, int lane) {
  const int i = lane & 31, hb = lane >> 5;
  const float inv = inverse_sum(l);
#pragma unroll
  for (int cb = 0; cb < kColBlocks; ++cb)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      bf16x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (__bf16)(o[cb][4 * g + e] * inv);
      *reinterpret_cast<bf16x4*>(own + i * (kHead * 2) + (((cb * 4 + g) ^ (i & 15)) << 4) + hb * 8) = v;
    }
  const int64_t left = blk.nq - wave_row;
  const int chunk = lane & 15;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const int r = n * 4 + (lane >> 4);
    const uint4 v = *reinterpret_cast<const uint4*>(own + r * (kHead * 2) + ((chunk ^ (r & 15)) << 4));
    if (r < left)
      *reinterpret_cast<uint4*>(a.out + ((blk.q0 + wave_row + r) * a.num_heads + head) * kHead + chunk * 8) = v;
  }
  if (a.lse && hb == 0 && i < left) a.lse[(blk.q0 + wave_row + i) * a.num_heads + head] = log_sum(m, l);
}

// blocks: of one head, at most.
template <bool SPLIT>
__global__ __launch_bounds__(64 * kWaves, 2) void prefill_kernel(PrefillArgs a, int64_t blocks) {
  __shared__ __attribute__((aligned(256))) Stage stage0, stage1;
  const int lane = threadIdx.x & 63, hb = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Split: workgroups are dealt to the 8 XCDs in turn, and each takes a contiguous
  // share of all heads' blocks, so that blocks of a head, which read the same
  // keys, share an L2.
  const int64_t nth = (int64_t)(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  Block blk;
  int64_t head, index;                    // the block's number in its head
  // Split: tiles [pos, stop) of all heads' tiles are this workgroup's, and pos
  // is tile `first` of the block.
  int64_t pos = 0, stop = 1, first = 0, request = 0, total = 0;
  if (SPLIT) {
    SplitPlan& plan = *reinterpret_cast<SplitPlan*>(&stage0);
    static_assert(sizeof(SplitPlan) <= sizeof(Stage), "the plan is made where the rows go");
    plan_split(a, plan, threadIdx.x);
    const int64_t head_tiles = uniform(plan.tiles[kPlanRequests]);
    total = head_tiles * a.num_heads;
    const int64_t shares = shares_of(a, total);
    if (nth >= shares) return;
    pos = total * nth / shares;
    stop = total * (nth + 1) / shares;
    head = pos / head_tiles;
    first = pos % head_tiles;
    int l = 0, h = kPlanRequests;
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if (uniform(plan.tiles[mid]) <= first) l = mid; else h = mid;
    }
    request = l;
    first -= uniform(plan.tiles[l]);
    request_rows(a, request, blk);
    int64_t block = 0, past = blocks_of(blk.nq);
    while (past - block > 1) {
      const int64_t mid = (block + past) >> 1;
      if (tiles_before(a, blk, mid) <= first) block = mid; else past = mid;
    }
    first -= tiles_before(a, blk, block);
    index = uniform(plan.blocks[l]) + block;
    blk.first = block * kRows;
  } else {
    // All heads of a block, the longest blocks first (of many requests, the last
    // ones), so that none begins when others end; where heads are a multiple of 8,
    // each stays on one XCD.  (Head after head, each XCD a contiguous share: 8192 x
    // 32 heads took 738 us and not 700, seven short chunks x 32 184 and not 140.)
    if ((int64_t)blockIdx.x >= blocks * a.num_heads) return;
    index = blockIdx.x / (unsigned)a.num_heads;
    head = blockIdx.x - index * a.num_heads;
    if (!(a.num_requests <= 64 ? find_longest(a, index, lane, blk) : find_block(a, blocks - 1 - index, lane, blk))) return;
  }
  const TileReads reads = tile_reads(lane);
  const TileLoads loads = tile_loads(a, kKeys, lane, wave);
  const float scale_log2 = fabsf(a.scale_log2);

  while (pos < stop) {
    const int64_t row = blk.first + wave * 32 + (lane & 31);     // the lane's query in its request
    const bool live = row < blk.nq;
    // keys it attends, and the most and fewest any of the wave's and the workgroup's do
    const int own_keys = (int)keys_of(a, blk, row);
    const int64_t wave_row = blk.first + wave * 32, end_row = last_row(blk);
    const int64_t wave_most =
        wave_row < blk.nq ? keys_of(a, blk, wave_row + 31 < end_row ? wave_row + 31 : end_row) : 0;
    const int64_t wave_least = keys_of(a, blk, wave_row);
    // the part [begin, end) of the block's keys
    const int64_t tiles = block_tiles(a, blk), last = SPLIT && first + (stop - pos) < tiles ? first + (stop - pos) : tiles;
    const int64_t begin = first * kKeys;
    int64_t end = keys_of(a, blk, end_row);
    if (SPLIT && last * kKeys < end) end = last * kKeys;

    RowState st;
    st.m = kNoMax;
    st.l = 0.f;
#pragma unroll
    for (int cb = 0; cb < kColBlocks; ++cb) st.o[cb] = f32x16{};
    {
      // a negative scale goes into the signs of q: the largest product is then the largest score
      const uint32_t sign = a.scale_log2 < 0.f ? 0x80008000u : 0u;
      const uint16_t* q = a.q + (blk.q0 + row) * a.q_token_stride + head * a.q_head_stride + hb * 8;
#pragma unroll
      for (int k = 0; k < kHeadSteps + kRopeSteps; ++k) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live) v = *reinterpret_cast<const uint4*>(q + k * 16);
        st.q[k] = __builtin_bit_cast(bf16x8, make_uint4(v.x ^ sign, v.y ^ sign, v.z ^ sign, v.w ^ sign));
      }
    }

    const char* up = reinterpret_cast<const char*>(a.kv + blk.k0 * a.kv_token_stride + head * a.kv_head_stride);
    const char* rope = reinterpret_cast<const char*>(a.rope + blk.k0 * a.rope_stride);
    // tiles may reach past the workgroup's keys, but not past the request's
    auto queue = [&](int64_t j0, Stage& st_to) {
      const char* u = up + j0 * a.kv_token_stride * 2;
      const char* r = rope + j0 * a.rope_stride * 2;
      const int64_t rows = blk.nk - j0;
      TileLoads t = loads;
      if (rows < kKeys) t = tile_loads(a, (int)rows, lane_here(), wave);
      load_tile(u, r, t, st_to, wave);
    };
    if (SPLIT) lds_barrier();     // the last part's reads are done
    if (begin < end) queue(begin, stage0);
    auto step = [&](int64_t j0, const Stage& cur, Stage& nxt) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      lds_barrier();              // every wave's rows are there, and nobody reads the other stage any more
      if (j0 + kKeys < end) queue(j0 + kKeys, nxt);
      if (j0 >= wave_most) return;
      // (Split, the offsets are worked out for every tile: one that is kept does not fit the
      // registers, and its reload waits for the rows on their way: 100 queries x 8 heads
      // behind 60000 keys 101 us so, 94 like this.)
      const TileReads at = SPLIT ? tile_reads(lane_here()) : reads;
      if (j0 + kKeys <= wave_least) {
        attend_tile<false>(st, cur, at, kKeys, scale_log2, lane);
      } else {
        const int left = own_keys - (int)j0;
        attend_tile<true>(st, cur, at, left < 0 ? 0 : (left < kKeys ? left : kKeys), scale_log2, lane);
      }
    };
    for (int64_t j0 = begin; j0 < end; j0 += 2 * kKeys) {
      step(j0, stage0, stage1);
      if (j0 + kKeys < end) step(j0 + kKeys, stage1, stage0);
    }

    const float l = st.l + other_half(st.l, lane);
    if (!SPLIT || (first == 0 && last == tiles)) {
      lds_barrier();              // nobody reads the stages any more
      write_rows(a, blk, wave_row, head, st.o, st.m, l, stage0.up + wave * (32 * kHead * 2), lane_here());
    } else {
      // A share holds at most one part that begins inside a block (its first),
      // and one that begins a block it does not end (its last).
      const int64_t at = ((first == 0 ? a.wgs : 0) + nth) * kWaves + wave;
      float* o = a.part_out + at * (32 * kHead) + lane_here() * 4;
#pragma unroll
      for (int cb = 0; cb < kColBlocks; ++cb)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<f32x4*>(o + (cb * 4 + g) * 256) =
              f32x4{st.o[cb][4 * g], st.o[cb][4 * g + 1], st.o[cb][4 * g + 2], st.o[cb][4 * g + 3]};
      if (hb == 0) a.part_ml[at * 32 + lane] = make_float2(st.m, l);
    }
    if (!SPLIT) return;

    if (first == 0 && index < blocks && threadIdx.x == 0) {
      // the block's last tile is held by the last share g with total g / shares <= that tile
      const int64_t g1 = last == tiles ? nth : ((pos + tiles) * shares_of(a, total) - 1) / total;
      int32_t* rec = a.part_rec + (head * blocks + index) * 2;
      rec[0] = (int32_t)nth;
      rec[1] = (int32_t)(g1 - nth + 1);
    }
    // on to the next block
    pos += last - first;
    first = 0;
    blk.first += kRows;
    ++index;
    while (blk.first >= blk.nq && pos < stop) {
      if (++request >= a.num_requests) {
        request = 0;
        index = 0;
        if (++head >= a.num_heads) return;
      }
      request_rows(a, request, blk);
      blk.first = 0;
    }
  }
}

// The blocks that a split launch left in parts: each part's accumulators are
// weighed by 2^(its maximum - the largest).  A workgroup takes one wave's 32 queries
// of a block, a wave of it 32 of their 128 columns, kJoinAhead parts in flight.
constexpr int kJoinAhead = 4;
__global__ __launch_bounds__(64 * kColBlocks) void prefill_join_kernel(PrefillArgs a, int64_t blocks) {
  const int lane = threadIdx.x & 63, hb = lane >> 5;
  const int cb = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t index = blockIdx.x / kWaves, head = blockIdx.y;
  const int wave = blockIdx.x % kWaves;
  Block blk;
  if (!find_block(a, index, lane, blk)) return;
  const int32_t* rec = a.part_rec + (head * blocks + index) * 2;
  const int g0 = rec[0], parts = rec[1];
  const int64_t row = blk.first + wave * 32 + (lane & 31);
  if (parts <= 1 || blk.first + wave * 32 >= blk.nq) return;
  f32x16 o = f32x16{};
  float m = kNoMax, l = 0.f;
  for (int p0 = 0; p0 < parts; p0 += kJoinAhead) {
    f32x4 po[kJoinAhead][4];
    float2 ml[kJoinAhead];
#pragma unroll
    for (int d = 0; d < kJoinAhead; ++d) {
      const int p = p0 + d < parts ? p0 + d : p0;
      const int64_t at = ((int64_t)(p == 0 ? a.wgs : p) + g0) * kWaves + wave;
      ml[d] = a.part_ml[at * 32 + (lane & 31)];
#pragma unroll
      for (int g = 0; g < 4; ++g)
        po[d][g] = *reinterpret_cast<const f32x4*>(a.part_out + at * (32 * kHead) + (cb * 4 + g) * 256 + lane * 4);
    }
#pragma unroll
    for (int d = 0; d < kJoinAhead; ++d) {
      if (p0 + d >= parts) continue;
      const float to = fmaxf(m, ml[d].x);
      const float f = __builtin_amdgcn_exp2f(m - to), g = __builtin_amdgcn_exp2f(ml[d].x - to);
      m = to;
      l = l * f + ml[d].y * g;
#pragma unroll
      for (int r = 0; r < 16; ++r) o[r] = o[r] * f + po[d][r >> 2][r & 3] * g;
    }
  }
  if (row >= blk.nq) return;
  const float inv = inverse_sum(l);
  const int64_t at = (blk.q0 + row) * a.num_heads + head;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    bf16x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (__bf16)(o[4 * g + e] * inv);
    *reinterpret_cast<bf16x4*>(a.out + at * kHead + cb * 32 + 8 * g + 4 * hb) = v;
  }
  if (a.lse && cb == 0 && hb == 0) a.lse[at] = log_sum(m, l);
}

}  // namespace

// A request's last block may be partial: at most num_requests blocks beyond the full ones.
int64_t prefill_blocks(int num_tokens, int num_requests) {
  return num_tokens / kRows + (num_requests < num_tokens ? num_requests : num_tokens);
}

int64_t prefill_threads(int num_tokens, int num_heads, int num_requests) {
  return (prefill_blocks(num_tokens, num_requests) * num_heads + 7) / 8 * 8 * 64 * kWaves;
}

SplitLayout prefill_split_layout(int num_tokens, int num_heads, int num_requests, int wgs) {
  const size_t parts = (size_t)2 * wgs * kRows;
  SplitLayout s;
  s.out_bytes = parts * kHead * sizeof(float);
  s.ml_bytes = parts * sizeof(float2);
  s.rec_bytes = (size_t)prefill_blocks(num_tokens, num_requests) * num_heads * 2 * sizeof(int32_t);
  return s;
}

hipError_t launch_prefill(const PrefillArgs& a, hipStream_t stream) {
  const int64_t blocks = prefill_blocks(a.num_tokens, a.num_requests);
  const int64_t grid = ((a.wgs > 0 ? a.wgs : blocks * a.num_heads) + 7) / 8 * 8;
  if (a.wgs == 0) {
    hipLaunchKernelGGL(prefill_kernel<false>, dim3((unsigned)grid), dim3(64 * kWaves), 0, stream, a, blocks);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(prefill_kernel<true>, dim3((unsigned)grid), dim3(64 * kWaves), 0, stream, a, blocks);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(prefill_join_kernel, dim3((unsigned)(blocks * kWaves), (unsigned)a.num_heads), dim3(64 * kColBlocks), 0,
                     stream, a, blocks);
  return hipGetLastError();
}

}  // namespace latent
