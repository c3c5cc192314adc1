// Latent attention, absorbed form, on gfx950: every head of a token reads the
// same cached rows, so a workgroup stages a tile of rows in LDS once for all
// its heads, and keys and values are the same bytes.
//
//   z[h, j] = scale * (s_j q_c[h] . c_j + q_r[h] . r_j)
//   out[h]  = sum_j softmax_j(z[h]) s_j c_j          (s_j = 1 in a bf16 cache)
//
// One pass over the rows with a running reference maximum and sum per head.
//
// Tiling.  A wave owns 16 heads, a workgroup 1, 2 or 4 waves (more than 64
// heads take several workgroups); a tile is 32 keys.  Both products are taken transposed,
//   S^T = K Q^T   (rows: keys,          columns: heads; 18 steps of 32 values),
//   O^T = V^T P^T (rows: latent values, columns: heads; one step of 32 keys),
// so that a lane keeps one head throughout: its column of S^T, that head's
// maximum and sum, and its column of O^T.  A lane's 8 scores of a tile are then
// exactly the elements of P^T that it has to feed to the second product, when
// the keys of that step are taken in the order the accumulators hold them:
// weights never leave their registers, and the waves of a workgroup share
// nothing but the rows.  Q (18 x 4 registers) and O^T (32 x 4) stay in
// registers for all keys, two waves to a SIMD.  K is read from LDS 16 bytes a
// lane, V by transposed reads of the same bytes; E4M3 rows stay codes in LDS
// and are widened as they are read.
//
// (Waves of 32 heads would halve the LDS reads, but need 144 + 256 registers for
// a whole row: with O^T in the accumulation registers, 1024 tokens x 128 heads x
// 2048 bf16 slots took 727 us at one wave to a SIMD, and every smaller shape longer
// than here.  A pair of waves that share 32 heads by halves of the row has to
// add its scores through LDS, with a second barrier a tile, and to repeat the
// softmax step: 748 us.)
//
// Rows of a tile come from anywhere in the cache, one kilobyte-long row a
// load instruction (bf16), straight into LDS, while the previous tile is
// computed.  Rows that are not selected are loaded as zeros: what the cache
// holds there is never used.
//
// Measured (MI355X): 1024 tokens x 128 heads x 2048 selected bf16 slots of a
// 65536-token cache 628-720 us over several cards, 810-930 TFLOP/s: the matrix
// cores are busy 42 % of the time at the 1.96 GHz they clock to, LDS 44 %, and
// the vector instructions take 43 %, which the two waves of a SIMD hardly get to
// overlap with the matrix ones.  8-bit rows 764-830 us: widening them makes that
// 70 %.  With 64, 32 and 16 heads bf16 375, 332 and 273 us, 8-bit 427, 341 and 330: two
// rings fill a CU whatever the heads, so few heads are few waves.  32 heads over 64
// whole sequences of 4K to 64K bf16 tokens: 417-437 us, 6.1 TB/s of rows; 8-bit 351.
// 64 tokens x 64 heads x 2048 8-bit slots 43-45 + 9 us, of which the
// rows are 19 us of traffic and writing and joining 256 parts of 128 KB about 18.
// One token x 32 heads x 2048 slots 12-13 + 4 us, one tile 10.6 + 4.

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

// A split launch's tiles, dealt evenly: the first `more` shares hold each + 1,
// the others `each`, in order.  (32-bit divisions: a 64-bit one is hundreds of
// instructions, which a launch of a few tiles waits for to be fetched.)
struct Shares {
  uint32_t count, each, more;
  __device__ __forceinline__ explicit Shares(const AttendArgs& a, uint32_t tiles) {
    const uint32_t most = tiles / kShareTiles;
    count = most < 1 ? 1 : most < (uint32_t)a.wgs ? most : (uint32_t)a.wgs;
    each = tiles / count;
    more = tiles - each * count;
  }
  __device__ __forceinline__ int begin(uint32_t share) const { return (int)(share * each + (share < more ? share : more)); }
  // the share that holds a tile
  __device__ __forceinline__ int owner(uint32_t tile) const {
    const uint32_t longer = more * (each + 1);
    return (int)(tile < longer ? tile / (each + 1) : more + (tile - longer) / each);
  }
};

// Where the keys of a token come from.
struct TokenKeys {
  int64_t token;
  int64_t len;               // keys (positions, or k)
  const int32_t* list;       // the token's slots, or its request's pages
};

// Where the list's entry for this lane's key (lane % 32) of a tile is: its
// slot, or its page.  Past the keys (of which there are some), the last one's.
template <bool PAGED>
__device__ __forceinline__ const int32_t* entry_of(const AttendArgs& a, const TokenKeys& tk, int64_t tile) {
  int64_t pos = tile * kTileKeys + (lane_here() & (kTileKeys - 1));
  pos = pos < tk.len ? pos : tk.len - 1;
  return tk.list + (PAGED ? pos >> a.log2_page : pos);      // (a token's keys are within its row of the page table)
}

// The slot of that key, or -1 when it selects nothing.
template <bool PAGED>
__device__ __forceinline__ int slot_of(const AttendArgs& a, const TokenKeys& tk, int entry, int64_t tile) {
  const int64_t pos = tile * kTileKeys + (lane_here() & (kTileKeys - 1));
  int64_t slot = entry;
  if (PAGED && entry >= 0) slot = ((int64_t)entry << a.log2_page) + (pos & (((int64_t)1 << a.log2_page) - 1));
  return pos < tk.len && slot >= 0 && slot < a.cache.num_slots ? (int)slot : -1;
}

// Tiles of [first, last) up to the last one that has a selected key; wave-uniform.
constexpr int kScan = 256;             // entries looked at together
struct ScanBlock {
  int slot[kScan / 64];
};
__device__ __forceinline__ void load_scan(const TokenKeys& tk, int64_t begin, int64_t base, int lane, ScanBlock& s) {
#pragma unroll
  for (int i = 0; i < kScan / 64; ++i) {
    const int64_t at = base - 1 - i * 64 - lane;
    s.slot[i] = at >= begin ? tk.list[at] : -1;
  }
}
__device__ __forceinline__ int64_t scan_begin(int64_t first) { return first * kTileKeys; }
__device__ __forceinline__ int64_t scan_end(const TokenKeys& tk, int64_t last) {
  return last * kTileKeys < tk.len ? last * kTileKeys : tk.len;
}
// s: the last block's entries.
__device__ __forceinline__ int64_t selected_tiles(const AttendArgs& a, const TokenKeys& tk, int64_t first, int64_t last,
                                                  ScanBlock& s, int lane) {
  const int64_t begin = scan_begin(first);
  for (int64_t base = scan_end(tk, last); base > begin; base -= kScan) {
    uint64_t any[kScan / 64];
#pragma unroll
    for (int i = 0; i < kScan / 64; ++i) any[i] = __ballot(s.slot[i] >= 0 && s.slot[i] < a.cache.num_slots);
#pragma unroll
    for (int i = 0; i < kScan / 64; ++i)
      if (any[i]) return (base - 1 - i * 64 - (int64_t)__builtin_ctzll(any[i])) / kTileKeys - first + 1;
    load_scan(tk, begin, base - kScan, lane, s);
  }
  return 0;
}

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

// The softmax step and the second product of a tile whose scores are s.
// mask: the tile's selected keys.
template <bool E4M3>
__device__ __forceinline__ void weigh_tile(HeadState& st, f32x4 (&s)[2], uint32_t lat, uint32_t scales,
                                           uint32_t mask, float scale_log2, const TileReads& at, int lane) {
  const int g = lane >> 4;
  if (mask != 0xFFFFFFFFu) {
    const uint32_t own = mask >> (4 * g);
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
  // each, as large as the rounding of the result itself.  The sum keeps them in fp32.
  bf16x8 p;
  float sum = 0.f;                        // a tile at a time: few additions to a large number
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    f32x4 w;
#pragma unroll
    for (int r = 0; r < 4; ++r) w[r] = __builtin_amdgcn_exp2f(fmaf(s[b][r], scale_log2, -st.m));
    sum += (w[0] + w[1]) + (w[2] + w[3]);
    if (E4M3) w *= read_lds<f32x4>(scales + 64 * b + 16 * g);
#pragma unroll
    for (int r = 0; r < 4; ++r) p[4 * b + r] = (__bf16)w[r];
  }
  st.l += sum;
  const uint32_t value = (uint32_t)here(at.value + (int)lat);
  auto use = [&](int cb, bf16x8 cols) { st.o[cb] = mfma16(cols, p, st.o[cb]); };
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

// Last of the n ascending starts at or below v, 64 at a time; wave-uniform.
__device__ __forceinline__ int64_t count_starts(const int32_t* starts, int64_t n, int64_t v, int lane) {
  int64_t c = 0;
  for (int64_t base = 1; base <= n; base += 64) {
    const int64_t at = base + lane;
    const int got = __popcll(__ballot(at <= n && (int64_t)starts[at <= n ? at : n] <= v));
    c += got;
    if (got < 64) break;
  }
  return c;
}

// Keys that token t, of request b, attends; those past the page table's row
// have no page.
__device__ __forceinline__ int64_t token_len(const AttendArgs& a, int64_t t, int64_t b) {
  const int64_t len = (int64_t)a.seq_lens[b] - ((int64_t)a.q_starts[b + 1] - t) + 1;
  const int64_t most = a.pages_per_row << a.log2_page;
  return len < 0 ? 0 : (len < most ? len : most);
}

// A split launch's plan of whole sequences: the tiles before each token, and its request.
struct SplitPlan {
  int32_t start[kPlanTokens + 1];
  uint16_t request[kPlanTokens];
};

// A token's tiles; one even when it has no key, so that somebody writes its row.
__device__ __forceinline__ int64_t token_tiles(int64_t len) {
  const int64_t n = (len + kTileKeys - 1) / kTileKeys;
  return n > 0 ? n : 1;
}

template <int NW>
__device__ void plan_split(const AttendArgs& a, SplitPlan& plan, int tid) {
  const int T = a.num_tokens;
  for (int t = tid; t <= T; t += 64 * NW) plan.start[t] = 0;
  lds_barrier();
  // request index + 1 at each request's first token, then carried along
  for (int b = tid; b < a.num_requests; b += 64 * NW) {
    const int q0 = a.q_starts[b], q1 = a.q_starts[b + 1];
    if (q1 > q0 && q0 >= 0 && q0 < T) plan.start[q0] = b + 1;
  }
  lds_barrier();
  const int end = a.q_starts[a.num_requests];
  if (tid < 64) {
    int carry = 0;
    for (int base = 0; base < T; base += 64) {
      const int t = base + tid;
      int v = t < T ? plan.start[t] : 0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (tid >= d) v = v > o ? v : o;
      }
      v = v > carry ? v : carry;
      carry = __shfl(v, 63);
      if (t < T) plan.request[t] = (uint16_t)(v > 0 ? v - 1 : 0);
    }
    int sum = 0;
    for (int base = 0; base < T; base += 64) {
      const int t = base + tid;
      int n = 0;
      if (t < T && t < end) n = (int)token_tiles(token_len(a, t, plan.request[t]));
      int v = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (tid >= d) v += o;
      }
      if (t < T) plan.start[t] = sum + v - n;
      sum += __shfl(v, 63);
    }
    if (tid == 0) plan.start[T] = sum;
  }
  lds_barrier();
}

// A wave's 16 rows of the output by way of LDS (`own`, the wave's), half a row
// at a time: a lane holds 8-byte pieces of one row, and writes 16 bytes of
// contiguous ones (16-byte chunks are flipped with their row, against bank conflicts).
constexpr int kOutBytes = kHeads * kLatent;
__device__ __forceinline__ void write_heads(const AttendArgs& a, int64_t token, int head0, const HeadState& st, float l,
                                            char* own) {
  const int lane = lane_here(), i = lane & 15, group = lane >> 4, chunk = lane & 31;
  const float inv = inverse_sum(l);
  const int64_t row = token * a.num_heads + head0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int c = 0; c < kColBlocks / 2; ++c) {
      bf16x4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = (__bf16)(st.o[half * (kColBlocks / 2) + c][r] * inv);
      *reinterpret_cast<bf16x4*>(own + i * kLatent + (((2 * c + (group >> 1)) ^ i) << 4) + (group & 1) * 8) = v;
    }
#pragma unroll
    for (int n = 0; n < kHeads / 2; ++n) {
      const int r = 2 * n + (lane >> 5);
      const uint4 v = *reinterpret_cast<const uint4*>(own + r * kLatent + ((chunk ^ r) << 4));
      if (head0 + r < a.num_heads)
        *reinterpret_cast<uint4*>(a.out + (row + r) * kLatent + half * (kLatent / 2) + chunk * 8) = v;
    }
  }
  if (a.lse && group == 0 && head0 + i < a.num_heads) a.lse[row + i] = log_sum(st.m, l);
}

template <int NW, int RINGS, bool E4M3, bool PAGED>
__global__ __launch_bounds__(64 * NW * RINGS, 2) void attend_kernel(AttendArgs a) {
  using L = Lds<NW, RINGS, E4M3>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) % NW, ring = __builtin_amdgcn_readfirstlane(tid >> 6) / NW;
  const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds + ring * L::kRingBytes;
  // Workgroups are dealt to the 8 XCDs in turn.  The head blocks of the same keys
  // follow each other on one XCD, so that all but the first find the rows in its L2.
  const int blocks = (a.num_heads + kHeads * NW - 1) / (kHeads * NW);
  const int xcd = blockIdx.x & 7, nth = (int)((blockIdx.x >> 3) / (unsigned)blocks);
  const int block = (int)(blockIdx.x >> 3) - nth * blocks;
  const bool live_wave = (block * NW + wave) * kHeads < a.num_heads;
  constexpr bool split = RINGS > 1;
  const int share = nth * 8 + xcd;      // split: this workgroup's number among those of its head block

  // this workgroup's tiles [lo, hi) of all tokens' tiles, beginning in token
  // t, whose first tile is number `start` and whose request is b
  int lo = 0, hi = INT32_MAX, start = 0;
  int64_t t, b = 0;
  uint32_t total = 0;
  if (split) {
    const uint32_t k_tiles = (uint32_t)token_tiles(a.k);
    if (PAGED) {
      plan_split<NW * RINGS>(a, *reinterpret_cast<SplitPlan*>(lds), tid);
      total = (uint32_t)__builtin_amdgcn_readfirstlane(reinterpret_cast<SplitPlan*>(lds)->start[a.num_tokens]);
    } else {
      total = (uint32_t)a.num_tokens * k_tiles;
    }
    const Shares shares(a, total);
    if ((uint32_t)share >= shares.count) return;
    lo = __builtin_amdgcn_readfirstlane(shares.begin(share));
    hi = __builtin_amdgcn_readfirstlane(shares.begin(share + 1));
    if (PAGED) {
      const SplitPlan& plan = *reinterpret_cast<SplitPlan*>(lds);
      int l = 0, h = a.num_tokens;
      while (h - l > 1) {
        const int mid = (l + h) >> 1;
        if (plan.start[mid] <= lo) l = mid; else h = mid;
      }
      t = __builtin_amdgcn_readfirstlane(l);
      start = __builtin_amdgcn_readfirstlane(plan.start[t]);
      b = __builtin_amdgcn_readfirstlane((int)plan.request[t]);
    } else {
      t = __builtin_amdgcn_readfirstlane((uint32_t)lo / k_tiles);
      start = (int)t * (int)k_tiles;
    }
  } else {
    // neighbouring tokens select neighbouring rows: each XCD takes a contiguous
    // share of the tokens
    const int64_t per = ((int64_t)a.num_tokens + 7) / 8;
    t = xcd * per + nth;
    if (nth >= per || t >= a.num_tokens) return;
    if (PAGED && t >= (int64_t)a.q_starts[a.num_requests]) return;
    if (PAGED) b = count_starts(a.q_starts, a.num_requests, t, lane);
  }

  const TileReads reads = tile_reads<E4M3>(lane);
  const float scale_log2 = fabsf(a.scale_log2);
  while (lo < hi) {
    // the part [first, last) of token t's n tiles
    TokenKeys tk;
    tk.token = t;
    if (PAGED) {
      while (t >= (int64_t)a.q_starts[b + 1]) ++b;
      tk.len = token_len(a, t, b);
      tk.list = a.page_table + b * a.pages_per_row;
    } else {
      tk.len = a.k;
      tk.list = a.indices + t * a.k;
    }
    const int n = (int)token_tiles(tk.len);
    const int first = lo - start, last = hi - start < n ? hi - start : n;
    const bool whole = first == 0 && last == n;

    // The ring: this wave's tiles are first + ring + RINGS i, tile i in stage i %
    // kStages; masks[d], the selected keys of the tile d after the one being
    // computed.  A tile's list entries are loaded one tile before its rows.
    // Entries (and scales) too are loaded into LDS, so that no load in the loop is
    // the compiler's to wait for: it would wait for the rows queued behind it.
    uint32_t masks[L::kAhead + 1];
    int into = 0;                         // the stage of the tile to be queued next
    const uint32_t own_entries = lds_base + L::kEntries + wave * 256;
    const uint32_t scales = lds_base + L::kScales + wave * L::kStages * 128;
    auto tile_of = [&](int i) { return (int64_t)(first + ring + RINGS * i); };
    auto load_entries = [&](int i) {
      queue_words_to_lds(entry_of<PAGED>(a, tk, tile_of(i)), own_entries + (uint32_t)(i & 1) * 128);
    };
    lds_barrier();                        // the last part's reads are done
    if (tk.len > 0) load_entries(0);
    ScanBlock scan;
    if (!PAGED) load_scan(tk, scan_begin(first), scan_end(tk, last), lane_here(), scan);

    // the queries (of a head past the last, the last's), on their way while the entries are waited for and the first rows queued
    uint4 q[kLatentSteps + kRopeSteps];
    {
      const int l = lane_here(), h = (block * NW + wave) * kHeads + (l & 15);
      const uint16_t* from = a.q + t * a.q_token_stride + (int64_t)(h < a.num_heads ? h : a.num_heads - 1) * a.q_head_stride +
                             (l >> 4) * 8;
#pragma unroll
      for (int k = 0; k < kLatentSteps + kRopeSteps; ++k) {
        q[k] = *reinterpret_cast<const uint4*>(from + k * 32);
      }
    }
    // Tiles past the part's last selected key hold nothing (a short row's tail).
    const int64_t tiles = PAGED ? (tk.len > 0 ? last - first : 0) : selected_tiles(a, tk, first, last, scan, lane_here());
    const int mine = __builtin_amdgcn_readfirstlane((int)tiles) - ring;        // this ring's are the i with RINGS i < mine
    auto queue = [&](int i, uint32_t& mask) {
      const int entry = read_lds<int>(own_entries + (uint32_t)(i & 1) * 128 + (lane_here() & 31) * 4);
      const int slot = slot_of<PAGED>(a, tk, entry, tile_of(i));
      mask = (uint32_t)__ballot(slot >= 0);
      if (RINGS * (i + 1) < mine) load_entries(i + 1);
      if (E4M3) {
        const float* at = slot >= 0 ? a.cache.scale + slot : reinterpret_cast<const float*>(kZeroRow);
        queue_words_to_lds(at, scales + into * 128);
      }
      load_tile<NW, E4M3>(a.cache, slot, lds_base + into * L::kStageBytes, wave);
      into = into + 1 < L::kStages ? into + 1 : 0;
    };
    // The entries: with selected slots, whose scan was loaded after them, they are there.
    if (PAGED) wait_loads<kLatentSteps + kRopeSteps>();
#pragma unroll
    for (int d = 0; d < L::kAhead; ++d) {
      masks[d] = 0;
      if (RINGS * d < mine) {
        queue(d, masks[d]);
        if (d + 1 < L::kAhead) wait_loads<L::kLoads>();        // the next entries
      }
    }
    HeadState st;
    st.m = kNoMax;
    st.l = 0.f;
#pragma unroll
    for (int cb = 0; cb < kColBlocks; ++cb) st.o[cb] = f32x4{};
    // a negative scale goes into the signs of q: the largest product is then the largest score
    const uint32_t sign = a.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int k = 0; k < kLatentSteps + kRopeSteps; ++k)
      st.q[k] = __builtin_bit_cast(bf16x8, make_uint4(q[k].x ^ sign, q[k].y ^ sign, q[k].z ^ sign, q[k].w ^ sign));
    int from = 0;                         // the stage of the tile being computed
    for (int i = 0; RINGS * i < mine + ring; ++i) {
      if (L::kAhead > 1 && RINGS * (i + 1) < mine)
        wait_loads<L::kLoads>();          // all but the next tile's rows
      else
        wait_loads<0>();
      lds_barrier();            // every wave's rows are there, and nobody reads the stage before any more
      if (RINGS > 1 && RINGS * i >= mine) break;               // (in the last round only)
      masks[L::kAhead] = 0;
      if (RINGS * (i + L::kAhead) < mine) queue(i + L::kAhead, masks[L::kAhead]);
      const uint32_t mask = masks[0];
#pragma unroll
      for (int d = 0; d < L::kAhead; ++d) masks[d] = masks[d + 1];
      const uint32_t stage = lds_base + from * L::kStageBytes, sc = scales + from * 128;
      from = from + 1 < L::kStages ? from + 1 : 0;
      f32x4 s[2];
      score_tile<E4M3>(st, s, stage, sc, reads, lane);
      weigh_tile<E4M3>(st, s, stage, sc, mask, scale_log2, reads, lane);
    }

    if (RINGS > 1) {
      // the second ring's waves hand theirs to the first's
      f32x4* other_o = reinterpret_cast<f32x4*>(lds + wave * (kHeads * kLatent * 4)) + lane;
      float2* other_ml = reinterpret_cast<float2*>(lds + NW * (kHeads * kLatent * 4) + wave * 512) + lane;
      lds_barrier();
      if (ring > 0) {
#pragma unroll
        for (int cb = 0; cb < kColBlocks; ++cb) other_o[cb * 64] = st.o[cb];
        *other_ml = make_float2(st.m, st.l);
      }
      lds_barrier();
      if (ring == 0) {
        const float2 ml = *other_ml;
        const float m = fmaxf(st.m, ml.x);
        const float f = __builtin_amdgcn_exp2f(st.m - m), g = __builtin_amdgcn_exp2f(ml.x - m);
        st.m = m;
        st.l = st.l * f + ml.y * g;
#pragma unroll
        for (int cb = 0; cb < kColBlocks; ++cb) st.o[cb] = st.o[cb] * f + other_o[cb * 64] * g;
      }
    }
    const bool writes = RINGS == 1 || ring == 0;

    // this lane's head: its sum is spread over four lanes
    const float l = sum_of_4(st.l);
    if (whole) {
      if (RINGS == 1) lds_barrier();      // nobody reads the stages any more
      if (writes && live_wave) write_heads(a, t, (block * NW + wave) * kHeads, st, l, lds + wave * (RINGS > 1 ? kHeads * kLatent * 4 : kOutBytes));
      if (split && tid == 0 && block == 0) {
        a.part_rec[2 * t] = 0;
        a.part_rec[2 * t + 1] = 1;
      }
    } else {
      // a part that begins its token is this workgroup's last, any other its first
      const int64_t slot = first == 0 ? a.wgs + share : share;
      const int64_t at = ((int64_t)block * 2 * a.wgs + slot) * NW + wave;
      if (writes && live_wave) {
        float* o = a.part_out + at * (kHeads * kLatent) + lane * 4;
#pragma unroll
        for (int cb = 0; cb < kColBlocks; ++cb) *reinterpret_cast<f32x4*>(o + cb * 256) = st.o[cb];
        if (lane < kHeads) a.part_ml[at * kHeads + lane] = make_float2(st.m, l);
      }
      if (first == 0 && tid == 0 && block == 0) {
        uint32_t again = total;           // (worked out here, not kept through the part)
        asm volatile("" : "+s"(again));
        const int g1 = Shares(a, again).owner((uint32_t)(start + n - 1));
        a.part_rec[2 * t] = share;
        a.part_rec[2 * t + 1] = g1 - share + 1;
      }
    }
    if (!split) return;
    lo = start + last;
    start += n;
    ++t;
  }
}

// Joins the parts of a token: out = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p.
// A workgroup takes 16 heads and kJoinBlocks blocks of 16 latent values; its
// waves take every fourth part each, with a running reference as in the main
// kernel and kJoinAhead parts' loads in flight, and are then joined through
// LDS.  Elements stay in the accumulators' order, so reads are contiguous.
// (With one part at a time a token in 64 parts took 22 us, all latency.)
constexpr int kJoinWaves = 4;
constexpr int kJoinAhead = 4;
constexpr int kJoinBlocks = 4;

struct JoinState {
  f32x4 o[kJoinBlocks];
  float m, l;
  __device__ __forceinline__ void add(float pm, float pl, const f32x4 (&po)[kJoinBlocks]) {
    const float to = fmaxf(m, pm);
    const float f = __builtin_amdgcn_exp2f(m - to), g = __builtin_amdgcn_exp2f(pm - to);
    m = to;
    l = l * f + pl * g;
#pragma unroll
    for (int i = 0; i < kJoinBlocks; ++i) o[i] = o[i] * f + po[i] * g;
  }
};

template <int NW>
__global__ __launch_bounds__(64 * kJoinWaves) void join_kernel(AttendArgs a) {
  __shared__ f32x4 others_o[kJoinWaves - 1][kJoinBlocks][64];
  __shared__ float2 others_ml[kJoinWaves - 1][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  const int heads = blockIdx.y, cb0 = blockIdx.z * kJoinBlocks;
  if (!a.indices && t >= (int64_t)a.q_starts[a.num_requests]) return;
  const int g0 = a.part_rec[2 * t], parts = a.part_rec[2 * t + 1];
  if (parts <= 1) return;
  const int64_t base = (int64_t)(heads / NW) * 2 * a.wgs;
  const int i = lane & 15, group = lane >> 4;
  auto place = [&](int p) { return (base + (p == 0 ? a.wgs + g0 : g0 + p)) * NW + heads % NW; };
  JoinState st;
  st.m = kNoMax;
  st.l = 0.f;
#pragma unroll
  for (int c = 0; c < kJoinBlocks; ++c) st.o[c] = f32x4{};
  for (int p0 = w; p0 < parts; p0 += kJoinWaves * kJoinAhead) {
    float2 ml[kJoinAhead];
    f32x4 o[kJoinAhead][kJoinBlocks];
#pragma unroll
    for (int d = 0; d < kJoinAhead; ++d) {
      const int p = p0 + d * kJoinWaves;
      const int64_t at = place(p < parts ? p : p0);
      ml[d] = a.part_ml[at * kHeads + i];
#pragma unroll
      for (int c = 0; c < kJoinBlocks; ++c)
        o[d][c] = *reinterpret_cast<const f32x4*>(a.part_out + at * (kHeads * kLatent) + (cb0 + c) * 256 + lane * 4);
    }
#pragma unroll
    for (int d = 0; d < kJoinAhead; ++d)
      if (p0 + d * kJoinWaves < parts) st.add(ml[d].x, ml[d].y, o[d]);
  }
  if (w > 0) {
#pragma unroll
    for (int c = 0; c < kJoinBlocks; ++c) others_o[w - 1][c][lane] = st.o[c];
    others_ml[w - 1][lane] = make_float2(st.m, st.l);
  }
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int other = 0; other < kJoinWaves - 1; ++other) {
    const float2 ml = others_ml[other][lane];
    f32x4 o[kJoinBlocks];
#pragma unroll
    for (int c = 0; c < kJoinBlocks; ++c) o[c] = others_o[other][c][lane];
    st.add(ml.x, ml.y, o);
  }
  const int head = heads * kHeads + i;
  if (head >= a.num_heads) return;
  const float inv = inverse_sum(st.l);
  const int64_t row = t * a.num_heads + head;
#pragma unroll
  for (int c = 0; c < kJoinBlocks; ++c) {
    bf16x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = (__bf16)(st.o[c][r] * inv);
    *reinterpret_cast<bf16x4*>(a.out + row * kLatent + (cb0 + c) * 16 + 4 * group) = v;
  }
  if (a.lse && cb0 == 0 && group == 0) a.lse[row] = log_sum(st.m, st.l);
}

int ceil_div(int a, int b) { return (int)(((int64_t)a + b - 1) / b); }

template <int NW, int RINGS, bool E4M3>
hipError_t launch(const AttendArgs& a, hipStream_t stream) {
  const int64_t shares = ceil_div(a.wgs > 0 ? a.wgs : a.num_tokens, 8);
  const dim3 grid((unsigned)(shares * 8 * ceil_div(a.num_heads, kHeads * NW))), block(64 * NW * RINGS);
  constexpr int kLds = Lds<NW, RINGS, E4M3>::kBytes;
  static_assert(sizeof(SplitPlan) <= (size_t)kLds, "the plan is made where the rows go");
  if (a.indices)
    hipLaunchKernelGGL((attend_kernel<NW, RINGS, E4M3, false>), grid, block, kLds, stream, a);
  else
    hipLaunchKernelGGL((attend_kernel<NW, RINGS, E4M3, true>), grid, block, kLds, stream, a);
  return hipGetLastError();
}

template <int NW, bool E4M3>
hipError_t launch(const AttendArgs& a, hipStream_t stream) {
  if (a.wgs == 0) return launch<NW, 1, E4M3>(a, stream);
  const hipError_t e = launch<NW, 2, E4M3>(a, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(join_kernel<NW>, dim3((unsigned)a.num_tokens, (unsigned)ceil_div(a.num_heads, kHeads), kColBlocks / kJoinBlocks),
                     dim3(64 * kJoinWaves), 0, stream, a);
  return hipGetLastError();
}

template <bool E4M3>
hipError_t launch_heads(const AttendArgs& a, hipStream_t stream) {
  switch (attend_waves(a.num_heads)) {
    case 1: return launch<1, E4M3>(a, stream);
    case 2: return launch<2, E4M3>(a, stream);
    default: return launch<4, E4M3>(a, stream);
  }
}

}  // namespace

int attend_waves(int num_heads) {
  const int groups = ceil_div(num_heads, kHeads);
  return groups <= 1 ? 1 : (groups <= 2 ? 2 : 4);
}

int attend_heads(int num_heads) { return kHeads * attend_waves(num_heads); }

int64_t attend_threads(int num_tokens, int num_heads) {
  const int64_t wgs = (int64_t)ceil_div(num_tokens, 8) * 8 * ceil_div(num_heads, attend_heads(num_heads));
  if (wgs > kMaxThreads) return wgs;
  const int64_t own = wgs * 64 * attend_waves(num_heads);
  const int64_t join = (int64_t)num_tokens * 64 * kJoinWaves;   // of a split launch: with 17 to 32 heads for any number of tokens
  return attend_waves(num_heads) == 2 && join > own ? join : own;
}

SplitLayout split_layout(int num_tokens, int num_heads, int wgs) {
  const int nw = attend_waves(num_heads);
  const size_t parts = (size_t)2 * wgs * ceil_div(num_heads, kHeads * nw) * nw;   // of one wave
  SplitLayout s;
  s.out_bytes = parts * kHeads * kLatent * sizeof(float);
  s.ml_bytes = parts * kHeads * sizeof(float2);
  s.rec_bytes = ((size_t)num_tokens * 2 * sizeof(int32_t) + 15) / 16 * 16;
  return s;
}

hipError_t launch_attend(const AttendArgs& a, bool e4m3, hipStream_t stream) {
  return e4m3 ? launch_heads<true>(a, stream) : launch_heads<false>(a, stream);
}

}  // namespace latent
