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

// Block `index` of the requests' blocks of kRows queries; false past the last.
// Wave-uniform, 64 requests at a time.
__device__ __forceinline__ bool find_block(const PrefillArgs& a, int64_t index, int lane, Block& blk) {
  int64_t before = 0;
  for (int64_t base = 0; base < a.num_requests; base += 64) {
    const int64_t b = base + lane;
    int64_t q0 = 0, q1 = 0;
    if (b < a.num_requests) {
      q0 = a.q_starts[b];
      q1 = a.q_starts[b + 1];
    }
    q1 = q1 < a.num_tokens ? q1 : a.num_tokens;
    const int n = q1 > q0 ? (int)((q1 - q0 + kRows - 1) / kRows) : 0;
    int incl = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    const uint64_t hit = __ballot(before + incl > index);
    if (hit) {
      const int src = (int)__builtin_ctzll(hit);
      const int64_t r = base + src;
      const int ahead = __builtin_amdgcn_readlane(incl - n, src);
      blk.first = (index - before - ahead) * kRows;
      blk.q0 = a.q_starts[r];
      const int64_t end = a.q_starts[r + 1];
      blk.nq = (end < a.num_tokens ? end : a.num_tokens) - blk.q0;
      blk.k0 = a.kv_starts[r];
      int64_t k1 = a.kv_starts[r + 1];
      k1 = k1 < a.num_kv ? k1 : a.num_kv;
      blk.nk = k1 > blk.k0 && blk.k0 >= 0 ? k1 - blk.k0 : 0;
      return blk.q0 >= 0;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
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
    const uint32_t key = (uint32_t)here(at.key + (int)stage), rope = (uint32_t)here(at.rope + (int)stage) + kKeys * kUpBytes;
    run_ahead<2 * (kHeadSteps + kRopeSteps), kReadsAhead>(
        [&](int n) {
          const int k = n >> 1, kb = n & 1;
          return read_lds<bf16x8>(k < kHeadSteps ? (key ^ (uint32_t)(k << 5)) + 32 * kb * kUpBytes
                                                 : (rope ^ (uint32_t)((k - kHeadSteps) << 5)) + 32 * kb * kRopeBytes);
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
  if (__any(top > st.m + kLazy)) {
    const float m = fmaxf(st.m, top);
    const float f = __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= f;
#pragma unroll
    for (int cb = 0; cb < kColBlocks; ++cb)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[cb][r] *= f;
  }
  // Weights in bf16 (the matrix cores' type): an unbiased half step of 2^-9 on
  // each, as large as the rounding of the result itself.  The sum keeps them in fp32.
  bf16x8 p[4];
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float w = __builtin_amdgcn_exp2f(fmaf(s[kb][r], scale_log2, -st.m));
      st.l += w;
      if (MASKED) s[kb][r] = w;
      p[2 * kb + ((r >> 2) & 1)][((r >> 3) << 2) + (r & 3)] = (__bf16)w;   // a step: rows 0..3 and 16..19 of each half
    }
  if (MASKED && values_not_finite(t, here(lane))) {
    add_values_one_by_one(st.o, s, t, limit, here(lane));
    return;
  }
  const uint32_t value = (uint32_t)here(at.value + (int)stage);
  run_ahead<4 * kColBlocks, kReadsAhead>(
      [&](int n) {
        // step k: rows 32 (k / 2) + 8 (k % 2) + 4 hb + 0..3 and those 16 on; rows 8 on swizzle with bits 0 and 1 flipped
        const int k = n / kColBlocks, cb = n % kColBlocks;
        const uint32_t v = (value ^ (uint32_t)((cb << 6) ^ (k & 1) * 48)) + (32 * (k >> 1) + 8 * (k & 1)) * kUpBytes;
        return join8(read_tr(v), read_tr(v + 16 * kUpBytes));
      },
      [&](int n, bf16x8 cols) { st.o[n % kColBlocks] = mfma(cols, p[n / kColBlocks], st.o[n % kColBlocks]); });
}

__global__ __launch_bounds__(64 * kWaves, 2) void prefill_kernel(PrefillArgs a, int64_t blocks) {
  __shared__ __attribute__((aligned(256))) Stage stage0, stage1;
  const int lane = threadIdx.x & 63, hb = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Heads in turn, and of a head its last (longest) blocks first; each XCD
  // (workgroups are dealt to the 8 of them in turn) takes a contiguous share,
  // so the blocks of a head, which read the same keys, share an L2.
  const int64_t units = blocks * a.num_heads, per = (units + 7) / 8;
  const int64_t unit = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int64_t)(blockIdx.x >> 3) >= per || unit >= units) return;
  const int64_t head = unit / blocks;
  Block blk;
  if (!find_block(a, blocks - 1 - unit % blocks, lane, blk)) return;

  const int64_t row = blk.first + wave * 32 + (lane & 31);     // the lane's query in its request
  const bool live = row < blk.nq;
  // keys it attends, and the most and fewest any of the wave's and the workgroup's do
  const int64_t shift = blk.nk - blk.nq + 1;
  auto keys_of = [&](int64_t r) {
    const int64_t n = a.causal ? shift + r : blk.nk;
    return n < 0 ? (int64_t)0 : (n < blk.nk ? n : blk.nk);
  };
  const int64_t own_keys = keys_of(row);
  const int64_t last_row = blk.first + kRows < blk.nq ? blk.first + kRows - 1 : blk.nq - 1;
  const int64_t wg_keys = keys_of(last_row);
  const int64_t wave_row = blk.first + wave * 32;
  const int64_t wave_most = wave_row < blk.nq ? keys_of(wave_row + 31 < last_row ? wave_row + 31 : last_row) : 0;
  const int64_t wave_least = keys_of(wave_row);

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
  const float scale_log2 = fabsf(a.scale_log2);

  const TileReads reads = tile_reads(lane);
  const TileLoads loads = tile_loads(a, kKeys, lane, wave);
  const char* up = reinterpret_cast<const char*>(a.kv + blk.k0 * a.kv_token_stride + head * a.kv_head_stride);
  const char* rope = reinterpret_cast<const char*>(a.rope + blk.k0 * a.rope_stride);
  // tiles may reach past the workgroup's keys, but not past the request's
  auto queue = [&](int64_t j0, Stage& st_to) {
    const char* u = up + j0 * a.kv_token_stride * 2;
    const char* r = rope + j0 * a.rope_stride * 2;
    const int64_t rows = blk.nk - j0;
    TileLoads t = loads;
    if (rows < kKeys) t = tile_loads(a, (int)rows, here(lane), wave);
    load_tile(u, r, t, st_to, wave);
  };
  if (wg_keys > 0) queue(0, stage0);
  auto step = [&](int64_t j0, const Stage& cur, Stage& nxt) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();              // every wave's rows are there, and nobody reads the other stage any more
    if (j0 + kKeys < wg_keys) queue(j0 + kKeys, nxt);
    if (j0 >= wave_most) return;
    if (j0 + kKeys <= wave_least) {
      attend_tile<false>(st, cur, reads, kKeys, scale_log2, lane);
    } else {
      const int64_t left = own_keys - j0;
      attend_tile<true>(st, cur, reads, (int)(left < 0 ? 0 : (left < kKeys ? left : kKeys)), scale_log2, lane);
    }
  };
  for (int64_t j0 = 0; j0 < wg_keys; j0 += 2 * kKeys) {
    step(j0, stage0, stage1);
    if (j0 + kKeys < wg_keys) step(j0 + kKeys, stage1, stage0);
  }

  const float l = st.l + other_half(st.l, lane);
  if (!live) return;
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  const int64_t at = (blk.q0 + row) * a.num_heads + head;
  uint16_t* out = a.out + at * kHead + 4 * hb;
#pragma unroll
  for (int cb = 0; cb < kColBlocks; ++cb)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      bf16x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (__bf16)(st.o[cb][4 * g + e] * inv);
      *reinterpret_cast<bf16x4*>(out + cb * 32 + 8 * g) = v;
    }
  if (a.lse && hb == 0) a.lse[at] = l > 0.f ? (st.m + __log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

hipError_t launch_prefill(const PrefillArgs& a, hipStream_t stream) {
  // a request's last block may be partial: at most num_requests blocks beyond the full ones
  const int64_t blocks = a.num_tokens / kRows + (a.num_requests < a.num_tokens ? a.num_requests : a.num_tokens);
  const int64_t grid = (blocks * a.num_heads + 7) / 8 * 8;
  if (grid > (int64_t)INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL(prefill_kernel, dim3((unsigned)grid), dim3(64 * kWaves), 0, stream, a, blocks);
  return hipGetLastError();
}

}  // namespace latent
