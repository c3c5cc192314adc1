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

__device__ __attribute__((aligned(16))) const char kZeroRow[kUpBytes] = {};

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

// Queues the loads of a tile's rows from key j0 on; rows past nk are zeros.
__device__ __forceinline__ void load_tile(const PrefillArgs& a, const Block& blk, int64_t head, int64_t j0, Stage& st,
                                          int lane, int wave) {
#pragma unroll
  for (int i = 0; i < kKeys / 2 / kWaves; ++i) {
    const int pair = wave * (kKeys / 2 / kWaves) + i;   // two rows an instruction
    const int key = 2 * pair + (lane >> 5);
    const int p = lane & 31;
    const char* row = j0 + key < blk.nk
        ? reinterpret_cast<const char*>(a.kv + (blk.k0 + j0 + key) * a.kv_token_stride + head * a.kv_head_stride)
        : kZeroRow;
    load_to_lds(row + (p ^ swizzle(key)) * 16, st.up + pair * 2 * kUpBytes);
  }
#pragma unroll
  for (int i = 0; i < kKeys / 8 / kWaves; ++i) {
    const int group = wave * (kKeys / 8 / kWaves) + i;  // eight rotary keys an instruction
    const int key = group * 8 + (lane >> 3);
    const char* row = j0 + key < blk.nk ? reinterpret_cast<const char*>(a.rope + (blk.k0 + j0 + key) * a.rope_stride) : kZeroRow;
    load_to_lds(row + ((lane ^ key) & 7) * 16, st.rope + group * 8 * kRopeBytes);
  }
}

struct RowState {
  bf16x8 q[kHeadSteps + kRopeSteps];
  f32x16 o[kColBlocks];
  float m;      // reference maximum (log2 units)
  float l;      // this lane's part of the sum
};

// One tile for a wave's 32 queries.  limit: the lane's query attends the
// tile's keys below it (any value; at least kKeys: all).
__device__ __forceinline__ void attend_tile(RowState& st, const Stage& t, int limit, bool masked, float scale_log2,
                                            int lane) {
  const int i = lane & 31, hb = lane >> 5;
  f32x16 s[2];
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    s[kb] = f32x16{};
    const char* up = t.up + (32 * kb + i) * kUpBytes;
    const char* rope = t.rope + (32 * kb + i) * kRopeBytes;
    const int sw = swizzle(i);
#pragma unroll
    for (int k = 0; k < kHeadSteps; ++k)
      s[kb] = mfma(*reinterpret_cast<const bf16x8*>(up + (((2 * k + hb) ^ sw) << 4)), st.q[k], s[kb]);
#pragma unroll
    for (int k = 0; k < kRopeSteps; ++k)
      s[kb] = mfma(*reinterpret_cast<const bf16x8*>(rope + ((((2 * k + hb) ^ i) & 7) << 4)), st.q[kHeadSteps + k], s[kb]);
  }
  float top = -INFINITY;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[kb][r] *= scale_log2;
      if (masked && 32 * kb + acc_row(r, hb) >= limit) s[kb][r] = -INFINITY;
      top = fmaxf(top, s[kb][r]);
    }
  top = fmaxf(top, other_half(top, lane));
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
      const float w = __builtin_amdgcn_exp2f(s[kb][r] - st.m);
      st.l += w;
      p[2 * kb + (r >> 3)][r & 7] = (__bf16)w;
    }
  const int j = lane & 15, quarter = (lane >> 4) & 1;
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int cb = 0; cb < kColBlocks; ++cb) {
      const int chunk = cb * 4 + 2 * quarter + ((j & 3) >> 1);
      bf16x4 v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = 16 * k + 8 * e + 4 * hb + (j >> 2);
        v[e] = read_tr(t.up + key * kUpBytes + kUpBytes / 2 + ((chunk ^ swizzle(key)) << 4) + (j & 1) * 8);
      }
      st.o[cb] = mfma(join8(v[0], v[1]), p[k], st.o[cb]);
    }
}

__global__ __launch_bounds__(64 * kWaves, 2) void prefill_kernel(PrefillArgs a, int64_t blocks) {
  __shared__ __attribute__((aligned(16))) Stage stage0, stage1;
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
    const uint16_t* q = a.q + (blk.q0 + row) * a.q_token_stride + head * a.q_head_stride + hb * 8;
#pragma unroll
    for (int k = 0; k < kHeadSteps + kRopeSteps; ++k) {
      st.q[k] = bf16x8{};
      if (live) st.q[k] = *reinterpret_cast<const bf16x8*>(q + k * 16);
    }
  }

  if (wg_keys > 0) load_tile(a, blk, head, 0, stage0, lane, wave);
  auto step = [&](int64_t j0, const Stage& cur, Stage& nxt) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();              // every wave's rows are there, and nobody reads the other stage any more
    if (j0 + kKeys < wg_keys) load_tile(a, blk, head, j0 + kKeys, nxt, lane, wave);
    if (j0 >= wave_most) return;
    const int64_t left = own_keys - j0;
    attend_tile(st, cur, (int)(left < 0 ? 0 : (left < kKeys ? left : kKeys)), j0 + kKeys > wave_least, a.scale_log2, lane);
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
