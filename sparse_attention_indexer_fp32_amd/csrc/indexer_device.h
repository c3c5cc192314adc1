// Device helpers shared by the indexer's scoring kernels: the matrix product of one
// query row's heads with a tile of keys and its epilogue.  Every kernel that goes
// through them gets the same fp32 value for the same query and key.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace indexer {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));


constexpr int kHeads = 32;
constexpr int kDim = 128;

// Eight fp8 codes (two dwords) -> eight bf16 values, exact.
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  bf16x8 r;
  r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
  r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
  return r;
}

// A lane's view of one query row: head h = lane % 32 and the half hb = lane / 32
// of the head dimension it feeds, as bf16, ready for the eight K steps; and
// the 16 head weights its accumulator rows carry.
struct RowOperand {
  bf16x8 a[8];
  float w[16];
};

// Step s of the contraction pairs, on both operands, the 8 values
// d = hb * 64 + s * 8 + (0..7) of the lane's half: every d in [0, 128) is used
// exactly once, and A and B agree on which d sits in which slot.
__device__ __forceinline__ void load_row(const uint8_t* q, const float* weights, int64_t row, bool live, int lane,
                                         RowOperand& op) {
  const int h = lane & 31, hb = lane >> 5;
  if (live) {
    const uint4* src = reinterpret_cast<const uint4*>(q + (row * kHeads + h) * kDim + hb * 64);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = src[i];
      op.a[2 * i] = widen8(v.x, v.y);
      op.a[2 * i + 1] = widen8(v.z, v.w);
    }
    // accumulator register r of this lane holds head (r / 4) * 8 + hb * 4 + r % 4
#pragma unroll
    for (int r = 0; r < 16; ++r) op.w[r] = weights[row * kHeads + (r >> 2) * 8 + hb * 4 + (r & 3)];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) op.a[i] = bf16x8{};
#pragma unroll
    for (int r = 0; r < 16; ++r) op.w[r] = 0.f;
  }
}

// Epilogue of one query row against a tile: relu of each head's dot
// product, the head weights, the partner half-wave's 16 heads, the position's
// scale.  Every lane returns the score of position n = lane % 32 of the tile
// (both half-waves hold it).  The order of the operations is fixed, so every
// kernel that calls this gets the same fp32 value.
//
// relu is a signed-integer max of the value's bits with 0: negative floats
// (and -0) have negative bit patterns and become +0, the rest pass unchanged.
// That is max(x, 0) for every non-NaN x in one instruction (a float max of an
// accumulator costs a quieting max first); a -0 from the float form could not
// change the sum either, which starts at +0.
__device__ __forceinline__ float relu(float x) { return __int_as_float(max(__float_as_int(x), 0)); }

__device__ __forceinline__ float finish_score(const RowOperand& op, const f32x16& acc, float scale, int lane) {
  float part = 0.f;
#pragma unroll
  for (int r = 0; r < 16; ++r) part = fmaf(op.w[r], relu(acc[r]), part);
  // The other 16 heads of the same position sit in lane ^ 32.  The swap
  // exchanges the upper half-wave of its first operand with the lower
  // half-wave of its second: with both = part, lane l < 32 finds lane l + 32
  // in the second result and lane l >= 32 finds lane l - 32 in the first.
  const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(part), __float_as_uint(part), false, false);
  const float other = __uint_as_float(lane < 32 ? sw[1] : sw[0]);
  return (part + other) * scale;
}

}  // namespace indexer
