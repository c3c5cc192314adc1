// Device helpers shared by the two latent attention kernels: matrix core and
// transposed LDS reads, the LDS chunk swizzle, asynchronous loads into LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace latent {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// 32x32x16 bf16 products summed in fp32.  Lane l = 32 hb + i.  Operands: a
// holds A[i][8 hb + (0..7)], b holds B[8 hb + (0..7)][i].  Accumulator register
// r holds C[8 (r / 4) + 4 hb + r % 4][i].
__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Row of accumulator register r (0..15) in half-wave hb.
__device__ __forceinline__ int acc_row(int r, int hb) { return 8 * (r >> 2) + 4 * hb + (r & 3); }

// LDS rows are cut in 16-byte chunks, and chunk c of a row sits at c ^
// swizzle(row) (the xor stays within 16 chunks, 256 bytes).  Two reads have
// to spread over the banks: 16-byte reads of one chunk of 8 consecutive rows
// (the low three bits take 8 values), and the transposed reads, whose 16
// lanes cover 32 bytes (a chunk pair) of 4 consecutive rows (the pair bits
// take 4 values): so the row's low two bits pick the pair, the third the
// chunk within it.
__device__ __forceinline__ int swizzle(int row) {
  return ((row & 3) << 1) | ((row >> 2) & 1) | (row & 8);
}

// Transposed read: the 16 lanes j of a quarter-wave name 4 rows of 16 16-bit
// columns, lane j the 8 bytes of row j / 4, columns 4 (j % 4) .. + 3, and lane
// j gets column j of the 4 rows.
__device__ __forceinline__ bf16x4 read_tr(const char* lds) {
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)lds));
}

__device__ __forceinline__ bf16x8 join8(bf16x4 lo, bf16x4 hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 16 bytes per lane from src (a per-lane address) into LDS at dst + 16 * lane
// (dst the same for the wave).  Asynchronous: counted by vmcnt.
__device__ __forceinline__ void load_to_lds(const char* src, char* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// Workgroup barrier that leaves vector loads in flight (they are waited for
// by count where their data is used).  LDS accesses before it have completed.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Value of the other half-wave's lane (l ^ 32).
__device__ __forceinline__ float other_half(float v, int lane) {
  const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(lane < 32 ? sw[1] : sw[0]);
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// Initial reference maximum of a running softmax: finite, so that masked
// scores (-inf) give weights of exactly 0 and never inf - inf.
constexpr float kNoMax = -1e30f;
// The running reference is moved only when a score passes it by more than
// 2^kLazy: weights then reach at most 2^kLazy, and the accumulators are
// rescaled a few times a row rather than at every tile.
constexpr float kLazy = 8.0f;

}  // namespace latent
