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
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// 32x32x16 bf16 products summed in fp32.  Lane l = 32 hb + i.  Operands: a
// holds A[i][8 hb + (0..7)], b holds B[8 hb + (0..7)][i].  Accumulator register
// r holds C[8 (r / 4) + 4 hb + r % 4][i].
__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 16x16x32 bf16 products summed in fp32.  Lane l = 16 g + i.  Operands: a holds
// A[i][8 g + (0..7)], b holds B[8 g + (0..7)][i].  Accumulator register r holds
// C[4 g + r][i].
__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Row of accumulator register r (0..15) of a 32x32 product in half-wave hb.
__device__ __forceinline__ int acc_row(int r, int hb) { return 8 * (r >> 2) + 4 * hb + (r & 3); }

// LDS rows are cut in 16-byte chunks, and chunk c of a row sits at c ^
// swizzle(row) (the xor stays within 16 chunks: 256 bytes, all 64 banks).  Reads
// that have to spread over the banks:
//   * 16 bytes a lane, 16 lanes at a time, lanes 0..3, 12..15, 20..23, 24..27 of a
//     half-wave and the rest: with lane = row that is 16 rows of one chunk, any
//     one-to-one map; with lane = 16 g + row and chunk c + g, rows 0..3 and
//     12..15 of c and rows 4..11 of c + 1, so a row's partner within a chunk
//     pair has to be row ^ 12;
//   * transposed, 32 lanes at a time: a chunk pair of 8 rows, or two neighbouring pairs of
//     4 rows, so rows differ in the pair's number, bits 0 and 1 of the row in
//     its upper two bits.
// Both hold for this linear map (and for rotary rows, 8 chunks and two rows to 256
// bytes, with chunk ^ row / 2).  (A map that missed the second lost half of all LDS
// cycles to conflicts, one that missed the first a quarter.)
__device__ __forceinline__ int swizzle(int row) {
  return ((row & 3) << 2) ^ ((row >> 1) & 2) ^ ((row >> 3) & 1) * 3;
}

// LDS reads by byte address.
template <typename T>
__device__ __forceinline__ T read_lds(uint32_t at) {
  typedef const __attribute__((address_space(3))) T* lds_ptr;
  return *(lds_ptr)at;
}

// Transposed read: the 16 lanes j of a quarter-wave name 4 rows of 16 16-bit
// columns, lane j the 8 bytes of row j / 4, columns 4 (j % 4) .. + 3, and lane
// j gets column j of the 4 rows.
__device__ __forceinline__ bf16x4 read_tr(uint32_t at) {
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)at));
}

// The same for 8-bit elements: lane j names 8 bytes (columns 8 (j % 2) .. + 7) of
// row j / 2 of 8, and gets column j of the 8 rows.
__device__ __forceinline__ u32x2 read_tr8(uint32_t at) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) i32x2* lds_ptr;
  const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_ptr)at);
  return __builtin_bit_cast(u32x2, v);
}

// Eight E4M3 codes as bf16, exactly.
__device__ __forceinline__ bf16x8 widen8(u32x2 codes) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.x, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.x, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.y, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.y, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ bf16x8 join8(bf16x4 lo, bf16x4 hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The lane's number, worked out where it is used (nothing is kept in a register for it).
__device__ __forceinline__ int lane_here() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
  return l;
}

// 16 bytes per lane from src (a per-lane address) into LDS at dst + 16 * lane
// (dst the same for the wave).  Asynchronous: counted by vmcnt.
__device__ __forceinline__ void load_to_lds(const char* src, char* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// The same, as instructions that the compiler does not count among its own
// loads: it puts a wait for all loads in front of an LDS read that may follow a
// load into the same array, and a ring of stages in one array is such.  The
// caller waits (wait_loads) and passes a barrier before it reads the bytes.
// lds: byte address in LDS.
__device__ __forceinline__ void queue_to_lds(const char* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(src), "s"(lds) : "m0", "memory");
}

// 4 bytes per lane of the lower half-wave, to lds + 4 * lane.
__device__ __forceinline__ void queue_words_to_lds(const void* src, uint32_t lds) {
  if (lane_here() < 32)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :: "v"(src), "s"(lds) : "m0", "memory");
}

// Waits until at most N of this wave's vector loads are in flight (they complete in order).
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

// Workgroup barrier that leaves vector loads in flight (they are waited for
// by count where their data is used).  LDS accesses before it have completed.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A run of N matrix instructions whose LDS reads are issued D instructions
// ahead: read(i) gives what step i takes from LDS, widen() of it the operand
// (one step ahead, so that no matrix instruction waits for the conversion right
// before it), use(i, operand) multiplies.  The compiler, left alone with few
// registers to spare, places each read right in front of its use, and every
// matrix instruction then waits for the LDS; the scheduling barriers keep the
// order written here.
__device__ __forceinline__ bf16x8 widen(bf16x8 rows) { return rows; }
__device__ __forceinline__ bf16x8 widen(u32x2 codes) { return widen8(codes); }

template <int N, int D, typename Read, typename Use>
__device__ __forceinline__ void run_ahead(Read read, Use use) {
  decltype(read(0)) held[D];
#pragma unroll
  for (int i = 0; i < D; ++i) held[i] = read(i);
  __builtin_amdgcn_sched_barrier(0);
  bf16x8 operand = widen(held[0]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    bf16x8 next = operand;
    if (i + 1 < N) next = widen(held[(i + 1) % D]);
    use(i, operand);
    if (i + D < N) held[i % D] = read(i + D);
    operand = next;
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Value of the other half-wave's lane (l ^ 32).
__device__ __forceinline__ float other_half(float v, int lane) {
  const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(lane < 32 ? sw[1] : sw[0]);
}

// The same value, computed where it is used: keeps what a rare path derives
// from it out of registers that the common path needs.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Maximum and sum over the four lanes that share lane % 16.  The swaps exchange
// the odd rows of 16 lanes (the upper half-wave) of their first operand with
// the even rows (the lower half) of their second: with both the same value, the
// two results hold a row's own value and its partner's.
__device__ __forceinline__ float max_of_4(float v) {
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float sum_of_4(float v) {
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

constexpr float kLn2 = 0.69314718055994530942f;
// A row's results from its reference m (log2 units) and its sum l: what its
// accumulators are multiplied by, and the logarithm of the sum of exponentials.
// The sum is 0 only where nothing weighs anything: 0 and -inf.  It is NaN where a
// score is NaN or +inf, and so are both results.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.0f / l; }
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2; }

// Initial reference maximum of a running softmax: no finite score is below it, and
// it is finite itself, so that masked scores (-inf) give weights of exactly 0 and
// never inf - inf.
constexpr float kNoMax = -3.40282347e38f;
// The running reference is moved only when a score (log2 units) passes it by more than
// kLazy: weights then reach at most 2^kLazy, and the accumulators are
// rescaled a few times a row rather than at every tile.
constexpr float kLazy = 8.0f;

// A weight's exponent is the product s * scale less the reference, which is such a
// product rounded.  One fused step leaves that rounding in the exponent: the same
// for all keys of a row, so it does no harm up to kFar, where it is at most 1,
// but at 2^31 it reaches 128, and weights overflow or vanish.  A tile whose
// reference is beyond kFar has its products rounded first (and scale 1 after that), so that
// the largest score's distance is exactly 0.
constexpr float kFar = 16777216.0f;

}  // namespace latent
