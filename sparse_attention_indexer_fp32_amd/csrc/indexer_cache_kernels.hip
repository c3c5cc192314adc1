// The indexer's keys and queries in 8 bits on gfx950: the append of keys to
// their paged cache, the queries in the same form, and cached keys laid in a row.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "indexer_paged_internal.h"

namespace indexer {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kHeads = 32;
constexpr int kDim = 128;
constexpr int kRope = 64;
constexpr int kLanes = 16;                // lanes of a row, 8 values each
constexpr int kThreads = 256;
constexpr int kRowsPerWg = kThreads / kLanes;
constexpr int64_t kMaxWgs = UINT32_MAX / kThreads;   // along x: the hardware counts threads in 32 bits

// ---- a row over 16 lanes ----------------------------------------------------------------------

// A row of 128 values lies in the 16 lanes of a DPP row, lane l holding values
// 8 l .. 8 l + 7 (one 16-byte load): sums, maxima and the mixing's exchanges between
// lanes are DPP moves, and nothing passes through LDS.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kXor3 = 0x1B, kXor7 = 0x141, kXor15 = 0x140;   // quad_perm (3 of them), row_half_mirror, row_mirror

__device__ __forceinline__ float from_xor4(float v) { return dpp<kXor3>(dpp<kXor7>(v)); }
__device__ __forceinline__ float from_xor8(float v) { return dpp<kXor7>(dpp<kXor15>(v)); }

__device__ __forceinline__ float row_sum(float v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kXor7>(v);
  v += dpp<kXor15>(v);
  return v;
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max_u32(v, dpp<kXor1>(v));
  v = max_u32(v, dpp<kXor2>(v));
  v = max_u32(v, dpp<kXor7>(v));
  v = max_u32(v, dpp<kXor15>(v));
  return v;
}

// Eight values of a vector of either type.
__device__ __forceinline__ void load8(const void* from, int fp32, int at, float (&v)[8]) {
  if (fp32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(from) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const bf16x8 h = *reinterpret_cast<const bf16x8*>(static_cast<const __bf16*>(from) + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  }
}

// The angles of a lane's values: interleaved, 4 pairs lie in the lane; by
// halves, value 8 l + j turns with that of lane l ^ 4 by angle (8 l + j) % 32.
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const TurnArgs& t, int64_t pos, int l, Angles& a) {
  if (l >= kRope / 8) return;
  const float* row = t.cos_sin + pos * kRope;
  if (t.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(row + 4 * l);
    const float4 s = *reinterpret_cast<const float4*>(row + kRope / 2 + 4 * l);
    a.c[0] = c.x; a.c[1] = c.y; a.c[2] = c.z; a.c[3] = c.w;
    a.s[0] = s.x; a.s[1] = s.y; a.s[2] = s.z; a.s[3] = s.w;
  } else {
    load8(row, 1, 8 * (l & 3), a.c);
    load8(row + kRope / 2, 1, 8 * (l & 3), a.s);
  }
}

__device__ __forceinline__ void rotate(int interleaved, int l, const Angles& a, float (&y)[8]) {
  if (interleaved) {
    if (l < kRope / 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = y[2 * i], v = y[2 * i + 1];
        y[2 * i] = u * a.c[i] - v * a.s[i];
        y[2 * i + 1] = v * a.c[i] + u * a.s[i];
      }
    }
  } else {
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = from_xor4(y[i]);     // every lane takes part
    if (l < kRope / 8) {
      const float sign = l < kRope / 16 ? -1.0f : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * a.c[i] + sign * o[i] * a.s[i];
    }
  }
}

// y[i] = sum_j (-1)^popcount(i & j) x[j] / sqrt(128): seven rounds of sums and
// differences, three within the lane and four between lanes, 56 additions a lane
// where the matrix takes 1024 products.
__device__ __forceinline__ void mix(int l, float (&y)[8]) {
#pragma unroll
  for (int bit = 1; bit < 8; bit <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & bit)) {
        const float u = y[i], v = y[i | bit];
        y[i] = u + v;
        y[i | bit] = u - v;
      }
  const float s1 = l & 1 ? -1.0f : 1.0f, s2 = l & 2 ? -1.0f : 1.0f, s4 = l & 4 ? -1.0f : 1.0f, s8 = l & 8 ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v = y[i];
    v = fmaf(v, s1, dpp<kXor1>(v));
    v = fmaf(v, s2, dpp<kXor2>(v));
    v = fmaf(v, s4, from_xor4(v));
    v = fmaf(v, s8, from_xor8(v));
    y[i] = v * 0.08838834764831845f;
  }
}

// The row's scale and this lane's eight codes.  The largest magnitude is an
// integer maximum of the bits without the sign: infinities and NaN come out on top,
// and such a row's scale is NaN.  A subnormal scale would have no finite inverse: rows
// below 448 * 2^-126 take the smallest normal one.
__device__ __forceinline__ float quantise(const float (&y)[8], uint2& codes) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_u32(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
  const float amax = __uint_as_float(row_max(top));
  const float scale = amax == 0.f                             ? 1.0f
                      : !(amax < INFINITY)                     ? __uint_as_float(0x7FC00000u)
                      : amax < 448.0f * 1.17549435e-38f ? 1.17549435e-38f
                                                               : amax / 448.0f;
  // The quotient by the reciprocal, corrected by its remainder (Markstein's
  // step), is rounded as a division's, unless the remainder leaves the normal numbers.
  float v[8];
  if (scale > 0x1p-60f) {
    const float inv = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = y[i] * inv;
      v[i] = fmaf(fmaf(-q, scale, y[i]), inv, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = y[i] / scale;
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  codes = make_uint2((uint32_t)lo, (uint32_t)hi);
  return scale;
}

__device__ __forceinline__ int64_t workgroup() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// ---- keys -------------------------------------------------------------------------------------

__global__ __launch_bounds__(kThreads) void key_store_kernel(StoreArgs a) {
  const int l = threadIdx.x & (kLanes - 1);
  const int64_t t = workgroup() * kRowsPerWg + threadIdx.x / kLanes;
  // lanes of a row leave together, so the others' DPP moves stay within whole rows
  if (t >= a.num_tokens) return;
  const int64_t slot = a.slot_map[t], pos = a.turn.cos_sin ? a.turn.positions[t] : 0;
  float y[8], w[8], bias[8];
  load8(a.k + t * a.k_stride, 0, 8 * l, y);
  if (a.norm_weight) {
    load8(a.norm_weight, a.norm_fp32, 8 * l, w);
    load8(a.norm_bias, a.norm_fp32, 8 * l, bias);
  }
  if (slot < 0 || slot >= a.num_slots) return;
  Angles angles;
  if (a.turn.cos_sin) {
    if (pos < 0 || pos >= a.turn.max_positions) return;
    load_angles(a.turn, pos, l, angles);
  }
  if (a.norm_weight) {
    // two passes over the registers: the variance of values far from 0 keeps its digits
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += y[i];
    const float mean = row_sum(sum) * (1.0f / kDim);
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] -= mean;
      sq = fmaf(y[i], y[i], sq);
    }
    const float inv = 1.0f / sqrtf(row_sum(sq) * (1.0f / kDim) + a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(y[i] * inv, w[i], bias[i]);
  }
  if (a.turn.cos_sin) rotate(a.turn.interleaved, l, angles, y);
  if (a.turn.hadamard) mix(l, y);
  uint2 codes;
  const float scale = quantise(y, codes);
  *reinterpret_cast<uint2*>(a.keys + slot * a.key_stride + 8 * l) = codes;
  if (l == 0) a.key_scale[slot] = scale;
}

// ---- queries ----------------------------------------------------------------------------------

__global__ __launch_bounds__(kThreads) void queries_kernel(QueryArgs a) {
  const int l = threadIdx.x & (kLanes - 1);
  const int64_t row = workgroup() * kRowsPerWg + threadIdx.x / kLanes, t = row / kHeads;
  const int h = (int)(row % kHeads);
  if (t >= a.num_tokens) return;
  const int64_t pos = a.turn.cos_sin ? a.turn.positions[t] : 0;
  float y[8];
  load8(a.q + t * a.q_token_stride + h * a.q_head_stride, 0, 8 * l, y);
  const float weight = a.weight_fp32 ? static_cast<const float*>(a.weights)[t * a.weight_stride + h]
                                     : (float)static_cast<const __bf16*>(a.weights)[t * a.weight_stride + h];
  Angles angles;
  if (a.turn.cos_sin) {
    if (pos < 0 || pos >= a.turn.max_positions) return;
    load_angles(a.turn, pos, l, angles);
    rotate(a.turn.interleaved, l, angles, y);
  }
  if (a.turn.hadamard) mix(l, y);
  uint2 codes;
  const float scale = quantise(y, codes);
  *reinterpret_cast<uint2*>(a.out_q + row * kDim + 8 * l) = codes;
  if (l == 0) a.out_weights[row] = weight * a.weight_scale * scale;
}

// ---- load -------------------------------------------------------------------------------------

// A wave copies kLoadRows consecutive rows, 8 lanes and 16 bytes a lane to each; lane
// i (mod kLoadRows) works out row i's slot.
constexpr int kLoadRows = 32;
constexpr int kLoadWgRows = kThreads / 64 * kLoadRows;

__global__ __launch_bounds__(kThreads) void key_load_kernel(KeyLoadArgs a) {
  const PagedKeys& c = a.cache;
  const int lane = threadIdx.x & 63;
  const int64_t first = workgroup() * kLoadWgRows + (threadIdx.x >> 6) * kLoadRows;
  const int64_t last = a.kv_starts[c.num_requests];
  const int64_t rows = last < a.num_rows ? last : a.num_rows;
  if (first >= rows) return;
  const int n = (int)(rows - first < kLoadRows ? rows - first : kLoadRows);
  const int mine = lane & (kLoadRows - 1);
  const int64_t row = first + (mine < n ? mine : n - 1);
  // the last request whose start is at or below the row
  int lo = 0, hi = c.num_requests;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if ((int64_t)a.kv_starts[mid] <= row) lo = mid; else hi = mid;
  }
  const int64_t pos = row - a.kv_starts[lo], col = pos >> c.log2_page;
  int64_t slot = -1;
  if (pos >= 0 && col < c.pages_per_row) {
    const int64_t page = c.page_table[lo * c.pages_per_row + col];
    if (page >= 0) slot = (page << c.log2_page) + (pos & (((int64_t)1 << c.log2_page) - 1));
  }
  if (slot >= c.num_slots) slot = -1;
  const float scale = slot >= 0 ? c.scale[slot] : 0.f;
  uint4 v[kLoadRows / 8];
#pragma unroll
  for (int i = 0; i < kLoadRows / 8; ++i) {
    const int s = __shfl((int)slot, i * 8 + (lane >> 3));
    v[i] = make_uint4(0, 0, 0, 0);
    if (s >= 0) v[i] = *reinterpret_cast<const uint4*>(c.keys + s * c.key_stride + (lane & 7) * 16);
  }
  if (lane < n) a.out_scale[first + lane] = scale;
#pragma unroll
  for (int i = 0; i < kLoadRows / 8; ++i) {
    const int r = i * 8 + (lane >> 3);
    if (r < n) *reinterpret_cast<uint4*>(a.out_keys + (first + r) * kDim + (lane & 7) * 16) = v[i];
  }
}

dim3 grid_of(int64_t items, int per) {
  const int64_t wgs = (items + per - 1) / per;
  return dim3((unsigned)(wgs < kMaxWgs ? wgs : kMaxWgs), (unsigned)((wgs + kMaxWgs - 1) / kMaxWgs));
}

}  // namespace

hipError_t launch_key_store(const StoreArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(key_store_kernel, grid_of(a.num_tokens, kRowsPerWg), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_queries(const QueryArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(queries_kernel, grid_of(a.num_tokens * kHeads, kRowsPerWg), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_key_load(const KeyLoadArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(key_load_kernel, grid_of(a.num_rows, kLoadWgRows), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace indexer
