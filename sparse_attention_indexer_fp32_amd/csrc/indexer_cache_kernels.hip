// The indexer's keys and queries in 8 bits on gfx950: the append of keys to
// their paged cache, the queries in the same form, and cached keys laid in a row.
//
// Each value is read and each code written once, and memory bounds all three (MI355X, host included):
// the queries of 8192 tokens 22.5-25 us, 4.2-4.7 TB/s read and written, where a large copy reaches 5.1; the load
// of 400000 rows 20.5 us, 5.1 TB/s; the store of 16000 keys 8.3 us and every smaller call as much,
// which is the host's part of a launch.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "indexer_paged_internal.h"

namespace indexer {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kHeads = 32;
constexpr int kDim = 128;
constexpr int kRope = 64;
constexpr int kLanes = 4;                 // lanes of a row
constexpr int kChunks = 4;                // chunks of 8 values that a lane holds of it
constexpr int kThreads = 256;
constexpr int kRowsPerWg = kThreads / kLanes;
constexpr int64_t kMaxWgs = UINT32_MAX / kThreads;   // along x: the hardware counts threads in 32 bits

// ---- a row over four lanes --------------------------------------------------------------------

// A row of 128 values lies in the four lanes of a quad: lane l holds the chunks of 8
// values l, 4 + l, 8 + l and 12 + l (16-byte loads, 64 bytes of a row to an instruction), so value 8
// c + e sits in lane c % 4.  Of the mixing's seven rounds five and both kinds of
// rotation (neighbours, and values 32 apart) then stay within the lane, all lanes
// turn as many values as the others, and what is left are exchanges within a quad, DPP moves.
// (16 lanes of 8 values each, where four rounds cross lanes and half of the lanes
// have nothing to turn: 8192 tokens x 32 heads 53 us against 22.)
struct Row {
  float v[kChunks * 8];      // chunk after chunk
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;      // quad_perm

__device__ __forceinline__ float quad_sum(float v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  return v;
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Eight values of a vector of either type.
__device__ __forceinline__ void load8(const void* from, int fp32, int at, float* v) {
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

__device__ __forceinline__ void load_row(const uint16_t* from, int l, Row& r) {
#pragma unroll
  for (int c = 0; c < kChunks; ++c) load8(from, 0, 32 * c + 8 * l, r.v + 8 * c);
}

// The angles of a lane's values.  Interleaved: those of the four pairs of
// chunk l, then of chunk 4 + l.  By halves chunk l turns with chunk 4 + l, by its 8 angles.
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const TurnArgs& t, int64_t pos, int l, Angles& a) {
  const float* row = t.cos_sin + pos * kRope;
  const int second = t.interleaved ? 16 + 4 * l : 8 * l + 4, first = t.interleaved ? 4 * l : 8 * l;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float4 c = *reinterpret_cast<const float4*>(row + (half ? second : first));
    const float4 s = *reinterpret_cast<const float4*>(row + kRope / 2 + (half ? second : first));
    a.c[4 * half] = c.x; a.c[4 * half + 1] = c.y; a.c[4 * half + 2] = c.z; a.c[4 * half + 3] = c.w;
    a.s[4 * half] = s.x; a.s[4 * half + 1] = s.y; a.s[4 * half + 2] = s.z; a.s[4 * half + 3] = s.w;
  }
}

__device__ __forceinline__ void turn(float& u, float& v, float c, float s) {
  const float a = u * c - v * s;
  v = v * c + u * s;
  u = a;
}

__device__ __forceinline__ void rotate(int interleaved, const Angles& a, Row& r) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(r.v[2 * i], r.v[2 * i + 1], a.c[i], a.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(r.v[i], r.v[8 + i], a.c[i], a.s[i]);
  }
}

// y[i] = sum_j (-1)^popcount(i & j) x[j]: seven rounds of sums and differences, 288
// instructions a lane where the matrix takes 4096 products.  (The factor 1 / sqrt(128) is left to the scale.)
__device__ __forceinline__ void mix(int l, Row& r) {
  float (&v)[8 * kChunks] = r.v;
#pragma unroll
  for (int bit = 1; bit < 8 * kChunks; bit <<= 1)
#pragma unroll
    for (int i = 0; i < 8 * kChunks; ++i)
      if (!(i & bit)) {
        const float a = v[i], b = v[i | bit];
        v[i] = a + b;
        v[i | bit] = a - b;
      }
  const float s1 = l & 1 ? -1.0f : 1.0f, s2 = l & 2 ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < 8 * kChunks; ++i) {
    v[i] = fmaf(v[i], s1, dpp<kXor1>(v[i]));
    v[i] = fmaf(v[i], s2, dpp<kXor2>(v[i]));
  }
}

// The scale of a row that is still to be multiplied by `factor`, and this lane's codes.  The largest
// magnitude is an integer maximum of the bits without the sign: infinities and
// NaN come out on top, and such a row's scale is NaN.  A step that is
// subnormal would have no finite reciprocal, and a scale that is loses digits: a row's scale is 2^-126 at least.
// The quotient by the reciprocal is corrected by its remainder (Markstein's step), which rounds it as a division
// does, unless the remainder leaves the normal numbers (or the step is NaN).  (Without the correction the queries of
// 8192 tokens took 22.1 us against 23.5, and values next to a tie of the codes fell either way.)  r is left as quotients.
__device__ __forceinline__ float quantise(Row& r, float factor, uint2 (&codes)[kChunks]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8 * kChunks; ++i) top = max_u32(top, __float_as_uint(r.v[i]) & 0x7FFFFFFFu);
  top = max_u32(top, dpp<kXor1>(top));
  top = max_u32(top, dpp<kXor2>(top));
  const float amax = __uint_as_float(top);
  const float least = 0x1p-126f / factor;
  const float step = amax == 0.f                  ? 1.0f
                     : !(amax < INFINITY)         ? __uint_as_float(0x7FC00000u)
                     : amax < 448.0f * least ? least
                                                  : amax / 448.0f;
  if (step > 0x1p-60f) {
    const float inv = 1.0f / step;
#pragma unroll
    for (int i = 0; i < 8 * kChunks; ++i) {
      const float q = r.v[i] * inv;
      r.v[i] = fmaf(fmaf(-q, step, r.v[i]), inv, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8 * kChunks; ++i) r.v[i] = r.v[i] / step;
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const float* v = r.v + 8 * c;
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    codes[c] = make_uint2((uint32_t)lo, (uint32_t)hi);
  }
  return amax == 0.f ? 1.0f : step * factor;
}

__device__ __forceinline__ void store_codes(uint8_t* to, int l, const uint2 (&codes)[kChunks]) {
#pragma unroll
  for (int c = 0; c < kChunks; ++c) *reinterpret_cast<uint2*>(to + 32 * c + 8 * l) = codes[c];
}

constexpr float kMixFactor = 0.08838834764831845f;   // 1 / sqrt(128)

__device__ __forceinline__ int64_t workgroup() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// ---- keys -------------------------------------------------------------------------------------

// Takes a row's mean from its values, and returns its variance.  Two passes over the registers: the variance of values
// far from 0 keeps its digits.
__device__ __forceinline__ float centre(Row& y) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8 * kChunks; ++i) sum += y.v[i];
  const float mean = quad_sum(sum) * (1.0f / kDim);
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < 8 * kChunks; ++i) {
    y.v[i] -= mean;
    sq = fmaf(y.v[i], y.v[i], sq);
  }
  return quad_sum(sq) * (1.0f / kDim);
}

__global__ __launch_bounds__(kThreads) void key_store_kernel(StoreArgs a) {
  const int l = threadIdx.x & (kLanes - 1);
  const int64_t t = workgroup() * kRowsPerWg + threadIdx.x / kLanes;
  // (lanes of a row leave together, so the others' DPP moves stay within whole rows)
  if (t >= a.num_tokens) return;
  // all that depends on nothing is loaded first; only the angles wait for a load
  const int64_t slot = a.slot_map[t], pos = a.turn.cos_sin ? a.turn.positions[t] : 0;
  Row y, w, bias;
  load_row(a.k + t * a.k_stride, l, y);
  if (a.norm_weight) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      load8(a.norm_weight, a.norm_fp32, 32 * c + 8 * l, w.v + 8 * c);
      load8(a.norm_bias, a.norm_fp32, 32 * c + 8 * l, bias.v + 8 * c);
    }
  }
  if (slot < 0 || slot >= a.num_slots) return;
  Angles angles;
  if (a.turn.cos_sin) {
    if (pos < 0 || pos >= a.turn.max_positions) return;
    load_angles(a.turn, pos, l, angles);
  }
  if (a.norm_weight) {
    float var = centre(y);
    float eps = a.eps;
    if (!(var < INFINITY)) {
      // values beyond 2^60, whose squares leave fp32: the same of the row divided by 2^70 (the lanes of a
      // row together; one that is not finite comes out as NaN)
      load_row(a.k + t * a.k_stride, l, y);
#pragma unroll
      for (int i = 0; i < 8 * kChunks; ++i) y.v[i] *= 0x1p-70f;
      var = centre(y);
      eps *= 0x1p-140f;
    }
    const float inv = 1.0f / sqrtf(var + eps);
#pragma unroll
    for (int i = 0; i < 8 * kChunks; ++i) y.v[i] = fmaf(y.v[i] * inv, w.v[i], bias.v[i]);
  }
  if (a.turn.cos_sin) rotate(a.turn.interleaved, angles, y);
  if (a.turn.hadamard) mix(l, y);
  uint2 codes[kChunks];
  const float scale = quantise(y, a.turn.hadamard ? kMixFactor : 1.0f, codes);
  store_codes(a.keys + slot * a.key_stride, l, codes);
  if (l == 0) a.key_scale[slot] = scale;
}

// ---- queries ----------------------------------------------------------------------------------

__global__ __launch_bounds__(kThreads) void queries_kernel(QueryArgs a) {
  const int l = threadIdx.x & (kLanes - 1);
  const int64_t row = workgroup() * kRowsPerWg + threadIdx.x / kLanes, t = row / kHeads;
  const int h = (int)(row % kHeads);
  if (t >= a.num_tokens) return;
  const int64_t pos = a.turn.cos_sin ? a.turn.positions[t] : 0;
  Row y;
  load_row(a.q + t * a.q_token_stride + h * a.q_head_stride, l, y);
  const float weight = a.weight_fp32 ? static_cast<const float*>(a.weights)[t * a.weight_stride + h]
                                     : (float)static_cast<const __bf16*>(a.weights)[t * a.weight_stride + h];
  if (a.turn.cos_sin) {
    if (pos < 0 || pos >= a.turn.max_positions) return;
    Angles angles;
    load_angles(a.turn, pos, l, angles);
    rotate(a.turn.interleaved, angles, y);
  }
  if (a.turn.hadamard) mix(l, y);
  uint2 codes[kChunks];
  const float scale = quantise(y, a.turn.hadamard ? kMixFactor : 1.0f, codes);
  store_codes(a.out_q + row * kDim, l, codes);
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
