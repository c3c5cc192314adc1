// The paged latent cache around the selection on gfx950: the plan of an append
// (pages and slots from request lengths), the store of new tokens (norm,
// rotation, 8-bit codes) and the load of rows as bf16.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "latent_device.h"
#include "latent_internal.h"

namespace latent {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// ---- plan of an append ------------------------------------------------------------------------

// q_start[b] = sum of new over requests before b, and page_start[b] the same
// of the pages each request needs beyond those it has.  One launch and no
// synchronisation among workgroups: every workgroup forms the sums over all
// requests itself (8 bytes a request, from cache), in tiles of kPlanTile, and
// then writes its own share of the tile's tokens and pages: blocks of
// kPlanThreads consecutive ones, dealt out round-robin, so one long prompt
// among single tokens still spreads over the device.  A token finds its
// request by a binary search of the tile's sums in LDS.
// Measured (MI355X): 64 requests of one token 4.7 us, 300 of 0 to 1024 tokens (150
// thousand of them) 9.0 us: the sums (loads of lengths, a scan) and one chain of
// table lookups, no bandwidth to speak of.  (Blocks dealt by a division for every
// block took 90 us for the latter.)
constexpr int kPlanThreads = 256;
constexpr int kPlanPer = 4;
constexpr int kPlanTile = kPlanThreads * kPlanPer;

struct PlanScan {
  int64_t tokens, pages;
};

__device__ __forceinline__ int32_t clamp_i32(int64_t v) { return v > (int64_t)INT32_MAX ? INT32_MAX : (int32_t)v; }

// The last of n ascending starts that is <= v (starts[0] <= v).
__device__ __forceinline__ int find_start(const int64_t* starts, int n, int64_t v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs a) {
  __shared__ int64_t q_start[kPlanTile + 1];
  __shared__ int64_t p_start[kPlanTile + 1];
  __shared__ int32_t kv_len[kPlanTile];
  __shared__ int32_t had[kPlanTile];
  __shared__ PlanScan wave_sum[kPlanThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t wg = blockIdx.x, nwg = gridDim.x;
  // this workgroup's first block (of kPlanThreads, dealt round-robin) that reaches item v or lies behind it
  auto first_block = [&](int64_t v) {
    const int64_t blk = v / kPlanThreads;
    return blk + (uint32_t)(wg + nwg - (uint32_t)blk % (uint32_t)nwg) % (uint32_t)nwg;
  };
  const int64_t page_mask = ((int64_t)1 << a.log2_page) - 1;
  const int64_t used = a.free_used ? a.free_used[0] : 0;
  int64_t tokens = 0, pages = 0;   // sums over the tiles before this one
  for (int64_t base = 0; base < a.num_requests; base += kPlanTile) {
    const int n = (int)(a.num_requests - base < kPlanTile ? a.num_requests - base : kPlanTile);
    int64_t kv[kPlanPer], nw[kPlanPer], pg[kPlanPer];
    PlanScan own{0, 0};
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int r = tid * kPlanPer + i;
      kv[i] = r < n ? a.kv_lens[base + r] : 0;
      nw[i] = r < n ? a.new_lens[base + r] : 0;
      kv[i] = kv[i] < 0 ? 0 : kv[i];
      nw[i] = nw[i] < 0 ? 0 : nw[i];
      int64_t have = (kv[i] + page_mask) >> a.log2_page, need = (kv[i] + nw[i] + page_mask) >> a.log2_page;
      have = have < a.pages_per_row ? have : a.pages_per_row;
      need = need < a.pages_per_row ? need : a.pages_per_row;
      pg[i] = need - have;
      if (r < n) {
        kv_len[r] = (int32_t)kv[i];
        had[r] = (int32_t)have;
      }
      own.tokens += nw[i];
      own.pages += pg[i];
    }
    PlanScan incl = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t t = __shfl_up(incl.tokens, d), p = __shfl_up(incl.pages, d);
      if (lane >= d) {
        incl.tokens += t;
        incl.pages += p;
      }
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int64_t qs = tokens + incl.tokens - own.tokens, ps = pages + incl.pages - own.pages;
    int64_t tile_tokens = 0, tile_pages = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) {
      if (w < wave) {
        qs += wave_sum[w].tokens;
        ps += wave_sum[w].pages;
      }
      tile_tokens += wave_sum[w].tokens;
      tile_pages += wave_sum[w].pages;
    }
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int r = tid * kPlanPer + i;
      q_start[r] = qs;
      p_start[r] = ps;
      if (r < n && wg == 0) {
        a.seq_lens[base + r] = clamp_i32(kv[i] + nw[i]);
        a.q_starts[base + r] = clamp_i32(qs);
      }
      qs += nw[i];
      ps += pg[i];
    }
    __syncthreads();
    // fresh pages of the tile's requests
    for (int64_t blk = first_block(pages); blk * kPlanThreads < pages + tile_pages; blk += nwg) {
      const int64_t p = blk * kPlanThreads + tid;
      if (p < pages || p >= pages + tile_pages) continue;
      const int r = find_start(p_start, n, p);
      const int64_t at = used + p;
      a.page_table[(base + r) * a.pages_per_row + had[r] + (p - p_start[r])] =
          at >= 0 && at < a.num_free ? a.free_pages[at] : -1;
    }
    // the tile's tokens
    const int64_t end = tokens + tile_tokens < a.num_tokens ? tokens + tile_tokens : a.num_tokens;
    for (int64_t blk = first_block(tokens); blk * kPlanThreads < end; blk += nwg) {
      const int64_t t = blk * kPlanThreads + tid;
      if (t < tokens || t >= end) continue;
      const int r = find_start(q_start, n, t);
      const int64_t pos = kv_len[r] + (t - q_start[r]);
      const int64_t col = pos >> a.log2_page;
      int64_t page = -1;
      if (col < had[r]) {
        page = a.page_table[(base + r) * a.pages_per_row + col];
      } else if (col < a.pages_per_row) {
        const int64_t at = used + p_start[r] + (col - had[r]);
        if (at >= 0 && at < a.num_free) page = a.free_pages[at];
      }
      const int64_t slot = (page << a.log2_page) + (pos & page_mask);
      a.slot_map[t] = page < 0 || slot > (int64_t)INT32_MAX ? -1 : (int32_t)slot;
      a.positions[t] = clamp_i32(pos);
    }
    tokens += tile_tokens;
    pages += tile_pages;
    __syncthreads();
  }
  // padding, and the totals
  for (int64_t blk = first_block(tokens); blk * kPlanThreads < a.num_tokens; blk += nwg) {
    const int64_t t = blk * kPlanThreads + tid;
    if (t < tokens || t >= a.num_tokens) continue;
    a.slot_map[t] = -1;
    a.positions[t] = -1;
  }
  if (wg == 0 && tid == 0) {
    a.q_starts[a.num_requests] = clamp_i32(tokens);
    a.free_used_out[0] = clamp_i32(used + pages);
  }
}

// ---- store ------------------------------------------------------------------------------------

// One wave per token: lane l holds latents 8l .. 8l + 7 (one 16-byte load) and
// one rotary element; the norm's sum of squares and the codes' largest
// magnitude are wave reductions, the rotation's partner element comes from
// another lane.  Nothing passes through LDS.
// Measured (MI355X): 16000 tokens into 8-bit slots 10.2 us, 29 MB read and stored (6
// us at a large copy's rate), into bf16 ones 9.5, 37 MB (7.5): vector instructions,
// about 200 a token in 8 bits, and the two loads in turn.  (Reductions by lane permutes through LDS and eight divisions took
// 12.7 us.)  64 tokens 3.0 us: a launch and two loads in turn (position, then angles).
constexpr int kStoreThreads = 256;

// Reductions over the wave in registers: within 16 lanes by DPP (pairs, quads,
// halves, rows), then over the four groups of 16.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, true);
}

__device__ __forceinline__ float wave_sum_f32(float v) {
  v += __uint_as_float(dpp<0xB1>(__float_as_uint(v)));     // quad_perm 1 0 3 2
  v += __uint_as_float(dpp<0x4E>(__float_as_uint(v)));     // quad_perm 2 3 0 1
  v += __uint_as_float(dpp<0x141>(__float_as_uint(v)));    // row_half_mirror
  v += __uint_as_float(dpp<0x140>(__float_as_uint(v)));    // row_mirror
  return sum_of_4(v);
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max_u32(v, dpp<0xB1>(v));
  v = max_u32(v, dpp<0x4E>(v));
  v = max_u32(v, dpp<0x141>(v));
  v = max_u32(v, dpp<0x140>(v));
  auto sw = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max_u32(sw[0], sw[1]);
  sw = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max_u32(sw[0], sw[1]);
}

template <bool E4M3>
__global__ __launch_bounds__(kStoreThreads) void store_kernel(StoreArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kStoreThreads / 64) + (threadIdx.x >> 6);
  if (t >= a.num_tokens) return;
  // all that depends on nothing is loaded first; only the angles wait for a load
  const int64_t slot = a.slot_map[t], pos = a.cos_sin ? a.positions[t] : 0;
  const uint16_t* row = a.kv + t * a.kv_stride;
  const bf16x8 c = *reinterpret_cast<const bf16x8*>(row + lane * 8);
  float r = (float)reinterpret_cast<const __bf16*>(row + kLatent)[lane];
  bf16x8 w;
  if (a.norm_weight) w = *reinterpret_cast<const bf16x8*>(a.norm_weight + lane * 8);
  if (slot < 0 || slot >= a.num_slots) return;
  // angle and partner of this lane's rotary element
  const int angle = a.interleaved ? lane >> 1 : lane & 31;
  const bool second = a.interleaved ? (lane & 1) != 0 : lane >= 32;
  if (a.cos_sin) {
    if (pos < 0 || pos >= a.max_positions) return;
    const float cs = a.cos_sin[pos * kRope + angle], sn = a.cos_sin[pos * kRope + kRope / 2 + angle];
    const float o = __shfl_xor(r, a.interleaved ? 1 : 32);
    r = second ? r * cs + o * sn : r * cs - o * sn;
  }
  reinterpret_cast<__bf16*>(a.rope + slot * a.rope_stride)[lane] = (__bf16)r;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = (float)c[i];
  if (a.norm_weight) {
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(y[i], y[i], sq);
    const float inv = 1.0f / sqrtf(wave_sum_f32(sq) * (1.0f / kLatent) + a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * inv * (float)w[i];
  }
  char* dst = a.latent + slot * a.latent_stride;
  if (!E4M3) {
    bf16x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (__bf16)y[i];
    *reinterpret_cast<bf16x8*>(dst + lane * 16) = o;
    return;
  }
  // Largest magnitude as an integer maximum of the bits without the sign:
  // infinities and NaN come out on top, and a row that has one gets a NaN for
  // its scale and so reads back as NaN.
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(y[i]) & 0x7FFFFFFFu;
    top = top > b ? top : b;
  }
  const float amax = __uint_as_float(wave_max_u32(top));
  // A subnormal scale would have no finite inverse: such rows (all below
  // 448 * 2^-126) take the smallest normal scale.
  const float scale = amax == 0.f                              ? 1.0f
                      : !(amax < INFINITY)                      ? __uint_as_float(0x7FC00000u)
                      : amax < 448.0f * 1.17549435e-38f ? 1.17549435e-38f
                                                                : amax / 448.0f;
  if (lane == 0) a.scale[slot] = scale;
  // y / scale, at most 448 and a rounding, which E4M3 rounds back to 448.  The
  // quotient by the reciprocal is corrected by its remainder (Markstein's step), which
  // rounds it as a division does, unless the remainder leaves the normal numbers (or
  // scale is NaN).
  if (scale > 0x1p-60f) {
    const float inv = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = y[i] * inv;
      y[i] = fmaf(fmaf(-q, scale, y[i]), inv, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] / scale;
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
  *reinterpret_cast<int2*>(dst + lane * 8) = make_int2(lo, hi);
}

// ---- load -------------------------------------------------------------------------------------

// A wave copies kLoadRows consecutive rows: lane l holds latents 8l .. 8l + 7
// of each (all rows' loads are issued before the first store), and 16 bytes of
// rotary key of one row.  By page table, the wave finds the request of its
// rows by counting the starts at or below each row, 64 at a time.
// Measured (MI355X): 400 thousand rows of 16 requests out of 8-bit pages 134-139 us,
// 5.2-5.4 TB/s read and written (a copy of 2 GiB: 4.9); 1000 bf16 slots 3.2 us.
constexpr int kLoadThreads = 256;
constexpr int kLoadRows = 8;

template <bool E4M3, bool PAGED>
__global__ __launch_bounds__(kLoadThreads) void load_kernel(LoadArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t first = ((int64_t)blockIdx.x * (kLoadThreads / 64) + (threadIdx.x >> 6)) * kLoadRows;
  int64_t rows = a.num_rows;
  if (PAGED) {
    const int64_t last = a.kv_starts[a.num_requests];
    rows = last < rows ? last : rows;
  }
  if (first >= rows) return;
  const int n = (int)(rows - first < kLoadRows ? rows - first : kLoadRows);
  // lane i (mod kLoadRows) works out row first + i's slot
  const int mine = lane & (kLoadRows - 1);
  const int64_t row = first + (mine < n ? mine : n - 1);
  int64_t slot = -1;
  if (PAGED) {
    // requests whose start is at or below each row: a few rows span few
    // requests, so after the first row's count the walk is short
    int64_t b = 0;
    for (int64_t base = 1; base <= a.num_requests; base += 64) {
      const int64_t at = base + lane;
      const bool below = at <= a.num_requests && (int64_t)a.kv_starts[at] <= first;
      const int c = __popcll(__ballot(below));
      b += c;
      if (c < 64) break;
    }
    while (b + 1 < a.num_requests && (int64_t)a.kv_starts[b + 1] <= row) ++b;
    const int64_t pos = row - a.kv_starts[b], col = pos >> a.log2_page;
    if (b < a.num_requests && pos >= 0 && col < a.pages_per_row) {
      const int64_t page = a.page_table[b * a.pages_per_row + col];
      if (page >= 0) slot = (page << a.log2_page) + (pos & (((int64_t)1 << a.log2_page) - 1));
    }
  } else {
    slot = a.slots[row];
  }
  if (slot >= a.cache.num_slots) slot = -1;
  const float scale = E4M3 && slot >= 0 ? a.cache.scale[slot] : 1.0f;
  uint4 raw[kLoadRows];
#pragma unroll
  for (int i = 0; i < kLoadRows; ++i) {
    const int64_t s = ((int64_t)__builtin_amdgcn_readlane((int)slot, i));
    raw[i] = make_uint4(0, 0, 0, 0);
    if (s >= 0) {
      const char* src = a.cache.latent + s * a.cache.latent_stride;
      if (E4M3) {
        const uint2 v = *reinterpret_cast<const uint2*>(src + lane * 8);
        raw[i].x = v.x;
        raw[i].y = v.y;
      } else {
        raw[i] = *reinterpret_cast<const uint4*>(src + lane * 16);
      }
    }
  }
  // rotary keys: 8 lanes a row, 16 bytes each
  const int rr = lane >> 3;
  const int rslot = __shfl((int)slot, rr);
  uint4 rope = make_uint4(0, 0, 0, 0);
  if (rslot >= 0) rope = *reinterpret_cast<const uint4*>(a.cache.rope + rslot * a.cache.rope_stride + (lane & 7) * 16);
#pragma unroll
  for (int i = 0; i < kLoadRows; ++i) {
    if (i >= n) break;
    uint4 o = raw[i];
    if (E4M3) {
      const float s = __shfl(scale, i);
      bf16x8 v;
      f32x2 p;
      p = __builtin_amdgcn_cvt_pk_f32_fp8(raw[i].x, false); v[0] = (__bf16)(p[0] * s); v[1] = (__bf16)(p[1] * s);
      p = __builtin_amdgcn_cvt_pk_f32_fp8(raw[i].x, true);  v[2] = (__bf16)(p[0] * s); v[3] = (__bf16)(p[1] * s);
      p = __builtin_amdgcn_cvt_pk_f32_fp8(raw[i].y, false); v[4] = (__bf16)(p[0] * s); v[5] = (__bf16)(p[1] * s);
      p = __builtin_amdgcn_cvt_pk_f32_fp8(raw[i].y, true);  v[6] = (__bf16)(p[0] * s); v[7] = (__bf16)(p[1] * s);
      o = __builtin_bit_cast(uint4, v);
    }
    *reinterpret_cast<uint4*>(a.out_latent + (first + i) * kLatent + lane * 8) = o;
  }
  if (rr < n) *reinterpret_cast<uint4*>(a.out_rope + (first + rr) * kRope + (lane & 7) * 8) = rope;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

hipError_t launch_append_plan(const PlanArgs& a, hipStream_t stream) {
  // a workgroup per 1024 tokens: each spends its time on the sums and two
  // dependent loads, so more of them only repeat the sums
  int64_t wgs = ceil_div(a.num_tokens, 1024);
  wgs = wgs < 1 ? 1 : (wgs > 256 ? 256 : wgs);
  hipLaunchKernelGGL(plan_kernel, dim3((unsigned)wgs), dim3(kPlanThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_cache_store(const StoreArgs& a, bool e4m3, hipStream_t stream) {
  const int64_t wgs = ceil_div(a.num_tokens, kStoreThreads / 64), most = kMaxThreads / kStoreThreads;
  const dim3 grid((unsigned)(wgs < most ? wgs : most), (unsigned)ceil_div(wgs, most));
  if (e4m3)
    hipLaunchKernelGGL(store_kernel<true>, grid, dim3(kStoreThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(store_kernel<false>, grid, dim3(kStoreThreads), 0, stream, a);
  return hipGetLastError();
}

int64_t load_threads(int64_t num_rows) { return ceil_div(num_rows, (kLoadThreads / 64) * kLoadRows) * kLoadThreads; }

hipError_t launch_cache_load(const LoadArgs& a, bool e4m3, hipStream_t stream) {
  const dim3 grid((unsigned)(load_threads(a.num_rows) / kLoadThreads)), block(kLoadThreads);
  if (a.slots) {
    if (e4m3)
      hipLaunchKernelGGL((load_kernel<true, false>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((load_kernel<false, false>), grid, block, 0, stream, a);
  } else {
    if (e4m3)
      hipLaunchKernelGGL((load_kernel<true, true>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((load_kernel<false, true>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace latent
