// Latent attention, absorbed form, over whole cached sequences that share
// prefixes, on gfx950: a group's shared positions are read once for all of its tokens.
//
// For a token of request b in group g, positions below shared_lens[g] come from
// the page table row of the group's first request, the others from b's own:
//   z[h, j] = scale * (s_j q_c[h] . c_j + q_r[h] . r_j)
//   out[h]  = sum_j softmax_j(z[h]) s_j c_j,
// and as every head of every token reads the same rows, (token, head) pairs are
// rows of one matrix: 64 neighbouring ones make a unit, whatever tokens and heads they
// are.  A unit of a group goes over the shared prefix, one of a request over the request's own keys
// (with several new tokens, each of its rows up to its own limit).  Softmax
// parts over disjoint keys add up, so a row's result is the sum of its parts of
// both units, and of as many more as the units were cut in.
//
// The tiling within a workgroup is the absorbed kernel's (attend_kernels.hip): waves of 16 rows, tiles
// of 32 keys staged once for four waves, and two workgroups on a CU, that drift apart, so that one
// multiplies while the other waits.  (One workgroup of two rings, in step at every tile's barrier,
// halves the parts: 64 requests x 32 heads behind 32768 positions 225 us against 213, 8 x 16 behind
// 4096 35 and 29.  A workgroup of eight waves that deals the scores out by keys and the values by
// latents, so that each byte of LDS is read half as often, needs two barriers a tile and the weights
// through LDS: 269.  Waves of 32 rows, one to a SIMD, with the softmax step laid between matrix
// instructions: 245.)
//
// Measured (MI355X): 64 requests x 32 heads behind 32768 positions 203 us + 15 of the join, up to 725
// TFLOP/s: matrix instructions, vector instructions and LDS are busy for 43 to 48 % of the time each,
// and 15 % is waiting for rows (with one row for all, from L1: 181).  8 x 16 behind 4096 20 + 5 us.
// 150 x 2 tokens x 20 heads over codes 225-237 us: vector instructions, 70 %.  (All 256 vector registers are in use; 12 of
// bf16 and 18 over codes are spilled around the parts, none is reloaded in the loop over the tiles.)

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attend_device.h"
#include "latent_device.h"
#include "latent_internal.h"
#include "share_plan.h"

namespace latent {
namespace {

constexpr int kThreads = 64 * kUnitWaves;

// What a unit costs beside its tiles, in tiles: its rows, starts and first keys are waited for, its
// part is written and read again.  (Counted by their tiles alone, the units of 64 requests with a
// single key each beside a prefix of 32768 all fell to one workgroup: 652 us, and 200 so; 150 x 2
// tokens of five groups 294 and 234.)
constexpr uint32_t kUnitCost = 4;

// The arguments, loaded anew: what is read through this does not stay in scalar registers, of which
// the loop over the tiles has few to spare, from one use to the next.
__device__ __forceinline__ SharedArgs args_here() {
#if defined(__HIP_DEVICE_COMPILE__)       // (the pass over the host's code knows no such pointers)
  typedef const __attribute__((address_space(4))) SharedArgs* args_ptr;
  args_ptr p = (args_ptr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *p;
#else
  return SharedArgs{};
#endif
}

// A group, or a request: the rows of its units and the keys they go over.
struct Entity {
  int32_t row0;          // first of its rows (token * heads + head, from the launch's first token on)
  int32_t rows;          // and how many this launch takes
  int32_t key0, keys;    // positions [key0, key0 + keys)
  int32_t list;          // row of the page table
  int32_t request;       // the request, or -1: a group
  int32_t before;        // its tokens before the first one, of this launch
};

__device__ __forceinline__ int64_t clamp_to(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : (v < hi ? v : hi); }

// A length, cut to what a row of the page table holds.
__device__ __forceinline__ int cached(const SharedArgs& a, int n) {
  return (int)clamp_to(n, 0, a.pages_per_row << a.log2_page);
}

// The group that request b is in, or -1.
__device__ __forceinline__ int group_of(const SharedArgs& a, int b) {
  if (a.num_groups == 0 || b < a.group_starts[0] || b >= a.group_starts[a.num_groups]) return -1;
  int lo = 0, hi = a.num_groups;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (a.group_starts[mid] <= b) lo = mid; else hi = mid;
  }
  return lo;
}

// Entity e: the groups, then the requests.
__device__ __forceinline__ Entity entity(const SharedArgs& a, int e) {
  Entity u;
  int b0, b1;
  if (e < a.num_groups) {
    b0 = (int)clamp_to(a.group_starts[e], 0, a.num_requests);
    b1 = (int)clamp_to(a.group_starts[e + 1], b0, a.num_requests);
    u.request = -1;
    u.key0 = 0;
    u.keys = cached(a, a.shared_lens[e]);
  } else {
    b0 = e - a.num_groups;
    b1 = b0 + 1;
    u.request = b0;
    const int g = group_of(a, b0);
    u.key0 = g < 0 ? 0 : cached(a, a.shared_lens[g]);
    u.keys = cached(a, a.seq_lens[b0]) - u.key0;
    u.keys = u.keys < 0 ? 0 : u.keys;
  }
  u.list = b0;
  const int64_t end = (int64_t)a.first_token + a.num_tokens;
  const int64_t t0 = clamp_to(a.q_starts[b0], a.first_token, end), t1 = clamp_to(a.q_starts[b1], t0, end);
  u.before = (int)(t0 - a.first_token);
  u.row0 = u.before * a.num_heads;
  u.rows = (int)(t1 - t0) * a.num_heads;
  return u;
}

__device__ __forceinline__ uint32_t cost_of(const Entity& u) {
  const uint32_t n = ((uint32_t)u.keys + kTileKeys - 1) / kTileKeys;
  return u.request >= 0 || n > 0 ? n + kUnitCost : 0;      // a request's rows are somebody's, with or without keys
}
__device__ __forceinline__ uint32_t blocks_of(const Entity& u) { return (uint32_t)((u.rows + kUnitRows - 1) / kUnitRows); }

// The first of an entity's pieces of 16 rows: pieces of different entities of one kind do
// not meet, as each has a token at least.
__device__ __forceinline__ int first_piece(const SharedArgs& a, const Entity& u) {
  return (u.request >= 0 ? a.pieces : 0) + u.row0 / 16 + u.before;
}

// The tile's keys that a limit leaves, as bits; `from`: the tile's first position.
__device__ __forceinline__ uint32_t below(int limit, int from) {
  const int n = limit - from;
  return n >= kTileKeys ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1;
}

// A tile whose keys count for some of the unit's rows only: a row that leaves a key out has a weight of 0
// for it, but 0 times an infinity is not 0, so rows of the cache that hold an infinity or a NaN are
// cleared.  What a row that does attend such a key has from it is kept: its score is never finite itself (a
// product with an infinity or a NaN in it is not).  Is it NaN or +inf, so is the row's sum, and with it all of the
// row's result.  Is it -inf, the key's weight is 0, and its row takes part as 0 times its values: where they
// are not finite that is NaN, added here, and nothing elsewhere, as in tiles that all rows attend whole.
// (Codes stand for no infinities, and a NaN among them gives a score of NaN.)

// Rows of the stage that hold one, eight rows a wave, as bits from this wave's first row on.
template <bool E4M3>
__device__ __forceinline__ uint32_t rows_not_finite(uint32_t stage, int wave) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const int lane = lane_here();
  constexpr int kBytes = E4M3 ? kLatent : kRowBytes;
  uint32_t rows = 0;
  for (int i = 0; i < kTileKeys / kUnitWaves; ++i) {
    bool bad = false;
    if (lane * 16 < kBytes) {
      const u32x4 w = read_lds<u32x4>(stage + (wave * (kTileKeys / kUnitWaves) + i) * kBytes + lane * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (E4M3) {
          // a code of all ones but the sign
          const uint32_t ones = w[j] & 0x7F7F7F7Fu;
          bad |= ((ones + 0x01010101u) & 0x80808080u) != 0;
        } else {
          bad |= (w[j] & 0x7F80u) == 0x7F80u || (w[j] & 0x7F800000u) == 0x7F800000u;
        }
      }
    }
    rows |= (uint32_t)__any(bad) << i;
  }
  return rows;
}

// 0 times the values of the stage's rows `rows` (bf16), added to the accumulators of the lanes whose
// row attends them.
__device__ __forceinline__ void add_nothing(HeadState& st, uint32_t stage, uint32_t rows, uint32_t mask) {
  const int lane = lane_here(), g = lane >> 4;
  for (; rows; rows &= rows - 1) {
    const int key = __builtin_ctz(rows);
    const uint32_t attends = (mask >> key & 1) ? 0xFFFFFFFFu : 0u;
    const uint32_t at = stage + key * kRowBytes + (((g >> 1) ^ swizzle(key)) << 4) + (g & 1) * 8;
#pragma unroll
    for (int cb = 0; cb < kColBlocks; ++cb) {
      const u32x2 v = read_lds<u32x2>((at ^ (uint32_t)((cb & 7) << 5)) + (cb >> 3) * 256);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t bits = (r & 1 ? v[r >> 1] & 0xFFFF0000u : v[r >> 1] << 16) & attends;
        st.o[cb][r] = fmaf(__uint_as_float(bits), 0.f, st.o[cb][r]);
      }
      __builtin_amdgcn_sched_barrier(0);     // reads ahead would take registers that the loop has not
    }
  }
}

// Clears this wave's rows among `rows`.
template <bool E4M3>
__device__ __forceinline__ void clear_rows(uint32_t stage, int wave, uint32_t rows) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) u32x4* lds_ptr;
  const int lane = lane_here();
  constexpr int kBytes = E4M3 ? kLatent : kRowBytes;
  for (uint32_t own = rows >> (wave * (kTileKeys / kUnitWaves)) & ((1u << (kTileKeys / kUnitWaves)) - 1); own; own &= own - 1)
    if (lane * 16 < kBytes)
      *(lds_ptr)(stage + (wave * (kTileKeys / kUnitWaves) + __builtin_ctz(own)) * kBytes + lane * 16) = u32x4{};
}

// The rows of codes of a wave's eight keys, where they lie in a row of slots from `slot` on: as
// load_tile, but with scalar addresses that step from row to row and offsets of 32 bits (strides are at
// most kMaxStride).  Vector instructions bound the kernel over codes, and addresses formed lane by lane
// are a sixth of them: 64 requests x 32 heads behind 32768 positions 251 us against 235.  (Rows of bf16
// are bound elsewhere, and for them the same took 231 us against 222, as it leaves too few scalar
// registers.)
constexpr int kWaveRows = kTileKeys / kUnitWaves;
constexpr int64_t kMaxStride = 1 << 24;
__device__ __forceinline__ void load_codes(const Cache& c, int slot, uint32_t lds, int wave) {
  const int lane = lane_here();
  const char* row = c.latent + (int64_t)slot * c.latent_stride;
  const uint32_t second = lane < 32 ? 0 : (uint32_t)c.latent_stride;      // two rows an instruction
  const uint32_t chunk = ((lane & 31) ^ code_swizzle(wave * kWaveRows + (lane >> 5))) * 16;
#pragma unroll
  for (int i = 0; i < kWaveRows; i += 2)
    queue_to_lds(row + i * c.latent_stride, (chunk ^ (uint32_t)(code_swizzle(i) * 16)) + second, lds + (wave * kWaveRows + i) * kLatent);
  const int key = lane >> 3;
  queue_to_lds(c.rope + (int64_t)slot * c.rope_stride,
               (uint32_t)key * (uint32_t)c.rope_stride + ((lane ^ ((wave * kWaveRows + key) >> 1)) & 7) * 16,
               lds + kTileCodes + wave * kWaveRows * kRopeBytes);
}

template <bool E4M3>
__global__ __launch_bounds__(kThreads, 2) void shared_kernel(SharedArgs) {
  using L = Lds<kUnitWaves, 1, E4M3>;
  typedef __attribute__((address_space(3))) uint8_t* byte_ptr;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int share = (int)blockIdx.x;
  auto weight = [&](int e) {
    const Entity u = entity(args_here(), e);
    return blocks_of(u) * cost_of(u);
  };
  // the plan is made where the rows go
  SharePlan& plan = *reinterpret_cast<SharePlan*>(lds);
  {
    const SharedArgs a = args_here();
    plan_shares<kThreads>(weight, a.num_groups + a.num_requests, (uint32_t)share, (uint32_t)a.wgs, kSharedTiles, plan);
  }
  const uint32_t total = __builtin_amdgcn_readfirstlane(plan.total);
  uint32_t lo = __builtin_amdgcn_readfirstlane(plan.begin), start = __builtin_amdgcn_readfirstlane(plan.start);
  const uint32_t hi = __builtin_amdgcn_readfirstlane(plan.end);
  int e = __builtin_amdgcn_readfirstlane(plan.entity);

  const TileReads whole_reads = tile_reads<E4M3>(lane);
  while (lo < hi) {
    const SharedArgs a = args_here();
    const float scale_log2 = fabsf(a.scale_log2);
    // the part [first, last) of the tiles of a unit, whose own cost comes before them
    const Entity u = entity(a, e);
    const uint32_t n = cost_of(u), blocks = blocks_of(u), block = (lo - start) / n, begin = start + block * n;
    const uint32_t until = hi - begin < n ? hi - begin : n;
    const bool begins = lo == begin;
    const int first = lo - begin > kUnitCost ? (int)(lo - begin - kUnitCost) : 0, last = until > kUnitCost ? (int)(until - kUnitCost) : 0;
    const int unit_row = u.row0 + (int)block * kUnitRows;
    const int unit_rows = u.rows - (int)block * kUnitRows < kUnitRows ? u.rows - (int)block * kUnitRows : kUnitRows;
    // Positions end where the request's last row of the unit does; `limit`, where this lane's row does.
    const int32_t* list = a.page_table + (int64_t)u.list * a.pages_per_row;
    const int own_row = wave * 16 + (lane & 15) < unit_rows ? wave * 16 + (lane & 15) : unit_rows - 1;
    const int nth_token = (int)((uint32_t)(unit_row + own_row) / (uint32_t)a.num_heads), token = a.first_token + nth_token;
    int limit = u.key0 + u.keys, end = limit, least = limit;
    if (u.request >= 0) {
      // a token's limit, less its number: the last one's is the length
      const int behind = a.seq_lens[u.request] - a.q_starts[u.request + 1] + 1;
      const int last_token = a.first_token + (int)((uint32_t)(unit_row + unit_rows - 1) / (uint32_t)a.num_heads);
      const int first_token = a.first_token + (int)((uint32_t)unit_row / (uint32_t)a.num_heads);
      limit = behind + token < limit ? behind + token : limit;
      end = behind + last_token < end ? behind + last_token : end;
      least = behind + first_token;
    }
    const bool live_wave = wave * 16 < unit_rows;
    const bool near_rows = a.cache.latent_stride <= kMaxStride && a.cache.rope_stride <= kMaxStride;

    uint32_t masks[L::kAhead + 1];
    int into = 0;                         // the stage of the tile to be queued next
    const uint32_t own_entries = lds_base + L::kEntries + wave * 256;
    const uint32_t scales = lds_base + L::kScales + wave * L::kStages * 128;
    // Tiles begin below 2^31, but the last one may reach past it: positions of single keys are unsigned.
    // (`end` is above 0 wherever there are tiles.)
    const uint32_t part_from = (uint32_t)u.key0 + (uint32_t)first * kTileKeys;
    auto from_of = [&](int i) { return (int)(part_from + (uint32_t)i * kTileKeys); };
    auto load_entries = [&](int i) {
      uint32_t pos = (uint32_t)from_of(i) + (lane_here() & (kTileKeys - 1));
      pos = pos < (uint32_t)end ? pos : (uint32_t)end - 1;
      queue_words_to_lds(list + (pos >> a.log2_page), own_entries + (uint32_t)(i & 1) * 128);
    };
    lds_barrier();                        // the plan's or the last part's reads are done
    const int used = end > u.key0 ? (int)(((uint32_t)(end - u.key0) + kTileKeys - 1) / kTileKeys) : 0;
    const int tiles = __builtin_amdgcn_readfirstlane((used < last ? used : last) - first);
    if (tiles > 0) load_entries(0);

    uint4 q[kLatentSteps + kRopeSteps];
    {
      const int l = lane_here();
      const uint16_t* from = a.q + (int64_t)token * a.q_token_stride +
                             (unit_row + own_row - nth_token * a.num_heads) * a.q_head_stride + (l >> 4) * 8;
#pragma unroll
      for (int k = 0; k < kLatentSteps + kRopeSteps; ++k) q[k] = *reinterpret_cast<const uint4*>(from + k * 32);
    }
    auto queue = [&](int i, uint32_t& mask) {
      const int entry = read_lds<int>(own_entries + (uint32_t)(i & 1) * 128 + (lane_here() & 31) * 4);
      const uint32_t pos = (uint32_t)from_of(i) + (lane_here() & (kTileKeys - 1));
      // (a page beyond 2^31 slots, or a negative one, is not there either)
      const int at = (int)(((uint32_t)entry << a.log2_page) + (pos & ((1u << a.log2_page) - 1)));
      const int slot = pos < (uint32_t)end && (uint32_t)entry <= 0x7FFFFFFFu >> a.log2_page && at < (int)a.cache.num_slots ? at : -1;
      mask = (uint32_t)__ballot(slot >= 0);
      if (i + 1 < tiles) load_entries(i + 1);
      if (E4M3) {
        const float* from = slot >= 0 ? a.cache.scale + slot : reinterpret_cast<const float*>(kZeroRow);
        queue_words_to_lds(from, scales + into * 128);
      }
      // this wave's keys: all there, and in one page?
      const int first_pos = from_of(i) + wave * kWaveRows;
      if (E4M3 && near_rows && (mask >> (wave * kWaveRows) & 0xFF) == 0xFF &&
          (first_pos >> a.log2_page) == ((first_pos + kWaveRows - 1) >> a.log2_page))
        load_codes(a.cache, __builtin_amdgcn_readlane(slot, wave * kWaveRows), lds_base + into * L::kStageBytes, wave);
      else
        load_tile<kUnitWaves, E4M3>(a.cache, slot, lds_base + into * L::kStageBytes, wave);
      into = into + 1 < L::kStages ? into + 1 : 0;
    };
    wait_loads<kLatentSteps + kRopeSteps>();
#pragma unroll
    for (int d = 0; d < L::kAhead; ++d) {
      masks[d] = 0;
      if (d < tiles) {
        queue(d, masks[d]);
        if (d + 1 < L::kAhead) wait_loads<L::kLoads>();        // the next entries
      }
    }
    HeadState st;
    st.m = kNoMax;
    st.l = 0.f;
#pragma unroll
    for (int cb = 0; cb < kColBlocks; ++cb) st.o[cb] = f32x4{};
    const uint32_t sign = a.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int k = 0; k < kLatentSteps + kRopeSteps; ++k)
      st.q[k] = __builtin_bit_cast(bf16x8, make_uint4(q[k].x ^ sign, q[k].y ^ sign, q[k].z ^ sign, q[k].w ^ sign));
    int stage_at = 0;                     // the stage of the tile being computed
    for (int i = 0; i < tiles; ++i) {
      if (L::kAhead > 1 && i + 1 < tiles)
        wait_loads<L::kLoads>();          // all but the next tile's rows
      else
        wait_loads<0>();
      lds_barrier();            // every wave's rows are there, and nobody reads the stage before any more
      masks[L::kAhead] = 0;
      if (i + L::kAhead < tiles) queue(i + L::kAhead, masks[L::kAhead]);
      const int from = from_of(i);
      const uint32_t mask = masks[0] & below(limit, from);
#pragma unroll
      for (int d = 0; d < L::kAhead; ++d) masks[d] = masks[d + 1];
      const uint32_t stage = lds_base + stage_at * L::kStageBytes, sc = scales + stage_at * 128;
      stage_at = stage_at + 1 < L::kStages ? stage_at + 1 : 0;
      // (over codes formed anew: kept, they would be spilled, and a reload waits for all rows on their way)
      const TileReads reads = E4M3 ? tile_reads<E4M3>(lane_here()) : whole_reads;
      f32x4 s[2];
      if (live_wave) score_tile<E4M3>(st, s, stage, sc, reads, lane);
      // (the same for all waves of the workgroup; rows of a unit end within 64 positions, so the difference
      // is a small one or positive)
      if (least < end && least - from < kTileKeys) {
        const uint32_t own = rows_not_finite<E4M3>(stage, wave);
        if (lane == 0) *(byte_ptr)(lds_base + L::kBytes + wave) = (uint8_t)own;
        lds_barrier();          // (all scores are computed, and the bytes read at the tile before are)
        const uint32_t rows = __builtin_amdgcn_readfirstlane(read_lds<uint32_t>(lds_base + L::kBytes));
        if (rows) {
          if (!E4M3 && live_wave) add_nothing(st, stage, rows, mask);
          lds_barrier();
          clear_rows<E4M3>(stage, wave, rows);
          lds_barrier();
        }
      }
      if (live_wave) {
        const bf16x8 p = weights_of_tile<E4M3, true>(st, s, sc, mask, scale_log2, lane);
        for_values<E4M3>(stage, reads, [&](int cb, bf16x8 cols) { st.o[cb] = mfma16(cols, p, st.o[cb]); });
      }
    }

    const SharedArgs after = args_here();
    const Entity v = entity(after, e);
    // this part's places: a unit's first part has its own, any other its share's
    const int piece = begins ? first_piece(after, v) + (int)block * kUnitWaves : 2 * after.pieces + share * kUnitWaves;
    const float l = sum_of_4(st.l);       // this lane's row: its sum is spread over four lanes
    if (live_wave) {
      const int64_t at = piece + wave;
      float* o = after.part_out + at * (kHeads * kLatent) + lane * 4;
#pragma unroll
      for (int cb = 0; cb < kColBlocks; ++cb) *reinterpret_cast<f32x4*>(o + cb * 256) = st.o[cb];
      if (lane < kHeads) after.part_ml[at * kHeads + lane] = make_float2(st.m, l);
    }
    if (begins && tid < unit_rows) {
      const Shares shares(total, (uint32_t)after.wgs, kSharedTiles);
      const int parts = (int)shares.owner(begin + n - 1) - share + 1;
      int4* rec = after.part_rec + 2 * ((int64_t)unit_row + tid);
      rec[v.request >= 0 ? 1 : 0] = make_int4(piece + (tid >> 4), 2 * after.pieces + (share + 1) * kUnitWaves + (tid >> 4), parts, tid & 15);
      if (v.request >= 0 && v.key0 == 0) rec[0] = make_int4(0, 0, 0, 0);       // no shared prefix
    }
    lo = begin + until;
    if (block + 1 == blocks && lo == begin + n) {
      start += blocks * n;
      if (lo < hi) e = __builtin_amdgcn_readfirstlane(next_entity(weight, e + 1, after.num_groups + after.num_requests));
    }
  }
}

// Joins a row's parts: out = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p.  As in the absorbed
// kernel's join, a workgroup takes 16 rows and kJoinBlocks blocks of 16 latent values, its waves every
// fourth part each, with kJoinAhead parts' loads in flight; but rows' parts lie in places of their own,
// so every lane finds its row's.
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

__global__ __launch_bounds__(64 * kJoinWaves) void shared_join_kernel(SharedArgs a) {
  __shared__ f32x4 others_o[kJoinWaves - 1][kJoinBlocks][64];
  __shared__ float2 others_ml[kJoinWaves - 1][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int cb0 = blockIdx.y * kJoinBlocks, group = lane >> 4;
  const int64_t row0 = (int64_t)a.first_token * a.num_heads;
  const int64_t row = (int64_t)blockIdx.x * 16 + (lane & 15);
  int64_t rows = ((int64_t)a.q_starts[a.num_requests] - a.first_token) * a.num_heads;
  const int64_t most = (int64_t)a.num_tokens * a.num_heads;
  rows = rows < most ? rows : most;
  if ((int64_t)blockIdx.x * 16 >= rows) return;
  int4 r0 = make_int4(0, 0, 0, 0), r1 = r0;
  if (row < rows) {
    r0 = a.part_rec[2 * row];
    r1 = a.part_rec[2 * row + 1];
  }
  // (places within the workspace also where starts do not ascend and rows have no record)
  const int places = 2 * a.pieces + a.wgs * kUnitWaves;
  r0.z = r0.z < 0 ? 0 : (r0.z < a.wgs ? r0.z : a.wgs);
  r1.z = r1.z < 0 ? 0 : (r1.z < a.wgs ? r1.z : a.wgs);
  const int parts = r0.z + r1.z;
  int longest = parts;
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const int o = __shfl_xor(longest, d);
    longest = o > longest ? o : longest;
  }
  JoinState st;
  st.m = kNoMax;
  st.l = 0.f;
#pragma unroll
  for (int c = 0; c < kJoinBlocks; ++c) st.o[c] = f32x4{};
  for (int p0 = w; p0 < longest; p0 += kJoinWaves * kJoinAhead) {
    float2 ml[kJoinAhead];
    f32x4 o[kJoinAhead][kJoinBlocks];
#pragma unroll
    for (int d = 0; d < kJoinAhead; ++d) {
      const int p = p0 + d * kJoinWaves;
      const int4 r = p < r0.z ? r0 : r1;
      const int nth = p < r0.z ? p : p - r0.z;
      ml[d] = make_float2(kNoMax, 0.f);
#pragma unroll
      for (int c = 0; c < kJoinBlocks; ++c) o[d][c] = f32x4{};
      if (p < parts) {
        const int64_t at = (int64_t)clamp_to(nth == 0 ? r.x : r.y + (int64_t)(nth - 1) * kUnitWaves, 0, places - 1);
        const int i = r.w & 15;
        ml[d] = a.part_ml[at * kHeads + i];
#pragma unroll
        for (int c = 0; c < kJoinBlocks; ++c)
          o[d][c] = *reinterpret_cast<const f32x4*>(a.part_out + at * (kHeads * kLatent) + (cb0 + c) * 256 + (group * 16 + i) * 4);
      }
    }
#pragma unroll
    for (int d = 0; d < kJoinAhead; ++d) st.add(ml[d].x, ml[d].y, o[d]);
  }
  if (w > 0) {
#pragma unroll
    for (int c = 0; c < kJoinBlocks; ++c) others_o[w - 1][c][lane] = st.o[c];
    others_ml[w - 1][lane] = make_float2(st.m, st.l);
  }
  __syncthreads();
  if (w > 0 || row >= rows) return;
#pragma unroll
  for (int other = 0; other < kJoinWaves - 1; ++other) {
    const float2 ml = others_ml[other][lane];
    f32x4 o[kJoinBlocks];
#pragma unroll
    for (int c = 0; c < kJoinBlocks; ++c) o[c] = others_o[other][c][lane];
    st.add(ml.x, ml.y, o);
  }
  const float inv = inverse_sum(st.l);
#pragma unroll
  for (int c = 0; c < kJoinBlocks; ++c) {
    bf16x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = (__bf16)(st.o[c][r] * inv);
    *reinterpret_cast<bf16x4*>(a.out + (row0 + row) * kLatent + (cb0 + c) * 16 + 4 * group) = v;
  }
  if (a.lse && cb0 == 0 && group == 0) a.lse[row0 + row] = log_sum(st.m, st.l);
}

template <bool E4M3>
hipError_t launch(const SharedArgs& a, hipStream_t stream) {
  constexpr int kLds = Lds<kUnitWaves, 1, E4M3>::kBytes + 16;      // the ring, a byte of bits a wave
  static_assert(kUnitWaves == 4 && kTileKeys == 8 * kUnitWaves, "a word of bits");
  static_assert(2 * (kLds + 1280) <= 160 * 1024, "two workgroups to a CU");
  hipLaunchKernelGGL(shared_kernel<E4M3>, dim3((unsigned)a.wgs), dim3(kThreads), kLds, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t blocks = ((int64_t)a.num_tokens * a.num_heads + 15) / 16;
  hipLaunchKernelGGL(shared_join_kernel, dim3((unsigned)blocks, kColBlocks / kJoinBlocks), dim3(64 * kJoinWaves), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

// Tokens of a launch: parts of 32 KB for every 16 of their rows, and for every one of them that begins a
// piece, within 1 GB; and tiles that 31 bits count.
int shared_tokens(int num_tokens, int num_heads, int64_t keys) {
  int64_t n = 16384 / (num_heads / 8 + 2);
  n = n < 1 ? 1 : (n < num_tokens ? n : num_tokens);
  const int64_t tiles = keys / kTileKeys + 2 + kUnitCost;
  auto units = [&](int64_t t) { return 2 * (t * num_heads / kUnitRows + t + 1); };
  while (n > 1 && units(n) > (int64_t)INT32_MAX / tiles) n = (n + 1) / 2;
  return units(n) > (int64_t)INT32_MAX / tiles ? 0 : (int)n;
}

int shared_pieces(int num_tokens, int num_heads) { return (int)((int64_t)num_tokens * num_heads / 16 + num_tokens + 1); }

SplitLayout shared_layout(int num_tokens, int num_heads, int wgs) {
  const size_t pieces = (size_t)2 * shared_pieces(num_tokens, num_heads) + (size_t)wgs * kUnitWaves;
  SplitLayout s;
  s.out_bytes = pieces * kHeads * kLatent * sizeof(float);
  s.ml_bytes = pieces * kHeads * sizeof(float2);
  s.rec_bytes = (size_t)num_tokens * num_heads * 2 * sizeof(int4);
  return s;
}

hipError_t launch_shared(const SharedArgs& a, bool e4m3, hipStream_t stream) {
  return e4m3 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace latent
