// mla_kvscaled.cu -- quantising write of new latent rows into an e4m3 cache
// with one power-of-two scale per block of G cache rows (mla_write_kv_scaled).
//
// A unit is one scale block that receives rows: its first new row (offset f in
// the block) leads it, the rows that follow it in the block belong to it, and
// the f rows before it were written by earlier calls.  The unit's threads load
// all of its new rows at once, reduce max |x|, choose the scale, and write the
// codes from the registers that still hold the rows: each value is read once and
// each code written once, which is the whole traffic unless a scale grows (the
// earlier rows' codes are then read and rewritten).
//
// Bound by memory, so by the loads in flight: the pieces a thread holds follow
// from G (four rows a warp at G = 1, a warp per unit up to G = 4, then a CTA of
// 128 to 512 threads), which keeps the registers low enough for 32 warps per SM.
// One kernel with 18 pieces for every G ran at one CTA of 8 warps per SM: 109 us
// for 136,000 rows at G = 64; and a warp that took one row at a time 65 us for
// 131,072 at G = 1, against 43 with four.
//
// Scale: 2^k, the smallest with max |x| <= 448 * 2^k.  With max |x| = m 2^e,
// m in [1, 2), and 448 = 1.75 * 2^8, that is k = e - 8, plus one when m > 1.75;
// both come from the bf16 bits, and x / 2^k is exact.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kRowPieces = 72;   // 16-byte pieces (8 values) of a new row
constexpr int kMaxGroup = 64;    // rows of a scale block at most
constexpr int kMinExp = -100;
constexpr int kWarpCta = 256;    // threads of a CTA whose warps take a unit each

struct WriteScaledParams {
  const uint4 *x;
  const int32_t *slots;
  uint2 *cache;
  float *scales;
  int *err;
  int num_rows, log_g, num_cache_rows;
  int window;  // rows whose units one CTA (or warp) writes
};

// Largest |x| of a packed pair and what was seen so far (NaN is passed over).
__device__ __forceinline__ __nv_bfloat162 pair_max(__nv_bfloat162 m, uint32_t v) {
  return __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&v)));
}

// bits of the larger of two bf16 magnitudes
__device__ __forceinline__ uint32_t max_bits(__nv_bfloat162 m) {
  const uint32_t u = *reinterpret_cast<const uint32_t *>(&m);
  return max(u & 0xffffu, u >> 16);
}

// bits of the larger finite one of two bf16 magnitudes
__device__ __forceinline__ uint32_t finite_bits(uint32_t v) {
  const uint32_t lo = v & 0x7fffu, hi = (v >> 16) & 0x7fffu;
  return max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u);
}

// The exponent k of the scale for a largest magnitude given as bf16 bits.
__device__ __forceinline__ int scale_exp(uint32_t bits) {
  const int k = static_cast<int>(bits >> 7) - 127 - 8 + ((bits & 0x7f) > 0x60 ? 1 : 0);
  return bits == 0 ? kMinExp : max(k, kMinExp);
}

__device__ __forceinline__ float pow2f(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

// Two bf16 values by a factor, as floats.
__device__ __forceinline__ float2 scaled(uint32_t v, float f) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, y;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmul.rn.f32x2 y, a, b;\n\t"
      "mov.b64 {%0, %1}, y;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "r"(v << 16), "r"(v & 0xffff0000u), "f"(f));
  return y;
}
__device__ __forceinline__ uint32_t codes4(float2 lo, float2 hi) {
  return __byte_perm(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3),
                     __nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3), 0x5410);
}
__device__ __forceinline__ float2 divided(uint32_t v, float d) {
  return make_float2(__uint_as_float(v << 16) / d, __uint_as_float(v & 0xffff0000u) / d);
}

__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> (16 * h)), __NV_E4M3);
    float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r));
    f = make_float2(f.x * ratio, f.y * ratio);
    out |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)) << (16 * h);
  }
  return out;
}

// One unit by `kTeam` threads (a warp, or the whole CTA): rows[0 .. n) are its
// new rows, ascending, n <= kG; first_slot is rows[0]'s cache row.  A CTA meets
// at one barrier: team[0 .. kTeam / 32) takes the warps' maxima and team[kTeam /
// 32] the old scale, in the other of two copies every unit.
template <int kTeam, int kG>
__device__ __forceinline__ void write_unit(const WriteScaledParams &p, const int *rows, int n, int first_slot, int t,
                                           uint32_t *team) {
  constexpr uint32_t kAll = 0xffffffffu;
  constexpr int kHeld = (kG * kRowPieces + kTeam - 1) / kTeam;  // pieces a thread holds
  const int pieces = n * kRowPieces;
  const int f = first_slot & ((1 << p.log_g) - 1), block = first_slot >> p.log_g;
  uint4 v[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = t + i * kTeam;
    v[i] = make_uint4(0, 0, 0, 0);
    if (c < pieces) v[i] = p.x[static_cast<int64_t>(rows[c / kRowPieces]) * kRowPieces + c % kRowPieces];
  }
  float old = 0.0f;
  if (f > 0 && (kTeam == 32 || t == 0)) old = p.scales[block];
  __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) m = pair_max(pair_max(pair_max(pair_max(m, v[i].x), v[i].y), v[i].z), v[i].w);
  uint32_t top = max_bits(m);
  if (top >= 0x7f80) {  // an infinity among them: only finite values count
    top = 0;
#pragma unroll 1
    for (int c = t; c < pieces; c += kTeam) {
      const uint4 u = p.x[static_cast<int64_t>(rows[c / kRowPieces]) * kRowPieces + c % kRowPieces];
      top = max(max(top, max(finite_bits(u.x), finite_bits(u.y))), max(finite_bits(u.z), finite_bits(u.w)));
    }
  }
  top = __reduce_max_sync(kAll, top);
  if (kTeam > 32) {
    if ((t & 31) == 0) team[t >> 5] = top;
    if (t == 0) team[kTeam / 32] = __float_as_uint(old);
    __syncthreads();
    top = __reduce_max_sync(kAll, (t & 31) < kTeam / 32 ? team[t & 31] : 0u);
    old = __uint_as_float(team[kTeam / 32]);
  }
  const float want = pow2f(scale_exp(top));
  const float scale = f > 0 ? fmaxf(old, want) : want;
  uint2 *dst = p.cache + static_cast<int64_t>(first_slot) * kRowPieces;  // the unit's slots follow one another
  if ((__float_as_uint(scale) & 0x7fffffu) == 0) {
    const float inv = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = t + i * kTeam;
      if (c < pieces)
        dst[c] = make_uint2(codes4(scaled(v[i].x, inv), scaled(v[i].y, inv)),
                            codes4(scaled(v[i].z, inv), scaled(v[i].w, inv)));
    }
  } else {  // a scale that another writer chose: divide
#pragma unroll 1
    for (int c = t; c < pieces; c += kTeam) {
      const uint4 u = p.x[static_cast<int64_t>(rows[c / kRowPieces]) * kRowPieces + c % kRowPieces];
      dst[c] = make_uint2(codes4(divided(u.x, scale), divided(u.y, scale)),
                          codes4(divided(u.z, scale), divided(u.w, scale)));
    }
  }
  if (f > 0 && scale > old) {
    const float ratio = old / scale;
    uint2 *prior = dst - f * kRowPieces;
#pragma unroll 2
    for (int c = t; c < f * kRowPieces; c += kTeam) {
      const uint2 u = prior[c];
      prior[c] = make_uint2(rescale4(u.x, ratio), rescale4(u.y, ratio));
    }
  }
  if (t == 0) p.scales[block] = scale;
}

// The slot map, `n` entries of it from `first` on held in shared memory.
struct Slots {
  const int32_t *map;
  const int *near;
  int first;
  uint32_t n;
  __device__ __forceinline__ int operator[](int r) const {
    const uint32_t k = static_cast<uint32_t>(r - first);
    return k < n ? near[k] : map[r];
  }
};

__device__ __forceinline__ bool has_slot(const WriteScaledParams &p, int s) { return s >= 0 && s < p.num_cache_rows; }

// Nearest slot before row `end` (a warp; -1: none).  Rows without one may be many: another shard's, or those
// before the first request's own.
__device__ __forceinline__ int slot_before(const WriteScaledParams &p, int end, int lane) {
  constexpr int kLook = 16;  // loads in flight
  for (; end > 0; end -= 32 * kLook) {
    int s[kLook];
#pragma unroll
    for (int i = 0; i < kLook; ++i) {
      const int r = end - 32 * (i + 1) + lane;
      s[i] = r >= 0 ? p.slots[r] : -1;
    }
#pragma unroll
    for (int i = 0; i < kLook; ++i) {
      const uint32_t got = __ballot_sync(0xffffffffu, has_slot(p, s[i]));
      if (got) return __shfl_sync(0xffffffffu, s[i], 31 - __clz(got));
    }
  }
  return -1;
}

// Leaders among rows r0 .. r0 + 31 (a warp): the row of lane l opens a unit.
// A row whose nearest earlier row with a slot lies in the same scale block
// follows a leader; rows without a slot (another shard's) are passed over.  A
// follower has the next cache row, or is recorded as out of order.
__device__ __forceinline__ uint32_t leaders(const WriteScaledParams &p, const Slots &slots, int r0, int r_end, int lane,
                                            int &slot) {
  const int r = r0 + lane;
  const int prior = r0 - 32 + lane >= 0 ? slots[r0 - 32 + lane] : -1;
  slot = r < r_end ? slots[r] : -1;
  if (slot >= p.num_cache_rows || slot < -1) {
    atomicCAS(p.err, 0, MLA_DEV_BAD_BLOCK_ID);
    slot = -1;
  }
  const uint32_t have = __ballot_sync(0xffffffffu, slot >= 0);
  if (have == 0) return 0;
  // the nearest earlier slot: in these 32 rows, or before them
  const uint32_t below = have & ((1u << lane) - 1u);
  int prev = __shfl_sync(0xffffffffu, slot, below ? 31 - __clz(below) : 0);
  const uint32_t got = __ballot_sync(0xffffffffu, has_slot(p, prior));
  const int before = got ? __shfl_sync(0xffffffffu, prior, 31 - __clz(got)) : slot_before(p, r0 - 32, lane);
  if (below == 0) prev = before;
  const bool follows = slot >= 0 && prev >= 0 && (prev >> p.log_g) == (slot >> p.log_g);
  if (follows && slot != prev + 1) atomicCAS(p.err, 0, MLA_DEV_BAD_BLOCK_ID);
  return __ballot_sync(0xffffffffu, slot >= 0 && !follows);
}

// 32 slots, row r's for lane 0 first (a warp): the rows of the unit among them go to rows[n ..).  False when
// the unit ends here: with another block's row, the block's last row, or before a row that is not the next one
// of its block (the unit's codes go to one run of cache rows).
__device__ __forceinline__ bool take_rows(const WriteScaledParams &p, int r, int s, int first_slot, int lane, int *rows,
                                          int &n, bool &blank) {
  const bool valid = has_slot(p, s);
  const uint32_t other = __ballot_sync(0xffffffffu, valid && (s >> p.log_g) != (first_slot >> p.log_g));
  const uint32_t upto = other ? (1u << (__ffs(other) - 1)) - 1u : 0xffffffffu;
  const uint32_t mine = __ballot_sync(0xffffffffu, valid) & upto;
  const int at = n + __popc(mine & ((1u << lane) - 1u));
  const bool here = mine >> lane & 1u, next = s == first_slot + at;
  const uint32_t odd = __ballot_sync(0xffffffffu, here && !next);
  const uint32_t good = odd ? mine & ((1u << (__ffs(odd) - 1)) - 1u) : mine;
  if (good >> lane & 1u) rows[at] = r + lane;
  n += __popc(good);
  blank = mine == 0;
  return (other | odd) == 0 && ((first_slot + n) & ((1 << p.log_g) - 1)) != 0;
}

// The rows of the unit that row r0 leads, among rows r0 .. end - 1 (a warp), into rows[]; returns how many,
// and whether later rows may belong to it.
__device__ __forceinline__ int members(const WriteScaledParams &p, const Slots &slots, int r0, int end, int first_slot,
                                       int lane, int *rows, bool &open) {
  int n = 0;
  bool blank;
  open = true;
  for (int b0 = r0; b0 < end && open; b0 += 32)
    open = take_rows(p, b0, b0 + lane < end ? slots[b0 + lane] : -1, first_slot, lane, rows, n, blank);
  open = open && end < p.num_rows;
  __syncwarp();
  return n;
}

// What a team shares while it looks for a unit's far rows.
template <int kG>
struct Far {
  int next, at, n;
  int rows[kG];
};

// The unit's rows from row `at` on, n of them being known (the whole team, kTeam threads: a warp or the CTA);
// copied behind the others into rows[] of every warp, returns how many there are now.  Between a unit's rows,
// and behind the last one in a step that is smaller than its capacity, any number of rows may have no slot.
// The first warp takes rows while they are near each other, then the team looks for the next one together,
// 16 slots a thread in flight: nine new rows in a capacity of 8,192 or 131,072 take 4.5-4.9 and 13-24 us at
// G >= 8 in a graph (each warp for itself, 32 slots at a time: 76-91 and 1,200-1,420), 32 slots a thread
// the same but slower steps without empty rows (22,200 rows at G = 2: 7.7 us against 7.5), 8 slots 5.0-5.6
// and 16-36.
template <int kTeam, int kG>
__device__ __forceinline__ int far_members(const WriteScaledParams &p, int first_slot, int at, int n, int t, int *rows,
                                        Far<kG> &far) {
  constexpr int kWarps = kTeam / 32, kLook = 16;
  const int lane = t & 31, warp = t >> 5, n0 = n;
  auto sync = [] {
    if (kTeam == 32) __syncwarp();
    else __syncthreads();
  };
  for (;;) {
    if (warp == 0) {  // up to 32 rows without a slot
      bool more = true, blank = false;
      int b0 = at;
      for (; b0 < p.num_rows && more && !blank; b0 += 32)
        more = take_rows(p, b0, b0 + lane < p.num_rows ? p.slots[b0 + lane] : -1, first_slot, lane, far.rows, n, blank);
      if (lane == 0) {
        far.at = b0;
        far.n = n;
        far.next = more ? p.num_rows : 0;
      }
    }
    sync();
    n = far.n;
    if (far.next == 0) break;
    // the next row with a slot: the warps take stretches of 32 kLook rows in turn
    sync();
    for (int64_t c0 = far.at + 32 * kLook * warp;; c0 += 32 * kLook * kWarps) {
      if (c0 >= __shfl_sync(0xffffffffu, *const_cast<volatile int *>(&far.next), 0)) break;
      int s[kLook], found = INT32_MAX;
#pragma unroll
      for (int i = 0; i < kLook; ++i) {
        const int64_t r = c0 + 32 * i + lane;
        s[i] = r < p.num_rows ? p.slots[r] : -1;
      }
#pragma unroll
      for (int i = kLook - 1; i >= 0; --i)
        if (has_slot(p, s[i])) found = 32 * i + lane;
      found = __reduce_min_sync(0xffffffffu, found);
      if (found != INT32_MAX) {
        if (lane == 0) atomicMin(&far.next, static_cast<int>(c0) + found);
        break;
      }
    }
    sync();
    at = far.next;
    if (at >= p.num_rows) break;
    sync();  // (next is written anew)
  }
  for (int i = n0 + lane; i < n; i += 32) rows[i] = far.rows[i];
  __syncwarp();
  return n;
}

// A CTA per unit: scale blocks of 8 rows or more.
template <int kThreads, int kG>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) write_scaled_cta(const WriteScaledParams p) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int s_lead[kMaxGroup], s_slot[kMaxGroup], s_units;
  __shared__ int s_rows[kThreads / 32][kG];
  __shared__ uint32_t s_team[2][kThreads / 32 + 1];
  __shared__ Far<kG> s_far;
  // The slots that the window and its last unit touch, and 32 before, in one load: leaders and members
  // read from the map are three loads, one after another, before the first row's (136,000 rows at
  // G = 64: 51.4 -> 48.4 us).
  constexpr int kNear = 32 + kMaxGroup + kG;
  __shared__ int s_near[kNear];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = blockIdx.x * p.window, r_end = min(p.num_rows, r0 + p.window);
  const Slots slots{p.slots, s_near, r0 - 32, kNear};
#pragma unroll
  for (int i = tid; i < kNear; i += kThreads) {
    const int r = r0 - 32 + i;
    s_near[i] = r >= 0 && r < p.num_rows ? p.slots[r] : -1;
  }
  __syncthreads();
  if (warp == 0) {
    int units = 0;
    for (int w0 = r0; w0 < r_end; w0 += 32) {
      int slot;
      const uint32_t lead = leaders(p, slots, w0, r_end, lane, slot);
      if (lead >> lane & 1u) {
        const int at = units + __popc(lead & ((1u << lane) - 1u));
        s_lead[at] = w0 + lane;
        s_slot[at] = slot;
      }
      units += __popc(lead);
    }
    if (lane == 0) s_units = units;
  }
  __syncthreads();
  const int units = s_units;
  const int near_end = min(p.num_rows, r0 - 32 + kNear);
  for (int u = 0; u < units; ++u) {  // every warp finds the unit's rows itself: a barrier less
    bool open;  // (the same in all warps, which read the same slots in shared memory)
    int n = members(p, slots, s_lead[u], near_end, s_slot[u], lane, s_rows[warp], open);
    if (open) n = far_members<kThreads, kG>(p, s_slot[u], near_end, n, tid, s_rows[warp], s_far);
    write_unit<kThreads, kG>(p, s_rows[warp], n, s_slot[u], tid, s_team[u & 1]);
    __syncwarp();
  }
}

// G = 1: every row has a scale of its own and no row before it, so a row needs
// nothing but itself.  A warp takes up to kRowsHeld rows at once, so that its
// loads do not wait for the row before.
constexpr int kRowsHeld = 4;
__global__ void __launch_bounds__(kWarpCta, 4) write_scaled_rows(const WriteScaledParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (kWarpCta / 32) + (threadIdx.x >> 5)) * p.window;
  int slot = lane < p.window && r0 + lane < p.num_rows ? p.slots[r0 + lane] : -1;
  if (slot >= p.num_cache_rows || slot < -1) {
    atomicCAS(p.err, 0, MLA_DEV_BAD_BLOCK_ID);
    slot = -1;
  }
  if (__ballot_sync(0xffffffffu, slot >= 0) == 0) return;
  constexpr int kHeld = (kRowPieces + 31) / 32;
  uint4 v[kRowsHeld][kHeld];
#pragma unroll
  for (int u = 0; u < kRowsHeld; ++u) {
    const bool live = __shfl_sync(0xffffffffu, slot, u) >= 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = lane + 32 * i;
      v[u][i] = make_uint4(0, 0, 0, 0);
      if (live && c < kRowPieces) v[u][i] = p.x[(r0 + u) * kRowPieces + c];
    }
  }
#pragma unroll
  for (int u = 0; u < kRowsHeld; ++u) {
    const int at = __shfl_sync(0xffffffffu, slot, u);
    if (at < 0) continue;
    __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      m = pair_max(pair_max(pair_max(pair_max(m, v[u][i].x), v[u][i].y), v[u][i].z), v[u][i].w);
    uint32_t top = max_bits(m);
    if (top >= 0x7f80) {  // an infinity among them: only finite values count
      top = 0;
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        top = max(max(top, max(finite_bits(v[u][i].x), finite_bits(v[u][i].y))),
                  max(finite_bits(v[u][i].z), finite_bits(v[u][i].w)));
    }
    const float scale = pow2f(scale_exp(__reduce_max_sync(0xffffffffu, top))), inv = 1.0f / scale;
    uint2 *dst = p.cache + static_cast<int64_t>(at) * kRowPieces;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = lane + 32 * i;
      if (c < kRowPieces)
        dst[c] = make_uint2(codes4(scaled(v[u][i].x, inv), scaled(v[u][i].y, inv)),
                            codes4(scaled(v[u][i].z, inv), scaled(v[u][i].w, inv)));
    }
    if (lane == 0) p.scales[at] = scale;
  }
}

// A warp per unit: scale blocks of 2 or 4 rows.
template <int kG>
__global__ void __launch_bounds__(kWarpCta, 4) write_scaled_warp(const WriteScaledParams p) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int s_rows[kWarpCta / 32][kG];
  __shared__ Far<kG> s_far[kWarpCta / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (kWarpCta / 32) + warp) * p.window;
  if (r0 >= p.num_rows) return;
  const int r_end = static_cast<int>(min(static_cast<int64_t>(p.num_rows), r0 + p.window));
  int slot;
  const Slots slots{p.slots, nullptr, 0, 0};
  uint32_t lead = leaders(p, slots, static_cast<int>(r0), r_end, lane, slot);
  while (lead) {
    const int l = __ffs(lead) - 1;
    lead &= lead - 1;
    const int first_slot = __shfl_sync(0xffffffffu, slot, l);
    const int r = static_cast<int>(r0) + l, end = min(p.num_rows, r + 32);
    bool open;
    int n = members(p, slots, r, end, first_slot, lane, s_rows[warp], open);
    if (open) n = far_members<32, kG>(p, first_slot, end, n, lane, s_rows[warp], s_far[warp]);
    write_unit<32, kG>(p, s_rows[warp], n, first_slot, lane, nullptr);
    __syncwarp();
  }
}

std::atomic<int> g_write_sms[64];

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_write_kv_scaled(int num_rows, const void *kv_new, const int32_t *slot_map, void *kv_cache,
                                          float *kv_scales, int scale_block, int64_t num_cache_rows,
                                          mla_stream_t stream) {
  if (num_rows < 0 || num_cache_rows < 1 || num_cache_rows > INT32_MAX || kv_cache == nullptr || kv_scales == nullptr ||
      (num_rows > 0 && (kv_new == nullptr || slot_map == nullptr))) {
    set_error("mla_write_kv_scaled: bad sizes or null pointers (T=%d, %lld cache rows)", num_rows,
              (long long)num_cache_rows);
    return MLA_ERR_INVALID_ARG;
  }
  if (scale_block < 1 || scale_block > kMaxGroup || (scale_block & (scale_block - 1)) != 0) {
    set_error("mla_write_kv_scaled: scale_block %d unsupported (power of two in [1, %d])", scale_block, kMaxGroup);
    return MLA_ERR_UNSUPPORTED;
  }
  if (num_cache_rows % scale_block != 0) {
    set_error("mla_write_kv_scaled: %lld cache rows are not whole scale blocks of %d", (long long)num_cache_rows,
              scale_block);
    return MLA_ERR_INVALID_ARG;
  }
  if ((reinterpret_cast<uintptr_t>(kv_new) | reinterpret_cast<uintptr_t>(kv_cache)) % 16 != 0) {
    set_error("mla_write_kv_scaled: kv_new and kv_cache must be 16-byte aligned");
    return MLA_ERR_INVALID_ARG;
  }
  if (num_rows == 0) return MLA_OK;
  int *err = device_error_word();
  if (err == nullptr) return MLA_ERR_CUDA;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  int sms = g_write_sms[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(SM count)");
    g_write_sms[dev].store(sms, std::memory_order_relaxed);
  }
  WriteScaledParams p{};
  p.x = static_cast<const uint4 *>(kv_new);
  p.slots = slot_map;
  p.cache = static_cast<uint2 *>(kv_cache);
  p.scales = kv_scales;
  p.err = err;
  p.num_rows = num_rows;
  p.log_g = __builtin_ctz(static_cast<unsigned>(scale_block));
  p.num_cache_rows = static_cast<int>(num_cache_rows);
  const bool by_cta = scale_block >= 8;
  // Rows per team: one while the GPU holds a team for every row (so that a step's few tokens spread out),
  // then as many as give one wave of teams (rounded down, a second wave of a few: 131,072 rows at G = 8 44.4
  // us against 40.4), within the list of leaders (64), a warp's lanes or the rows that it holds.  Teams of
  // CTAs have nine pieces a thread (G = 16 with 256 threads: 43.4 us against 39.4), but at G = 8, whose 64
  // threads would be slow for a step's few rows (1,152 rows: 4.0 us against 3.2).
  const int team_warps = !by_cta ? 1 : scale_block == 8 ? 4 : scale_block / 4;
  const int teams = sms * 64 / team_warps, most = by_cta ? kMaxGroup : scale_block == 1 ? kRowsHeld : 32;
  int window = (num_rows + teams - 1) / teams;
  window = window < 1 ? 1 : (window > most ? most : window);
  p.window = window;
  const int per_cta = by_cta ? window : window * (kWarpCta / 32);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(num_rows) + per_cta - 1) / per_cta));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (scale_block) {
    case 1: e = launch_pdl(write_scaled_rows, grid, dim3(kWarpCta), 0, s, p); break;
    case 2: e = launch_pdl(write_scaled_warp<2>, grid, dim3(kWarpCta), 0, s, p); break;
    case 4: e = launch_pdl(write_scaled_warp<4>, grid, dim3(kWarpCta), 0, s, p); break;
    case 8: e = launch_pdl(write_scaled_cta<128, 8>, grid, dim3(128), 0, s, p); break;
    case 16: e = launch_pdl(write_scaled_cta<128, 16>, grid, dim3(128), 0, s, p); break;
    case 32: e = launch_pdl(write_scaled_cta<256, 32>, grid, dim3(256), 0, s, p); break;
    default: e = launch_pdl(write_scaled_cta<512, 64>, grid, dim3(512), 0, s, p); break;
  }
  return e == cudaSuccess ? MLA_OK : cuda_fail(e, "write_kv_scaled launch");
}
