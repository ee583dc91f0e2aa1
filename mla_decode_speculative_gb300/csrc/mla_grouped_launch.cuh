// mla_grouped_launch.cuh -- the merge of the units that the split cuts, and the
// two launches of a call, for one configuration.  Included by the translation
// units that instantiate them.
#pragma once
#include <atomic>

#include "mla_grouped.cuh"

namespace mla {
namespace grouped {

// Merge of one cut unit: its parts are record 1 of the chunk with its first
// tile and record 0 of the chunks after it.  A warp takes a row's map:
// statistics with a lane per part, then the parts' outputs, 64 W values over 32
// lanes, weighted by 2^(m - M) / L; the difference of the maps and its norm go
// through shared memory.  Bound by round trips, so the first parts' outputs are
// read beside the statistics, 8 or 12 at a time: with four of them and a warp per
// row 16 units of ten parts took 5 us more than no merge, 24 differential ones of
// seven 6 us (now 4.3 each).  Four warps per row and map were slower but for units
// of a hundred parts (48 window units 28.7 -> 32.6).
constexpr int kMergeRows = 4;

template <int kV>
__device__ __forceinline__ void load_row(const float *o, float (&v)[kV]) {
  if constexpr (kV == 2) {
    *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(o);
  } else {
#pragma unroll
    for (int k = 0; k < kV; k += 4) *reinterpret_cast<float4 *>(v + k) = *reinterpret_cast<const float4 *>(o + k);
  }
}

template <int kW, int kMaps, int kNC>
__global__ void __launch_bounds__(32 * kMergeRows *kMaps) grouped_merge(const __grid_constant__ Params p) {
  constexpr int kNR = kNC / kMaps, kDv = 64 * kW, kV = kDv / 32;
  constexpr int kAhead = kW == 4 ? 8 : 12;
  __shared__ float weight[kMergeRows * kMaps][kMaxCtas];
  __shared__ alignas(16) float other[kMergeRows][kMaps == 2 ? kDv : 4];
  grid_dep_wait();
  grid_dep_launch();
  const int first = static_cast<int>(blockIdx.x), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 u = *reinterpret_cast<const int4 *>(p.meta + first);  // q0, qlen, g, rb
  const int last = p.meta[first].last, step = p.meta[first].step;
  if (last < 0) return;
  const int m = kMaps == 2 ? warp & 1 : 0, slot = warp / kMaps;  // the warps of a row lie together
  const int parts = (last - first) / step + 1, c = static_cast<int>(blockIdx.y) * kMergeRows + slot;
  int t, h;
  const bool there = column_row(p, u.w, c, u.y, t, h);
  if (!there) {
    if (kMaps == 2) __syncthreads();
    return;
  }
  h += u.z * p.group;
  const int64_t row = (static_cast<int64_t>(u.x) + t) * p.num_heads + h;
  auto record = [&](int i) { return (static_cast<int64_t>(first) + i * step) * 2 + (i == 0 ? 1 : 0); };
  const float *stats = p.part_stat + m * kNR + c;
  const float *outs = p.part_o + (m * kNR + c) * kDv + lane * kV;
  const float m0 = lane < parts ? stats[record(lane) * 2 * kNC] : kLowest;
  const float l0 = lane < parts ? stats[record(lane) * 2 * kNC + kNC] : 0.0f;
  float ahead[kAhead][kV], gain[kV], lam = 0.0f;
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (i < parts) load_row<kV>(outs + record(i) * kNC * kDv, ahead[i]);
  if (kMaps == 2) {
    lam = p.lambda[h];
#pragma unroll
    for (int k = 0; k < kV; ++k) gain[k] = p.gain != nullptr ? p.gain[lane * kV + k] : 1.0f;
  }
  float top = m0;
  for (int i = lane + 32; i < parts; i += 32) top = fmaxf(top, stats[record(i) * 2 * kNC]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.0f;
  bool there_all = true;
  for (int i = lane; i < parts; i += 32) {
    const float mi = i < 32 ? m0 : stats[record(i) * 2 * kNC], li = i < 32 ? l0 : stats[record(i) * 2 * kNC + kNC];
    // -1: the row saw nothing in this part, whose outputs are no numbers.  A weight of zero is one
    // like any other: outputs that are not finite reach the row through it.
    const float w = li == 0.0f ? -1.0f : exp2f(mi - top);
    weight[warp][i] = w;
    there_all = there_all && !(li < 0.0f);
    sum += li == 0.0f ? 0.0f : w * li;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (!__all_sync(0xffffffffu, there_all)) {  // a wait gave up (both maps' warps see it): the row stays as it was
    if (kMaps == 2) __syncthreads();
    return;
  }
  if (lane == 0) p.lse[row * kMaps + m] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
  __syncwarp();
  float y[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) y[k] = 0.0f;
  for (int base = 0;;) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float w = base + i < parts ? weight[warp][base + i] : -1.0f;
#pragma unroll
      for (int k = 0; k < kV; ++k) y[k] += w < 0.0f ? 0.0f : w * ahead[i][k];
    }
    base += kAhead;
    if (base >= parts) break;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (base + i < parts) load_row<kV>(outs + record(base + i) * kNC * kDv, ahead[i]);
  }
  const float by = (sum == 0.0f ? 0.0f : 1.0f / sum) * (m == 1 ? lam : 1.0f);
#pragma unroll
  for (int k = 0; k < kV; ++k) y[k] *= by;
  if (kMaps == 2) {
    if (m == 1)
#pragma unroll
      for (int k = 0; k < kV; ++k) other[slot][lane * kV + k] = y[k];
    __syncthreads();
    if (m == 1) return;
#pragma unroll
    for (int k = 0; k < kV; ++k) y[k] -= other[slot][lane * kV + k];
    if (p.gain != nullptr) {
      float sq = 0.0f;
#pragma unroll
      for (int k = 0; k < kV; ++k) sq += y[k] * y[k];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      const float norm = rsqrtf(sq * (1.0f / kDv) + p.eps);
#pragma unroll
      for (int k = 0; k < kV; ++k) y[k] = sum == 0.0f ? 0.0f : y[k] * norm * gain[k];
    }
  }
  uint32_t packed[kV / 2];
#pragma unroll
  for (int k = 0; k < kV; k += 2) packed[k / 2] = pack_bf16(y[k], y[k + 1]);
  __nv_bfloat16 *dst = p.out + row * kDv + lane * kV;
  if constexpr (kV == 2) *reinterpret_cast<uint32_t *>(dst) = packed[0];
  else if constexpr (kV == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(packed[0], packed[1]);
  else *reinterpret_cast<uint4 *>(dst) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
}

template <int kW, int kMaps, int kNC>
mla_status launch_as(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const Params &p, int grid, bool merge,
                     cudaStream_t stream) {
  using C = Config<kW, kMaps, kNC>;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (!((ready.load(std::memory_order_relaxed) >> (dev & 63)) & 1u)) {
    e = cudaFuncSetAttribute(grouped_kernel<kW, kMaps, kNC>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "grouped kernel shared memory");
    ready.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  }
  e = launch_pdl(grouped_kernel<kW, kMaps, kNC>, dim3(grid), dim3(C::kThreads), C::kSmem, stream, q, k, v, p);
  if (e != cudaSuccess) return cuda_fail(e, "grouped launch");
  if (!merge) return MLA_OK;
  const int rows = p.rows_per_block * p.heads_per_block;  // of a unit
  e = launch_pdl(grouped_merge<kW, kMaps, kNC>, dim3(grid, (rows + kMergeRows - 1) / kMergeRows), dim3(32 * kMergeRows * kMaps), 0, stream, p);
  return e == cudaSuccess ? MLA_OK : cuda_fail(e, "grouped merge launch");
}

}  // namespace grouped
}  // namespace mla
