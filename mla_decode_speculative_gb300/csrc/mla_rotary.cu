// mla_rotary.cu -- rotary positions of one or several axes on queries and keys
// (mla_rotary), and the same with the keys and values written to the rows of a
// paged K/V cache (mla_rotary_write).
//
// The angle of pair i in a row is positions[axes[i]][row] * turns[i] modulo
// 2^64, in units of 2^-64 turns: an integer product that wraps around is the
// exact remainder, so a position of a million costs no accuracy (in float32
// 10^6 * 0.9 is off by 0.03 radians).  Its top 32 bits, as a signed fraction
// in [-1/2, 1/2) turns, go to sincospi in float32.
//
// Memory bound: 4 bytes per value for about 3 operations, once the sines are
// shared: a block takes whole rows (or part of one), makes their sines once in
// shared memory, and its threads go over the rows' heads in stretches of 16
// bytes, so that what a warp touches is one run of memory.  A thread's first
// stretch is read before the sines are made.  Values that are only copied (v,
// the dims past R) are blocks of the same launch.  Large calls live from many
// blocks an SM (8 of 32 registers a thread, four stretches a thread), small ones
// from short code (4 blocks): 16,400 rows of 32 + 8 heads of 128 and 8 of values
// 63.3 us against 75.0 with 4 blocks an SM, 620 rows of the same 3.7 against 5.2
// with 8; four stretches in flight a thread, at two blocks an SM, 91 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kJobs = 5;        // q, k rotated; q, k behind the rotated part; v
constexpr int kEach = 4;        // items a thread has at most
constexpr int kTable = 1024;    // sines of a block

// Division by a fixed d: n / d for n * d < 2^32 (n < rows x width <= 1024 by the
// width, n < width by the lanes, which the host checks).
struct Div {
  uint32_t d, m;
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return m == 0 ? n : __umulhi(n, m); }
};
Div divisor(uint32_t d) { return Div{d, d == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + d - 1) / d)}; }

// Items of a job: (row, head, lane), lane fastest; `width` items a row.
struct Job {
  const uint16_t *src;
  uint16_t *dst;
  int64_t src_row, src_head, dst_row, dst_head;
  int first_block;  // of the launch
  int width;        // heads x lanes
  int rows;         // rows a block
  int blocks_row;   // blocks a row (1 if rows > 1)
  int items;        // items a block
  Div by_width, by_lanes;
  int vec;          // pairs (rotation) or values (copy) of an item: 8, 4 or 1
  int rotate, by_slot;
};

struct Params {
  Job job[kJobs];
  int num_jobs, num_rows, num_axes, pairs;
  const int32_t *positions;
  int64_t axis_stride;
  const int64_t *turns;
  const int32_t *axes;
  const int32_t *slot_map;
  int64_t num_cache_rows;
  int *err;
};

template <int V>
struct Vec;
template <>
struct Vec<8> { using T = uint4; };
template <>
struct Vec<4> { using T = uint2; };
template <>
struct Vec<1> { using T = uint16_t; };

template <int V>
union Pack {
  typename Vec<V>::T raw;
  __nv_bfloat16 h[V];
};

// Cache row of row r's keys and values, -1 for none.
__device__ __forceinline__ int64_t slot_of(const Params &p, int r) {
  const int s = p.slot_map[r];
  if (s < -1 || s >= p.num_cache_rows) {
    atomicCAS(p.err, 0, MLA_DEV_BAD_BLOCK_ID);
    return -1;
  }
  return s;
}

// cos, sin of pair q of row r.
__device__ __forceinline__ float2 turn_of(const Params &p, int r, int q) {
  int a = p.axes != nullptr ? p.axes[q] : 0;
  if (a < 0 || a >= p.num_axes) {
    atomicCAS(p.err, 0, MLA_DEV_BAD_AXIS);
    a = 0;
  }
  const int64_t pos = p.positions[a * p.axis_stride + r];
  const uint64_t turn = static_cast<uint64_t>(pos) * static_cast<uint64_t>(p.turns[q]);
  float2 cs;
  sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &cs.y, &cs.x);
  return cs;
}

// A block's rows [r0, r1), items [at, end) of them (counted from row r0).
// kV: values a load has; rotation: an item is kV pairs, read as two of them.
template <int kV, bool kRotate, bool kNeighbours>
__device__ __forceinline__ void run_job(const Params &p, const Job &j, int r0, int r1, uint32_t at, uint32_t end, float *table) {
  using T = typename Vec<kV>::T;
  const int lanes = static_cast<int>(j.by_lanes.d);
  Pack<kV> a, b;
  int row = 0, at_a = 0, at_b = 0, lane = 0;
  int64_t to = -1;
  auto load = [&](uint32_t i) {
    to = -1;
    if (i >= end) return;
    const uint32_t r = j.rows > 1 ? j.by_width(i) : 0, hl = i - r * j.width, h = j.by_lanes(hl);
    row = static_cast<int>(r);
    lane = static_cast<int>(hl - h * lanes);
    at_a = (kRotate && kNeighbours ? 2 * kV : kV) * lane;
    at_b = kNeighbours ? at_a + kV : p.pairs + at_a;
    const uint16_t *x = j.src + (r0 + static_cast<int64_t>(r)) * j.src_row + h * j.src_head;
    a.raw = *reinterpret_cast<const T *>(x + at_a);
    if (kRotate) b.raw = *reinterpret_cast<const T *>(x + at_b);
    const int64_t out = j.by_slot ? slot_of(p, r0 + row) : r0 + row;
    to = out < 0 ? -1 : out * j.dst_row + h * j.dst_head;
  };
  uint32_t i = at + threadIdx.x;
  load(i);
  if (kRotate) {
    // row by row: the (cos, sin) of pairs kV l + 2 k, + 1 of lane l at 16-byte place k * lanes + l
    for (int u = threadIdx.x; u < (r1 - r0) * p.pairs; u += kThreads) {
      const int r = u / p.pairs, q = u - r * p.pairs;
      const int place = kV == 1 ? q : ((q % kV) / 2 * lanes + q / kV) * 2 + q % 2;
      reinterpret_cast<float2 *>(table)[r * p.pairs + place] = turn_of(p, r0 + r, q);
    }
    __syncthreads();
  }
  while (true) {
    if (to >= 0) {
      uint16_t *y = j.dst + to;
      if (kRotate) {
        const float *t = table + 2 * row * p.pairs;
        Pack<kV> oa, ob;
        auto turn = [&](int e, float c, float s) {  // pair e of the item
          // neighbours: values 2e, 2e + 1 of the run a, b
          Pack<kV> &pu = kNeighbours && 2 * e >= kV ? b : a, &pv = kNeighbours && 2 * e + 1 < kV ? a : b;
          Pack<kV> &ou = kNeighbours && 2 * e >= kV ? ob : oa, &ov = kNeighbours && 2 * e + 1 < kV ? oa : ob;
          const int iu = kNeighbours ? (2 * e) % kV : e, iv = kNeighbours ? (2 * e + 1) % kV : e;
          const float u = __bfloat162float(pu.h[iu]), v = __bfloat162float(pv.h[iv]);
          ou.h[iu] = __float2bfloat16_rn(u * c - v * s);
          ov.h[iv] = __float2bfloat16_rn(v * c + u * s);
        };
        if constexpr (kV == 1) {
          const float2 cs = reinterpret_cast<const float2 *>(t)[lane];
          turn(0, cs.x, cs.y);
        } else {
#pragma unroll
          for (int e = 0; e < kV; e += 2) {
            const float4 cs = reinterpret_cast<const float4 *>(t)[e / 2 * lanes + lane];
            turn(e, cs.x, cs.y);
            turn(e + 1, cs.z, cs.w);
          }
        }
        *reinterpret_cast<T *>(y + at_a) = oa.raw;
        *reinterpret_cast<T *>(y + at_b) = ob.raw;
      } else {
        *reinterpret_cast<T *>(y + at_a) = a.raw;
      }
    }
    i += kThreads;
    if (i >= end) break;
    load(i);
  }
}

template <bool kNeighbours, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) rotary_kernel(const __grid_constant__ Params p) {
  __shared__ alignas(16) float table[2 * kTable];
  grid_dep_wait();
  grid_dep_launch();
  int n = 0;
  while (n + 1 < p.num_jobs && static_cast<int>(blockIdx.x) >= p.job[n + 1].first_block) ++n;
  const Job &j = p.job[n];
  const int block = static_cast<int>(blockIdx.x) - j.first_block;
  const int group = block / j.blocks_row, part = block - group * j.blocks_row;
  const int r0 = group * j.rows, r1 = min(r0 + j.rows, p.num_rows);
  const uint32_t at = static_cast<uint32_t>(part) * j.items;
  const uint32_t end = min(at + j.items, static_cast<uint32_t>(r1 - r0) * j.width);
  if (j.rotate) {
    if (j.vec == 8) run_job<8, true, kNeighbours>(p, j, r0, r1, at, end, table);
    else if (j.vec == 4) run_job<4, true, kNeighbours>(p, j, r0, r1, at, end, table);
    else run_job<1, true, kNeighbours>(p, j, r0, r1, at, end, table);
  } else {
    if (j.vec == 8) run_job<8, false, false>(p, j, r0, r1, at, end, table);
    else if (j.vec == 4) run_job<4, false, false>(p, j, r0, r1, at, end, table);
    else run_job<1, false, false>(p, j, r0, r1, at, end, table);
  }
}

// Largest of 8, 4, 1 values that every address of the tensor (from value `at`
// on) and `run` are a multiple of.
int vector_of(const mla_heads &t, int at, int run) {
  for (int v : {8, 4}) {
    const uintptr_t bytes = static_cast<uintptr_t>(v) * 2;
    if (run % v == 0 && at % v == 0 && reinterpret_cast<uintptr_t>(t.src) % bytes == 0 &&
        reinterpret_cast<uintptr_t>(t.dst) % bytes == 0 && t.src_row % v == 0 && t.src_head % v == 0 &&
        t.dst_row % v == 0 && t.dst_head % v == 0)
      return v;
  }
  return 1;
}

mla_status check_heads(const char *what, const char *name, const mla_heads &t, int min_dim, int rows) {
  if (t.heads < 0 || t.heads > 65536) {
    set_error("%s: %s has %d heads", what, name, t.heads);
    return MLA_ERR_INVALID_ARG;
  }
  if (t.heads == 0) return MLA_OK;
  if (t.dim < min_dim || t.dim > 65536) {
    set_error("%s: %s has %d values a head (%d to 65536)", what, name, t.dim, min_dim);
    return MLA_ERR_INVALID_ARG;
  }
  if (rows > 0 && (t.src == nullptr || t.dst == nullptr)) {
    set_error("%s: null %s", what, name);
    return MLA_ERR_INVALID_ARG;
  }
  if (t.src_row < 0 || t.src_head < 0 || t.dst_row < 0 || (t.heads > 1 && t.dst_head < t.dim)) {
    set_error("%s: strides of %s (heads of %d values %lld elements apart)", what, name, t.dim,
              (long long)t.dst_head);
    return MLA_ERR_INVALID_ARG;
  }
  if (rows > 0 && t.src == t.dst && (t.src_row != t.dst_row || t.src_head != t.dst_head)) {
    set_error("%s: %s in place with two different strides", what, name);
    return MLA_ERR_INVALID_ARG;
  }
  if (reinterpret_cast<uintptr_t>(t.src) % 2 != 0 || reinterpret_cast<uintptr_t>(t.dst) % 2 != 0) {
    set_error("%s: %s is not 2-byte aligned", what, name);
    return MLA_ERR_INVALID_ARG;
  }
  return MLA_OK;
}

// One launch over the tensors that are there.
mla_status run(const mla_rotary_args *a, bool write, mla_stream_t stream) {
  const char *what = write ? "mla_rotary_write" : "mla_rotary";
  if (a == nullptr) {
    set_error("%s: null argument struct", what);
    return MLA_ERR_INVALID_ARG;
  }
  if (a->num_rows < 0 || a->num_axes < 1 || a->axis_stride < 0) {
    set_error("%s: num_rows %d, num_axes %d, axis_stride %lld", what, a->num_rows, a->num_axes,
              (long long)a->axis_stride);
    return MLA_ERR_INVALID_ARG;
  }
  if (a->rot_dim < 2 || a->rot_dim > 512 || a->rot_dim % 2 != 0) {
    set_error("%s: rot_dim %d unsupported (even, 2 to 512)", what, a->rot_dim);
    return MLA_ERR_UNSUPPORTED;
  }
  const mla_heads *tensors[3] = {&a->q, &a->k, &a->v};
  const char *names[3] = {"q", "k", "v"};
  for (int i = 0; i < 3; ++i) {
    const mla_status st = check_heads(what, names[i], *tensors[i], i < 2 ? a->rot_dim : 1, a->num_rows);
    if (st != MLA_OK) return st;
  }
  if (!write && a->v.heads != 0) {
    set_error("mla_rotary: v is for mla_rotary_write");
    return MLA_ERR_INVALID_ARG;
  }
  if (write && (a->k.heads == 0 || a->v.heads == 0)) {
    set_error("mla_rotary_write: k and v are needed");
    return MLA_ERR_INVALID_ARG;
  }
  if (write && (a->num_cache_rows < 1 || a->num_cache_rows > INT32_MAX)) {
    set_error("mla_rotary_write: %lld cache rows", (long long)a->num_cache_rows);
    return MLA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 3; ++i) {  // rows of an output must not meet
    const mla_heads &t = *tensors[i];
    const int64_t rows = write && i > 0 ? a->num_cache_rows : a->num_rows;
    const int64_t span = t.heads > 0 ? (t.heads - 1) * t.dst_head + t.dim : 0;
    if (t.heads > 0 && rows > 1 && (t.dst_row < t.dim || (t.dst_row < span && t.dst_head < t.dst_row * rows))) {
      set_error("%s: rows of %s's output are %lld elements apart, a row spans %lld", what, names[i],
                (long long)t.dst_row, (long long)span);
      return MLA_ERR_INVALID_ARG;
    }
  }
  if (a->num_rows > 0 && (a->positions == nullptr || a->turns == nullptr || (write && a->slot_map == nullptr))) {
    set_error("%s: null positions, turns or slot_map", what);
    return MLA_ERR_INVALID_ARG;
  }
  if (a->num_rows == 0 || (a->q.heads == 0 && a->k.heads == 0)) return MLA_OK;
  int *err = device_error_word();
  if (err == nullptr) return MLA_ERR_CUDA;

  Params p{};
  p.num_rows = a->num_rows;
  p.num_axes = a->num_axes;
  p.pairs = a->rot_dim / 2;
  p.positions = a->positions;
  p.axis_stride = a->axis_stride;
  p.turns = a->turns;
  p.axes = a->axes;
  p.slot_map = a->slot_map;
  p.num_cache_rows = a->num_cache_rows;
  p.err = err;
  int64_t blocks = 0;
  bool too_wide = false, large = false;
  auto add = [&](const mla_heads &t, bool rotate, int at, int dim, bool by_slot) {
    Job &j = p.job[p.num_jobs++];
    j.src = static_cast<const uint16_t *>(t.src) + at;
    j.dst = static_cast<uint16_t *>(t.dst) + at;
    j.src_row = t.src_row;
    j.src_head = t.src_head;
    j.dst_row = t.dst_row;
    j.dst_head = t.dst_head;
    j.rotate = rotate;
    j.by_slot = by_slot;
    j.vec = vector_of(t, at, rotate ? p.pairs : dim);
    const int lanes = (rotate ? p.pairs : dim) / j.vec;
    if (static_cast<int64_t>(t.heads) * lanes * lanes > UINT32_MAX) too_wide = true;
    j.width = t.heads * lanes;
    // Items a thread has: four, or what leaves the GPU two blocks an SM.
    const int64_t share = static_cast<int64_t>(p.num_rows) * j.width / (304 * kThreads);
    large |= share >= kEach;
    const int each = static_cast<int>(share < 1 ? 1 : (share > kEach ? kEach : share)) * kThreads;
    const int most = rotate ? kTable / p.pairs : 65536;
    j.rows = each / j.width < 1 ? 1 : (each / j.width > most ? most : each / j.width);
    j.blocks_row = j.rows > 1 || j.width <= each ? 1 : (j.width + each - 1) / each;
    j.items = j.blocks_row > 1 ? each : j.rows * j.width;
    j.by_width = divisor(static_cast<uint32_t>(j.width));
    j.by_lanes = divisor(static_cast<uint32_t>(lanes));
    j.first_block = static_cast<int>(blocks);
    blocks += static_cast<int64_t>((p.num_rows + j.rows - 1) / j.rows) * j.blocks_row;
  };
  const int R = a->rot_dim;
  if (a->q.heads > 0) add(a->q, true, 0, R, false);
  if (a->k.heads > 0) add(a->k, true, 0, R, write);
  if (a->v.heads > 0) add(a->v, false, 0, a->v.dim, true);
  if (a->q.heads > 0 && a->q.dim > R && a->q.src != a->q.dst) add(a->q, false, R, a->q.dim - R, false);
  if (a->k.heads > 0 && a->k.dim > R && a->k.src != a->k.dst) add(a->k, false, R, a->k.dim - R, write);
  if (too_wide || blocks > INT32_MAX) {
    set_error("%s: %d rows of these heads are too many", what, a->num_rows);
    return MLA_ERR_UNSUPPORTED;
  }
  const dim3 grid(static_cast<unsigned>(blocks)), threads(kThreads);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      a->neighbours ? (large ? launch_pdl(rotary_kernel<true, 8>, grid, threads, 0, s, p) : launch_pdl(rotary_kernel<true, 4>, grid, threads, 0, s, p))
                    : (large ? launch_pdl(rotary_kernel<false, 8>, grid, threads, 0, s, p) : launch_pdl(rotary_kernel<false, 4>, grid, threads, 0, s, p));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e, "rotary launch");
}

}  // namespace
}  // namespace mla

extern "C" {

mla_status mla_rotary(const mla_rotary_args *a, mla_stream_t stream) { return mla::run(a, false, stream); }

mla_status mla_rotary_write(const mla_rotary_args *a, mla_stream_t stream) { return mla::run(a, true, stream); }

}  // extern "C"
