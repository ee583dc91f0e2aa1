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
// Memory bound: 4 bytes per value for about 3 operations.  A thread holds the
// sines of up to 8 pairs of one row and goes over several heads with them (16
// bytes a load, two loads a head, four heads in flight), so a row's sines are
// made once per 8 heads.  Values that are only copied (v, the dims past R) are
// blocks of the same launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kJobs = 5;       // q, k rotated; q, k behind the rotated part; v
constexpr int kMaxHeads = 16;  // heads a thread takes at most

struct Job {
  const uint16_t *src;
  uint16_t *dst;
  int64_t src_row, src_head, dst_row, dst_head;
  int first_block;  // of the launch
  int heads, chunks, per;  // heads in all; head chunks; heads a chunk
  int lanes;        // threads a row
  int units;        // copies: vectors a head
  int vec;          // pairs (rotation) or values (copy) a thread takes at once: 8, 4 or 1
  int rotate, by_slot;
};

struct Params {
  Job job[kJobs];
  int num_jobs, num_rows, num_axes, pairs, neighbours;
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

// Pairs V * lane .. V * lane + V - 1 of the heads h0 .. h1 - 1 of one row.
template <int V>
__device__ __forceinline__ void rotate_heads(const Params &p, const Job &j, int r, int lane, int h0, int h1) {
  int64_t out_row = r;
  if (j.by_slot) {
    out_row = slot_of(p, r);
    if (out_row < 0) return;
  }
  const int i0 = V * lane;
  float c[V], s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    int a = p.axes != nullptr ? p.axes[i0 + i] : 0;
    if (a < 0 || a >= p.num_axes) {
      atomicCAS(p.err, 0, MLA_DEV_BAD_AXIS);
      a = 0;
    }
    const int64_t pos = p.positions[a * p.axis_stride + r];
    const uint64_t turn = static_cast<uint64_t>(pos) * static_cast<uint64_t>(p.turns[i0 + i]);
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s[i], &c[i]);
  }
  // the pairs' values: a run in each half of the rotated part, or one run of twice the length
  const int at_a = p.neighbours ? 2 * i0 : i0;
  const int at_b = p.neighbours ? 2 * i0 + V : p.pairs + i0;
  const uint16_t *src = j.src + static_cast<int64_t>(r) * j.src_row;
  uint16_t *dst = j.dst + out_row * j.dst_row;
  using T = typename Vec<V>::T;
  for (int h = h0; h < h1; h += 4) {
    Pack<V> a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (h + k < h1) {
        const uint16_t *x = src + (h + k) * j.src_head;
        a[k].raw = *reinterpret_cast<const T *>(x + at_a);
        b[k].raw = *reinterpret_cast<const T *>(x + at_b);
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (h + k < h1) {
        Pack<V> oa, ob;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float x, y;
          if (p.neighbours) {  // values 2i, 2i + 1 of the run a, b
            x = __bfloat162float(2 * i < V ? a[k].h[(2 * i) % V] : b[k].h[(2 * i) % V]);
            y = __bfloat162float(2 * i + 1 < V ? a[k].h[(2 * i + 1) % V] : b[k].h[(2 * i + 1) % V]);
          } else {
            x = __bfloat162float(a[k].h[i]);
            y = __bfloat162float(b[k].h[i]);
          }
          const __nv_bfloat16 u = __float2bfloat16_rn(x * c[i] - y * s[i]);
          const __nv_bfloat16 w = __float2bfloat16_rn(y * c[i] + x * s[i]);
          if (p.neighbours) {
            (2 * i < V ? oa : ob).h[(2 * i) % V] = u;
            (2 * i + 1 < V ? oa : ob).h[(2 * i + 1) % V] = w;
          } else {
            oa.h[i] = u;
            ob.h[i] = w;
          }
        }
        uint16_t *y = dst + (h + k) * j.dst_head;
        *reinterpret_cast<T *>(y + at_a) = oa.raw;
        *reinterpret_cast<T *>(y + at_b) = ob.raw;
      }
  }
}

// Vectors lane, lane + lanes, .. of the heads h0 .. h1 - 1 of one row, copied.
template <int V>
__device__ __forceinline__ void copy_heads(const Params &p, const Job &j, int r, int lane, int h0, int h1) {
  int64_t out_row = r;
  if (j.by_slot) {
    out_row = slot_of(p, r);
    if (out_row < 0) return;
  }
  const uint16_t *src = j.src + static_cast<int64_t>(r) * j.src_row;
  uint16_t *dst = j.dst + out_row * j.dst_row;
  using T = typename Vec<V>::T;
  for (int u = lane; u < j.units; u += j.lanes)
    for (int h = h0; h < h1; h += 4) {
      T x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (h + k < h1) x[k] = *reinterpret_cast<const T *>(src + (h + k) * j.src_head + u * V);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (h + k < h1) *reinterpret_cast<T *>(dst + (h + k) * j.dst_head + u * V) = x[k];
    }
}

__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Params p) {
  grid_dep_wait();
  grid_dep_launch();
  int n = 0;
  while (n + 1 < p.num_jobs && static_cast<int>(blockIdx.x) >= p.job[n + 1].first_block) ++n;
  const Job &j = p.job[n];
  const int block = static_cast<int>(blockIdx.x) - j.first_block;
  const int rows = kThreads / j.lanes;  // rows a block
  const int r = (block / j.chunks) * rows + static_cast<int>(threadIdx.x) / j.lanes;
  const int lane = static_cast<int>(threadIdx.x) % j.lanes;
  if (static_cast<int>(threadIdx.x) >= rows * j.lanes || r >= p.num_rows) return;
  const int h0 = (block % j.chunks) * j.per, h1 = min(h0 + j.per, j.heads);
  if (j.rotate) {
    if (j.vec == 8) rotate_heads<8>(p, j, r, lane, h0, h1);
    else if (j.vec == 4) rotate_heads<4>(p, j, r, lane, h0, h1);
    else rotate_heads<1>(p, j, r, lane, h0, h1);
  } else {
    if (j.vec == 8) copy_heads<8>(p, j, r, lane, h0, h1);
    else if (j.vec == 4) copy_heads<4>(p, j, r, lane, h0, h1);
    else copy_heads<1>(p, j, r, lane, h0, h1);
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
  p.neighbours = a->neighbours != 0;
  p.positions = a->positions;
  p.axis_stride = a->axis_stride;
  p.turns = a->turns;
  p.axes = a->axes;
  p.slot_map = a->slot_map;
  p.num_cache_rows = a->num_cache_rows;
  p.err = err;
  int64_t blocks = 0;
  auto add = [&](const mla_heads &t, bool rotate, int at, int dim, bool by_slot) {
    Job &j = p.job[p.num_jobs++];
    j.src = static_cast<const uint16_t *>(t.src) + at;
    j.dst = static_cast<uint16_t *>(t.dst) + at;
    j.src_row = t.src_row;
    j.src_head = t.src_head;
    j.dst_row = t.dst_row;
    j.dst_head = t.dst_head;
    j.heads = t.heads;
    j.rotate = rotate;
    j.by_slot = by_slot;
    j.vec = vector_of(t, at, rotate ? p.pairs : dim);
    j.units = (rotate ? p.pairs : dim) / j.vec;
    j.lanes = j.units < kThreads ? j.units : kThreads;
    // Heads a thread goes over with its sines: as many as leave the GPU 152 x
    // 1024 threads, 16 at most.
    const int64_t threads = static_cast<int64_t>(p.num_rows) * j.lanes * t.heads;
    int64_t per = threads / (152 * 1024);
    per = per < 1 ? 1 : (per > kMaxHeads ? kMaxHeads : per);
    j.per = static_cast<int>(per);
    j.chunks = (t.heads + j.per - 1) / j.per;
    j.first_block = static_cast<int>(blocks);
    const int rows = kThreads / j.lanes;
    blocks += static_cast<int64_t>((p.num_rows + rows - 1) / rows) * j.chunks;
  };
  const int R = a->rot_dim;
  if (a->q.heads > 0) add(a->q, true, 0, R, false);
  if (a->k.heads > 0) add(a->k, true, 0, R, write);
  if (a->v.heads > 0) add(a->v, false, 0, a->v.dim, true);
  if (a->q.heads > 0 && a->q.dim > R && a->q.src != a->q.dst) add(a->q, false, R, a->q.dim - R, false);
  if (a->k.heads > 0 && a->k.dim > R && a->k.src != a->k.dst) add(a->k, false, R, a->k.dim - R, write);
  if (blocks > INT32_MAX) {
    set_error("%s: %d rows need too many blocks", what, a->num_rows);
    return MLA_ERR_UNSUPPORTED;
  }
  const cudaError_t e = launch_pdl(rotary_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0,
                                   reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? MLA_OK : cuda_fail(e, "rotary launch");
}

}  // namespace
}  // namespace mla

extern "C" {

mla_status mla_rotary(const mla_rotary_args *a, mla_stream_t stream) { return mla::run(a, false, stream); }

mla_status mla_rotary_write(const mla_rotary_args *a, mla_stream_t stream) { return mla::run(a, true, stream); }

}  // extern "C"
