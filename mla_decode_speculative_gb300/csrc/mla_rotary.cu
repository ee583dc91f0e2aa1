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
// shared: a block takes up to 1,024 items of 16 bytes of each half (or of two
// neighbouring runs), from wherever they begin in a row, makes the sines of the rows
// that it meets once in shared memory, and goes over them, so that what a warp touches
// is one run of memory.  (Times here are calls in a graph on one state: no host time, and
// what is smaller than L2 stays there.)  q and k are one sequence of heads, with the same
// sines: one head of each, 39,000 rows of 128, 11.3 us against 26.6 apart.  A thread's first item
// is read before the sines are made.  Values that are only copied (v, the dims past R
// of a small call) are blocks of the same launch.  Large calls live from many blocks an
// SM (8 of 32 registers a thread, four items a thread), small ones from short code
// (4 blocks): 16,400 rows of 32 + 8 heads of 128 and 8 of values 63.9 us (6.5 TB/s,
// 0.97 of a copy's rate; the same on fresh inputs) against 74 with 4 blocks an SM, 620
// rows of the same 3.9 against 5.1 with 8; 9,001 rows of 64 + 1 heads of 64 26.6 (5.6
// TB/s; on fresh inputs 28.1), 128 rows of 16 + 1 2.2.  With one head the sines bound it: 160,000 rows of 96 37 us, half a
// copy's rate.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kJobs = 5;        // q, k rotated (as one, if their alignment is); q, k behind the rotated part; v
constexpr int kEach = 4;        // items a thread has at most
constexpr int kTable = 1024;    // sines of a block
constexpr double kL2Bytes = 129e6;

// Division by a fixed d: n / d for n * d < 2^32 (n < 2 x kThreads x kEach by a
// width up to that, n < width by the lanes, which the host checks).
struct Div {
  uint32_t d, m;
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return m == 0 ? n : __umulhi(n, m); }
};
Div divisor(uint32_t d) { return Div{d, d == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + d - 1) / d)}; }

// A tensor of a job.
struct Side {
  const uint16_t *src;
  uint16_t *dst;
  int64_t src_row, src_head, dst_row, dst_head;
  int by_slot;
};

// Items of a job: (row, head, lane), lane fastest; `width` items a row.
struct Job {
  Side side[2];
  int split;        // heads of the first tensor: the second's follow
  int first_block;  // of the launch
  int width;        // heads x lanes
  int rot;          // lanes that rotate; those behind them copy the values past R
  int items;        // items a block: of whole rows, or from anywhere in a row on
  uint64_t width_m; // 2^64 / width, rounded up
  Div by_width, by_lanes;
  int vec;          // pairs (rotation) or values (copy) of an item: 8, 4 or 1
  int rotate;
};

struct Params {
  Job job[kJobs];
  int num_jobs, num_rows, num_axes, pairs;
  Div by_pairs;
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

// Items [at, end) of a block, counted from row r0.  kV: values a load has; rotation:
// an item is kV pairs, read as two of them.
template <int kV, bool kRotate, bool kNeighbours, bool kTail>
__device__ __forceinline__ void run_job(const Params &p, const Job &j, int r0, uint32_t at, uint32_t end, float *table) {
  using T = typename Vec<kV>::T;
  const int lanes = static_cast<int>(j.by_lanes.d);
  const int rot = kTail ? j.rot : lanes;
  const uint32_t width = j.width;
  // row of an item; of a wide row there are two parts at most
  auto row_of = [&](uint32_t i) { return width > kThreads * kEach ? (i >= width ? 1u : 0u) : j.by_width(i); };
  Pack<kV> a, b;
  int row = 0, at_a = 0, at_b = 0, lane = 0;
  uint16_t *y = nullptr;  // where its head goes
  auto load = [&](uint32_t i) {
    y = nullptr;
    if (i >= end) return;
    const uint32_t r = row_of(i), hl = i - r * width;
    uint32_t h = j.by_lanes(hl);
    row = static_cast<int>(r);
    lane = static_cast<int>(hl - h * lanes);
    at_a = (kRotate && kNeighbours ? 2 * kV : kV) * lane;
    at_b = kNeighbours ? at_a + kV : p.pairs + at_a;
    if (kTail && lane >= rot) at_b = (at_a = 2 * (p.pairs + kV * (lane - rot))) + kV;
    const bool second = kRotate && h >= static_cast<uint32_t>(j.split);
    if (second) h -= j.split;
    const Side &t = j.side[second];
    const uint16_t *x = t.src + (r0 + static_cast<int64_t>(r)) * t.src_row + h * t.src_head;
    a.raw = *reinterpret_cast<const T *>(x + at_a);
    if (kRotate) b.raw = *reinterpret_cast<const T *>(x + at_b);
    const int64_t out = t.by_slot ? slot_of(p, r0 + row) : r0 + row;
    if (out >= 0) y = t.dst + out * t.dst_row + h * t.dst_head;
  };
  uint32_t i = at + threadIdx.x;
  load(i);
  if (kRotate) {
    // row by row: the (cos, sin) of pairs kV l + 2 k, + 1 of lane l at 16-byte place k * rot + l;
    // a thread keeps its pair
    const int abreast = static_cast<int>(p.by_pairs(kThreads)), r_first = static_cast<int>(p.by_pairs(threadIdx.x));
    const int q = static_cast<int>(threadIdx.x) - r_first * p.pairs, rows = static_cast<int>(row_of(end - 1)) + 1;
    if (r_first < abreast && r_first < rows) {
      int axis = p.axes != nullptr ? p.axes[q] : 0;
      if (axis < 0 || axis >= p.num_axes) {
        atomicCAS(p.err, 0, MLA_DEV_BAD_AXIS);
        axis = 0;
      }
      const uint64_t per = static_cast<uint64_t>(p.turns[q]);
      const int32_t *pos = p.positions + axis * p.axis_stride + r0;
      const int place = kV == 1 ? q : ((q % kV) / 2 * rot + q / kV) * 2 + q % 2;
      float2 *to = reinterpret_cast<float2 *>(table) + place;
      for (int r = r_first; r < rows; r += abreast) {
        const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos[r])) * per;
        float2 cs;
        sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &cs.y, &cs.x);
        to[r * p.pairs] = cs;
      }
    }
    __syncthreads();
  }
  while (true) {
    if (y != nullptr) {
      if (kTail && lane >= rot) {
        *reinterpret_cast<T *>(y + at_a) = a.raw;
        *reinterpret_cast<T *>(y + at_b) = b.raw;
      } else if (kRotate) {
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
            const float4 cs = reinterpret_cast<const float4 *>(t)[e / 2 * rot + lane];
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

template <bool kNeighbours, int kBlocks, bool kTail>
__global__ void __launch_bounds__(kThreads, kBlocks) rotary_kernel(const __grid_constant__ Params p) {
  __shared__ alignas(16) float table[2 * kTable];
  grid_dep_wait();
  grid_dep_launch();
  int n = 0;
  while (n + 1 < p.num_jobs && static_cast<int>(blockIdx.x) >= p.job[n + 1].first_block) ++n;
  const Job &j = p.job[n];
  const uint64_t first = static_cast<uint64_t>(blockIdx.x - j.first_block) * j.items;
  const int r0 = static_cast<int>(j.width_m == 0 ? first : __umul64hi(first, j.width_m));
  const uint32_t at = static_cast<uint32_t>(first - static_cast<uint64_t>(r0) * j.width);
  const uint32_t end = static_cast<uint32_t>(min(static_cast<uint64_t>(at + j.items), static_cast<uint64_t>(p.num_rows - r0) * j.width));
  if (j.rotate) {
    if (j.vec == 8) run_job<8, true, kNeighbours, kTail>(p, j, r0, at, end, table);
    else if (j.vec == 4) run_job<4, true, kNeighbours, kTail>(p, j, r0, at, end, table);
    else run_job<1, true, kNeighbours, kTail>(p, j, r0, at, end, table);
  } else {
    if (j.vec == 8) run_job<8, false, false, false>(p, j, r0, at, end, table);
    else if (j.vec == 4) run_job<4, false, false, false>(p, j, r0, at, end, table);
    else run_job<1, false, false, false>(p, j, r0, at, end, table);
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

  Params p{};
  p.num_rows = a->num_rows;
  p.num_axes = a->num_axes;
  p.pairs = a->rot_dim / 2;
  p.by_pairs = divisor(static_cast<uint32_t>(p.pairs));
  p.positions = a->positions;
  p.axis_stride = a->axis_stride;
  p.turns = a->turns;
  p.axes = a->axes;
  p.slot_map = a->slot_map;
  p.num_cache_rows = a->num_cache_rows;
  int64_t blocks = 0;
  int64_t all = 0;
  const int64_t wave = 4 * 152 * kThreads;  // threads of four blocks an SM
  bool too_wide = false;
  // Values at .. at + dim - 1 of the heads of t, and of `also` behind them; rotated
  // with `tail` more that are copied.
  auto add = [&](const mla_heads &t, bool by_slot, bool rotate, int at, int dim, int tail, const mla_heads *also, bool also_by_slot) {
    Job &j = p.job[p.num_jobs++];
    auto side = [&](const mla_heads &x, bool slots) {
      return Side{static_cast<const uint16_t *>(x.src) + at, static_cast<uint16_t *>(x.dst) + at, x.src_row, x.src_head, x.dst_row, x.dst_head, slots};
    };
    j.side[0] = side(t, by_slot);
    j.side[1] = also != nullptr ? side(*also, also_by_slot) : j.side[0];
    j.split = t.heads;
    const int heads = t.heads + (also != nullptr ? also->heads : 0);
    j.rotate = rotate;
    j.vec = vector_of(t, at, rotate ? p.pairs : dim);
    j.rot = (rotate ? p.pairs : dim) / j.vec;
    const int lanes = j.rot + tail / (2 * j.vec);
    if (static_cast<int64_t>(heads) * lanes * lanes > UINT32_MAX) {  // heads x lanes may not be an int
      too_wide = true;
      return;
    }
    j.width = heads * lanes;
    // Items a thread has: what the GPU takes at once with four blocks an SM, up to four
    // (with two an SM: 7,000 rows of 9 heads of 80 and 3 of values 10.1 -> 6.9 us).
    const int64_t total = static_cast<int64_t>(p.num_rows) * j.width;
    const int each = static_cast<int>(std::min<int64_t>((total + wave - 1) / wave, kEach)) * kThreads;
    all += total;
    const int most = kTable / p.pairs;  // rows whose sines fit
    const int whole = std::min(most, each / j.width);
    j.items = each;
    if (rotate && whole > 0) {
      // whole rows leave threads idle, stretches from anywhere make a row's sines twice: items for
      // the rounds of threads, a round of items at twice a round of sines
      auto rounds = [&](int n, int of) { return (n + of - 1) / of; };
      const int abreast = kThreads / p.pairs, met = (each + j.width - 2) / j.width + 1;
      const int64_t cost_whole = 2 * rounds(whole * j.width, kThreads) + rounds(whole, abreast) + 1;
      const int64_t cost_any = 2 * (each / kThreads) + rounds(met, abreast) + 1;
      if (met > most || whole * j.width * cost_any >= each * cost_whole) j.items = whole * j.width;
    }
    j.width_m = j.width == 1 ? 0 : UINT64_MAX / j.width + 1;
    if (static_cast<double>(total) * j.width > 9e18) too_wide = true;
    j.by_width = divisor(static_cast<uint32_t>(j.width));
    j.by_lanes = divisor(static_cast<uint32_t>(lanes));
    j.first_block = static_cast<int>(blocks);
    blocks += (total + j.items - 1) / j.items;
  };
  // The values past R (of which an item takes as many as it would rotate) go with the
  // rotated ones where they divide so and the call is larger than L2: copied by other
  // blocks, their sectors come and go twice (7,900 rows of 72 heads of 80 turned by 40,
  // 8 of values: 110 us against 56.6; 6,500 rows of 48 + 8: 20.7 against 22.3).
  const int R = a->rot_dim, vq = vector_of(a->q, 0, p.pairs), vk = vector_of(a->k, 0, p.pairs);
  auto values = [](const mla_heads &t) { return static_cast<double>(t.heads) * t.dim; };
  const bool join = 4.0 * a->num_rows * (values(a->q) + values(a->k) + values(a->v)) > kL2Bytes;
  auto fits = [&](int heads, int vec, int tail) {
    const int64_t lanes = p.pairs / vec + tail / (2 * vec);
    return tail % (2 * vec) == 0 && heads * lanes * lanes <= UINT32_MAX;
  };
  auto behind = [&](const mla_heads &t) { return t.heads > 0 && t.src != t.dst ? t.dim - R : 0; };
  const int tail_q = behind(a->q), tail_k = behind(a->k);
  int with_q = join && fits(a->q.heads, vq, tail_q) ? tail_q : 0, with_k = join && fits(a->k.heads, vk, tail_k) ? tail_k : 0;
  const bool both = a->q.heads > 0 && a->k.heads > 0 && vq == vk;
  if (both && with_q == 0) with_k = 0;
  if (both && with_q == with_k && fits(a->q.heads + a->k.heads, vq, with_q)) {
    add(a->q, false, true, 0, R, with_q, &a->k, write);
  } else {
    if (a->q.heads > 0) add(a->q, false, true, 0, R, with_q, nullptr, false);
    if (a->k.heads > 0) add(a->k, write, true, 0, R, with_k, nullptr, false);
  }
  if (a->v.heads > 0) add(a->v, true, false, 0, a->v.dim, 0, nullptr, false);
  if (tail_q > with_q) add(a->q, false, false, R, tail_q, 0, nullptr, false);
  if (tail_k > with_k) add(a->k, write, false, R, tail_k, 0, nullptr, false);
  if (too_wide || blocks > INT32_MAX) {
    set_error("%s: %d rows of these heads are too many", what, a->num_rows);
    return MLA_ERR_UNSUPPORTED;
  }
  int *err = device_error_word();
  if (err == nullptr) return MLA_ERR_CUDA;
  p.err = err;
  const bool large = all > 7 * wave, neighbours = a->neighbours != 0;
  const bool tail = with_q + with_k > 0;
  const dim3 grid(static_cast<unsigned>(blocks)), threads(kThreads);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const auto kernel = tail ? (neighbours ? rotary_kernel<true, 8, true> : rotary_kernel<false, 8, true>)
                      : large ? (neighbours ? rotary_kernel<true, 8, false> : rotary_kernel<false, 8, false>)
                              : (neighbours ? rotary_kernel<true, 4, false> : rotary_kernel<false, 4, false>);
  const cudaError_t e = launch_pdl(kernel, grid, threads, 0, s, p);
  return e == cudaSuccess ? MLA_OK : cuda_fail(e, "rotary launch");
}

}  // namespace
}  // namespace mla

extern "C" {

mla_status mla_rotary(const mla_rotary_args *a, mla_stream_t stream) { return mla::run(a, false, stream); }

mla_status mla_rotary_write(const mla_rotary_args *a, mla_stream_t stream) { return mla::run(a, true, stream); }

}  // extern "C"
