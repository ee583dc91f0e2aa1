// mla_tables.cu -- block tables and slot map of a step, made on the device
// from the requests' lengths (mla_update_block_tables).
//
// A request that grows takes blocks from the front of the ring of free ids,
// one that shrinks (drafts taken back, finished) returns its last blocks to
// the ring's end, both in request order, so request b's place is a prefix sum
// over the requests before it.  Blocks returned in a call are not dealt in it:
// what is read ([head, head + count) of the ring, table entries below held_b
// and those being returned) and what is written (ring places from head +
// count on, table entries from held_b on) never overlap, so one launch
// without a grid barrier does it all: every CTA makes the prefix sums of all
// requests for itself in shared memory (one pass over the lengths and
// qo_indptr, 12 B bytes from L2) and then takes its share of the dealt blocks,
// the returned blocks and the new tokens, reading the lengths of their
// requests once more.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kTabThreads = 256;
constexpr int kMaxTableReqs = 16384;  // two prefix sums and the row offsets in shared memory: 192 KB

struct TabParams {
  mla_table_args a;
  int32_t *lens_out;  // or null
  int *err;
  uint32_t bs_mul;  // n / block_size = (n + umulhi(n, bs_mul)) >> bs_shift, 0 <= n < 2^31
  int bs_shift;
};

// With l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, (n + floor(m n / 2^32)) >> l is n / d for
// every n < 2^32 (Granlund and Montgomery, division by invariant integers); n < 2^31 keeps the sum in 32
// bits.  A division by a variable is 20 instructions or more, and a prompt's look-ups are bound by the ALU
// (884,000 tokens: 10.3 -> 8.2 us).
__device__ __forceinline__ int div_bs(const TabParams &p, int n) {
  return static_cast<int>((static_cast<uint32_t>(n) + __umulhi(static_cast<uint32_t>(n), p.bs_mul)) >> p.bs_shift);
}

__device__ __forceinline__ void tab_error(const TabParams &p, int code) { atomicCAS(p.err, 0, code); }

// Blocks that hold the shard's part of the first n tokens, within the table.
__device__ __forceinline__ int blocks_of(const TabParams &p, int n, bool &over) {
  const mla_table_args &a = p.a;
  const int loc = n <= 0 ? 0 : a.world_size == 1 ? n : il_count(n, a.world_size, a.rank, a.interleave);
  const int full = div_bs(p, loc), blocks = full + (full * a.block_size != loc);
  over = blocks > a.block_table_stride;
  return over ? a.block_table_stride : blocks;
}

// (head + k) % C for head < C, k <= C.
__device__ __forceinline__ int ring_place(int head, int k, int C) {
  const uint32_t at = static_cast<uint32_t>(head) + static_cast<uint32_t>(k);
  return static_cast<int>(at >= static_cast<uint32_t>(C) ? at - static_cast<uint32_t>(C) : at);
}

// The last b with sums[b] <= k, for k < sums[B].
__device__ __forceinline__ int owner_of(const int *sums, int B, int k) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= k) lo = mid;
    else hi = mid;
  }
  return lo;
}

// kPer: new tokens' rows that a thread takes in a row.
template <int kPer>
__global__ void __launch_bounds__(kTabThreads) update_tables_kernel(const TabParams p) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ int sums[];  // off [B + 1], roff [B + 1], qo_indptr [B + 1]
  __shared__ int warp_tot[2][kTabThreads / 32];
  const mla_table_args &a = p.a;
  const int B = a.num_reqs, T = a.num_rows, C = a.num_blocks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first_cta = blockIdx.x == 0;
  int *off = sums, *roff = sums + B + 1, *ind = sums + 2 * (B + 1);
  bool bad_ind = false;
  int carry_t = 0, carry_r = 0;
  for (int b0 = 0; b0 < B; b0 += kTabThreads) {
    const int b = b0 + tid;
    int take = 0, rel = 0;
    if (b < B) {
      bool over_h, over_n;
      const int prev = a.prev_lens[b], L = a.seq_lens[b];
      const int held = blocks_of(p, prev, over_h), need = blocks_of(p, L, over_n);
      take = max(need - held, 0);
      rel = max(held - need, 0);
      const int q0 = a.qo_indptr[b], q1 = a.qo_indptr[b + 1];
      ind[b] = q0;
      bad_ind |= q1 < q0;
      if (first_cta) {
        if (over_h || over_n) tab_error(p, MLA_DEV_LEN_BOUND);
        if (prev < 0 || L < 0 || (q1 >= q0 && q1 - q0 > L)) tab_error(p, MLA_DEV_BAD_QLEN);
      }
    }
    int st = take, sr = rel;  // inclusive scans over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int yt = __shfl_up_sync(0xffffffffu, st, o), yr = __shfl_up_sync(0xffffffffu, sr, o);
      if (lane >= o) {
        st += yt;
        sr += yr;
      }
    }
    if (lane == 31) {
      warp_tot[0][warp] = st;
      warp_tot[1][warp] = sr;
    }
    __syncthreads();
    int bt = carry_t, br = carry_r;
#pragma unroll
    for (int w = 0; w < kTabThreads / 32; ++w) {
      if (w < warp) {
        bt += warp_tot[0][w];
        br += warp_tot[1][w];
      }
      carry_t += warp_tot[0][w];
      carry_r += warp_tot[1][w];
    }
    if (b < B) {
      off[b] = bt + st - take;
      roff[b] = br + sr - rel;
    }
    __syncthreads();
  }
  const int n_take = carry_t, n_rel = carry_r;
  const int total = a.qo_indptr[B];
  if (tid == 0) ind[B] = total;
  bad_ind |= a.qo_indptr[0] != 0 || total < 0 || total > T;
  bad_ind = __syncthreads_or(bad_ind) != 0;
  const int head = a.ring_in[0], count = a.ring_in[1];
  const int dealt = min(n_take, count);
  // (free blocks and returned ones are different blocks of the pool, so the
  // ring places written stay clear of those read)
  const bool bad_ring = head < 0 || head >= C || count < 0 || static_cast<int64_t>(count) + n_rel > C;
  const bool good = !bad_ind && !bad_ring;
  if (first_cta && tid == 0) {
    if (bad_ind) tab_error(p, MLA_DEV_BAD_INDPTR);
    if (bad_ring) tab_error(p, MLA_DEV_BAD_FREE_RING);
    if (good && n_take > count) tab_error(p, MLA_DEV_NO_FREE_BLOCK);
    a.ring_out[0] = good ? ring_place(head, dealt, C) : head;
    a.ring_out[1] = good ? count - dealt + n_rel : count;
  }
  const int first = blockIdx.x * kTabThreads + tid, step = gridDim.x * kTabThreads;
  if (p.lens_out != nullptr)
    for (int b = first; b < B; b += step) p.lens_out[b] = good ? max(a.seq_lens[b], 0) : a.prev_lens[b];
  if (!good) {
    for (int r = first; r < T; r += step) a.slot_map[r] = -1;
    return;
  }
  // dealt block k (-1: the ring had too few, or holds a bad id)
  auto dealt_id = [&](int k) {
    if (k >= count) return -1;
    const int id = a.free_ring[ring_place(head, k, C)];
    if (id >= 0 && id < C) return id;
    tab_error(p, MLA_DEV_BAD_BLOCK_ID);
    return -1;
  };
  bool over;
  for (int k = first; k < n_take; k += step) {
    const int b = owner_of(off, B, k);
    const int e = blocks_of(p, a.prev_lens[b], over) + k - off[b];
    a.block_table[static_cast<int64_t>(b) * a.block_table_stride + e] = dealt_id(k);
  }
  for (int k = first; k < n_rel; k += step) {
    const int b = owner_of(roff, B, k);
    const int e = blocks_of(p, a.seq_lens[b], over) + k - roff[b];
    int id = a.block_table[static_cast<int64_t>(b) * a.block_table_stride + e];
    if (id < 0 || id >= C) {
      tab_error(p, MLA_DEV_BAD_BLOCK_ID);
      id = -1;
    }
    a.free_ring[ring_place(head, count + k, C)] = id;
  }
  // A thread's rows: one search for their request and one look-up per block
  // they touch.
  const int I = a.interleave, W = a.world_size, cycle = I * W, bs = a.block_size;  // (I W fits: checked)
  const bool whole = kPer == 4 && (reinterpret_cast<uintptr_t>(a.slot_map) & 15) == 0;
  for (int64_t r0 = kPer * static_cast<int64_t>(first); r0 < T; r0 += kPer * static_cast<int64_t>(step)) {
    int slot[kPer], q1 = -1, shift = 0, held = 0, need = 0, b = 0, e = -1, in = 0, id = -1;
    bool fits = false, next = false;  // next: the row before was local position e * bs + in - 1
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = static_cast<int>(r0) + i;
      slot[i] = -1;
      if (r0 + i >= total) continue;
      if (r >= q1) {  // the first row, or the next request's
        b = owner_of(ind, B, r);
        const int L = a.seq_lens[b];
        q1 = ind[b + 1];
        fits = q1 - ind[b] <= L;
        shift = L - q1;  // row r is position r + shift
        held = blocks_of(p, a.prev_lens[b], over);
        need = blocks_of(p, L, over);
        next = false;
      }
      const int g = r + shift;
      int j = g;  // in the shard's index space
      if (W > 1) {
        const int turn = g / cycle, in_turn = g - turn * cycle, owner = in_turn / I;
        if (owner != a.rank) continue;
        j = turn * I + in_turn - owner * I;
      }
      if (!fits) continue;
      int at = e;
      if (next) {
        if (in == bs) {
          in = 0;
          ++at;
        }
      } else {
        at = div_bs(p, j);
        in = j - at * bs;
        e = -1;
      }
      if (at != e) {
        e = at;
        id = -1;
        if (e < held) {
          id = a.block_table[static_cast<int64_t>(b) * a.block_table_stride + e];
          if (id < 0 || id >= C) {
            tab_error(p, MLA_DEV_BAD_BLOCK_ID);
            id = -1;
          }
        } else if (e < need) {
          id = dealt_id(off[b] + e - held);
        }
      }
      if (id >= 0) slot[i] = id * bs + in;
      ++in;
      next = true;  // a shard's tokens follow one another in its own index space
    }
    if (whole && r0 + kPer <= T) {
      *reinterpret_cast<int4 *>(a.slot_map + r0) =
          make_int4(slot[0], slot[kPer > 1 ? 1 : 0], slot[kPer > 2 ? 2 : 0], slot[kPer - 1]);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (r0 + i < T) a.slot_map[r0 + i] = slot[i];
    }
  }
}

std::atomic<bool> g_tab_attr[2][64];

mla_status update_block_tables(const mla_table_args *a, int32_t *lens_out, mla_stream_t stream) {
  if (a == nullptr || a->num_reqs < 0 || a->num_rows < 0 || a->world_size < 1 || a->rank < 0 ||
      a->rank >= a->world_size || a->interleave < 1 ||
      static_cast<int64_t>(a->interleave) * a->world_size > INT32_MAX) {
    set_error("mla_update_block_tables: bad sizes, rank or interleave");
    return MLA_ERR_INVALID_ARG;
  }
  if (a->block_size < 1 || a->num_blocks < 1 || a->block_table_stride < 1 ||
      static_cast<int64_t>(a->num_blocks) * a->block_size > INT32_MAX) {
    set_error("mla_update_block_tables: block_size=%d num_blocks=%d block_table_stride=%d (cache rows must fit int32)",
              a->block_size, a->num_blocks, a->block_table_stride);
    return MLA_ERR_INVALID_ARG;
  }
  if (static_cast<int64_t>(a->num_reqs) * a->block_table_stride > INT32_MAX) {
    set_error("mla_update_block_tables: %d x %d table entries overflow int32", a->num_reqs, a->block_table_stride);
    return MLA_ERR_INVALID_ARG;
  }
  if (a->qo_indptr == nullptr || a->free_ring == nullptr || a->ring_in == nullptr || a->ring_out == nullptr ||
      (a->ring_out < a->ring_in + 2 && a->ring_in < a->ring_out + 2) || (a->num_rows > 0 && a->slot_map == nullptr) ||
      (a->num_reqs > 0 && (a->prev_lens == nullptr || a->seq_lens == nullptr || a->block_table == nullptr))) {
    set_error("mla_update_block_tables: null pointer, or ring_out overlaps ring_in");
    return MLA_ERR_INVALID_ARG;
  }
  const auto overlaps = [&](const int32_t *lens) { return lens_out < lens + a->num_reqs && lens < lens_out + a->num_reqs; };
  if (lens_out != nullptr && a->num_reqs > 0 && (overlaps(a->prev_lens) || overlaps(a->seq_lens))) {
    set_error("mla_update_block_tables_lens: lens_out overlaps prev_lens or seq_lens");
    return MLA_ERR_INVALID_ARG;
  }
  if (a->num_reqs > kMaxTableReqs) {
    set_error("mla_update_block_tables: %d requests above the supported %d", a->num_reqs, kMaxTableReqs);
    return MLA_ERR_UNSUPPORTED;
  }
  int *err = device_error_word();
  if (err == nullptr) return MLA_ERR_CUDA;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  // A step's few tokens one per thread, so that their look-ups run side by side
  // (27,600 tokens on a shard: 5.1 us against 9.4 with four); a prompt's many four per
  // thread (884,000 tokens: 10.9 -> 8.2 us).
  const bool many = a->num_rows > 65536;
  auto kern = many ? update_tables_kernel<4> : update_tables_kernel<1>;
  if (!g_tab_attr[many][dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             3 * (kMaxTableReqs + 1) * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(tables smem)");
    g_tab_attr[many][dev].store(true, std::memory_order_relaxed);
  }
  int shift = 0;
  while ((1LL << shift) < a->block_size) ++shift;
  const uint64_t rest = (1ULL << shift) - static_cast<uint64_t>(a->block_size);
  const TabParams p{*a, lens_out, err, static_cast<uint32_t>((rest << 32) / static_cast<uint64_t>(a->block_size) + 1), shift};
  // up to 8 CTAs per SM's worth; tables without tokens still get a thread per request
  const int rows = many ? a->num_rows / 4 + 1 : a->num_rows;
  const int items = rows > a->num_reqs ? rows : a->num_reqs;
  int grid = (items + kTabThreads - 1) / kTabThreads;
  grid = grid < 1 ? 1 : (grid > 1216 ? 1216 : grid);
  e = launch_pdl(kern, dim3(grid), dim3(kTabThreads), 3 * (static_cast<size_t>(a->num_reqs) + 1) * sizeof(int),
                 reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? MLA_OK : cuda_fail(e, "update_block_tables launch");
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_update_block_tables(const mla_table_args *a, mla_stream_t stream) {
  return update_block_tables(a, nullptr, stream);
}

extern "C" mla_status mla_update_block_tables_lens(const mla_table_args *a, int32_t *lens_out, mla_stream_t stream) {
  if (lens_out == nullptr && (a == nullptr || a->num_reqs != 0)) {
    set_error("mla_update_block_tables_lens: null lens_out");
    return MLA_ERR_INVALID_ARG;
  }
  return update_block_tables(a, lens_out, stream);
}
