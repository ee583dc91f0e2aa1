// mla_grouped.cuh -- the decode kernel of grouped-query and differential
// attention over a paged K/V cache, and what its launcher and its merge share
// with it.
//
// For every row (verify row t of request b, query head of group g) and map m:
//   s_j = sm_scale <q_m, k_{j,g,m}>,  o_m = sum_j softmax(s)_j v_{j,g}
// with an online base-2 softmax.  The rows of a group (heads x verify rows) go
// over their keys and values together, so the cache is read once per group:
// 2 R flops a byte for R rows, so memory decides (282 flops a byte is the ridge)
// as long as the tensor cores, the softmax and the copies run beside each other.
//
//  * Tile = 128 tokens of one group.  Both products have the tokens' or the
//    values' dims as M and the rows as N, which costs the same tensor time for
//    16 rows as for 64:
//        S_m^T[128 tokens, NR rows] = K_m[128, D] . Q_m[NR, D]^T     (K-major A and B)
//        O^T[dims, NC columns]     += V^T[dims, 128] . P^T[128, NC]  (MN-major A and B)
//    NC = maps x NR columns: the two maps of the differential form are columns
//    of one product with the values, which are thus read once.
//  * A token's row of a group is W chunks of 64 values (W = 1, 2, 4: the keys of
//    all maps, or the values).  The tensor map splits cache rows in eights, so
//    that one box brings a page as [8 rows][chunk][row][128 bytes]: the same
//    uniform strides for pages of 8 as of 128, read by both products as they
//    are (128-byte swizzle).
//  * Copies in the order of use, K(t + 1) before V(t), through a ring of slots
//    of at most 32 KB (two chunks); the stream of tiles runs on from part to part.
//  * Balanced split: a unit (request, group, row block) is kOverhead positions
//    and then its tiles; the positions of all units, laid end to end, are cut
//    into equal chunks, one per SM.  A chunk holds at most two units that it
//    does not hold whole: its first and its last.  So there are two partial
//    records per SM, whatever the batch, and the merge looks at 152 chunks.
//  * Softmax: a thread has one token and all columns of its group of warps (32
//    at most), in registers.  The reference maximum moves only when a score
//    passes it by 2^8; sums are float32 per thread and column.
//  * Tokens that no row sees are neither loaded (whole pages) nor multiplied:
//    their values in shared memory are set to zero.  A token that some rows see
//    is looked at, and a value in it that is not finite is zeroed too and
//    spoils the rows that see it (0 x NaN would spoil the others).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_internal.h"
#include "mla_ptx.cuh"

namespace mla {
namespace grouped {

constexpr int kTile = 128;
constexpr int kMaxReqs = 1024;    // requests of one launch (tabulated in shared memory)
constexpr int kOverhead = 2;      // positions a unit counts beside its tiles
constexpr int kMinChunk = 6;      // positions a chunk has at least
constexpr int kMaxCtas = 152;

// A unit that is cut across chunks: written by the chunk with its first tile.
struct Meta {
  int b, g, rb;
  int last;  // chunk of its last tile; -1: no such unit starts in this chunk
};

struct Params {
  const int32_t *qo_indptr, *row_len, *subpage_table;
  __nv_bfloat16 *out;
  float *lse;
  const float *lambda, *gain;
  float eps;
  float *part_o;     // [chunk][2][NC][64 W] unnormalised outputs
  float *part_stat;  // [chunk][2][2][NC] base-2 maxima, sums
  Meta *meta;        // [chunk]
  int *err;
  long long wait_budget, drain_budget;
  float scale_log2;
  int num_reqs, num_rows, num_heads, num_kv_heads, group, max_qlen, max_len, window;
  int subpage_stride, page_size, page_groups;  // page_groups: num_cache_rows / 8
  int rows_per_block;   // verify rows of a row block (group <= NR)
  int heads_per_block;  // query heads of a row block: group, or NR if group > NR
  int head_blocks;      // row blocks a verify row's group is cut into (1 if group <= NR)
};

// Rows of a row block: column c of block rb is verify row t, head h of the group.
__device__ __forceinline__ bool column_row(const Params &p, int rb, int c, int qlen, int &t, int &h) {
  if (p.head_blocks == 1) {
    const int dt = c / p.group;
    t = rb * p.rows_per_block + dt;
    h = c - dt * p.group;
    return dt < p.rows_per_block && t < qlen;
  }
  t = rb / p.head_blocks;
  h = (rb - t * p.head_blocks) * p.heads_per_block + c;
  return c < p.heads_per_block && h < p.group && t < qlen;
}

__device__ __forceinline__ int blocks_of(const Params &p, int qlen) {
  return p.head_blocks == 1 ? (qlen + p.rows_per_block - 1) / p.rows_per_block : qlen * p.head_blocks;
}

template <int kW, int kMaps, int kNC>
struct Config {
  static constexpr int kNR = kNC / kMaps;           // columns of a map
  static constexpr int kCW = kW < 2 ? kW : 2;       // chunks of a slot
  static constexpr int kNS = kW / kCW;              // slots of a key tile, and of a value tile
  static constexpr int kDv = 64 * kW;
  static constexpr int kSlotBytes = kTile * 128 * kCW;
  static constexpr int kQChunkBytes = kNR * 128;
  static constexpr int kQBytes = kW * kQChunkBytes;
  static constexpr int kQBufs = kQBytes <= 8192 ? 2 : 1;
  static constexpr int kPBytes = kTile * 128;
  static constexpr int kMiscBytes = 16 * 1024;
  static constexpr int kFit = (232448 - 1024 - kMiscBytes - kQBufs * kQBytes - 2 * kPBytes) / kSlotBytes;
  static constexpr int kSlots = kFit > 10 ? 10 : kFit;
  static constexpr int kGroups = kNC > 32 ? 2 : 1;  // groups of four softmax warps
  static constexpr int kCols = kNC / kGroups;       // columns of a group
  static constexpr int kSoftmaxWarps = 4 * kGroups;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 2);
  static constexpr int kBlocks = kW < 2 ? 1 : kW / 2;  // blocks of O^T: 128 dims each (64 if W = 1)
  static constexpr int kTmemUsed = kNC * (2 + kBlocks);
  static constexpr int kTmemCols = kTmemUsed <= 64 ? 64 : (kTmemUsed <= 128 ? 128 : 256);
  static constexpr int kOffQ = kSlots * kSlotBytes;
  static constexpr int kOffP = kOffQ + kQBufs * kQBytes;
  static constexpr int kOffMisc = kOffP + 2 * kPBytes;
  static constexpr int kSmem = kOffMisc + kMiscBytes + 1024;
  static_assert(kTmemUsed <= 256 && kNR % 16 == 0 && kSlots >= 2 * kNS + (kNS == 1) && kSmem <= 232448, "configuration");
};

struct Misc {
  uint64_t full[10], empty[10];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2], fin;
  uint32_t tmem_base;
  int abort, stop[2];
  int start[kMaxReqs + 1];                // positions before request b
  int lo[kMaxReqs], hi[kMaxReqs];         // tokens that some row of the request sees: lo .. hi - 1
  alignas(16) float red[2][4][32];        // [group of warps][warp][column]
  alignas(16) float stat_m[64], stat_l[64];
  int col_lo[64], col_hi[64];             // what a column of this part sees
  unsigned bad[2];                        // columns of a group that see a value that is not finite
};
static_assert(sizeof(Misc) <= 16 * 1024, "misc");

// A part: the tiles a .. b - 1 (of n) of a unit that lie in this chunk.
struct Part {
  int b, g, rb;   // request, group, row block
  int q0, qlen;
  int lo, hi;     // tokens the request sees
  int tile0;      // tile index of the unit's tile 0
  int a, e, n;
  int start;      // position of the unit
};

// Goes over a chunk's parts in order; every role has its own.
struct Walk {
  const Params &p;
  const Misc &m;
  int pos_a, pos_e;     // the chunk
  int b, j, per, units;
  __device__ Walk(const Params &p_, const Misc &m_, int a, int e) : p(p_), m(m_), pos_a(a), pos_e(e) {
    int lo = 0, hi = p.num_reqs;  // first request that ends behind a
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (m.start[mid + 1] <= a) lo = mid + 1;
      else hi = mid;
    }
    b = lo;
    j = 0;
    enter();
    if (b < p.num_reqs && a < e) j = (a - m.start[b]) / per;
  }
  __device__ void enter() {
    while (b < p.num_reqs && m.start[b + 1] == m.start[b]) ++b;
    if (b >= p.num_reqs) return;
    const int tiles = m.hi[b] > m.lo[b] ? (m.hi[b] + kTile - 1) / kTile - m.lo[b] / kTile : 0;
    per = tiles + kOverhead;
    units = (m.start[b + 1] - m.start[b]) / per;
  }
  __device__ bool next(Part &o) {
    while (b < p.num_reqs) {
      const int s = m.start[b] + j * per;
      if (s >= pos_e) return false;
      const int first = s + kOverhead, n = per - kOverhead;
      o.a = max(pos_a, first) - first;
      o.e = min(pos_e, first + n) - first;
      const bool take = n > 0 ? o.e > o.a : s >= pos_a;
      if (take) {
        o.b = b;
        o.q0 = p.qo_indptr[b];
        o.qlen = p.qo_indptr[b + 1] - o.q0;
        const int blocks = units / p.num_kv_heads;
        o.g = j / blocks;
        o.rb = j - o.g * blocks;
        o.lo = m.lo[b];
        o.hi = m.hi[b];
        o.tile0 = o.lo / kTile;
        o.n = n;
        o.start = s;
        if (n == 0) o.a = o.e = 0;
      }
      if (++j == units) {
        ++b;
        j = 0;
        enter();
      }
      if (take) return true;
    }
    return false;
  }
};

// Slot of the i-th slot use of the stream, and the parity of its full barrier.
// K(t) is use kNS (2 t - 1) (0 for t = 0), V(t) use kNS (2 t + 2); the use that
// would be K of the tile behind the last stays empty.
template <class C>
__device__ __forceinline__ uint32_t k_use(uint32_t t) { return t == 0 ? 0 : C::kNS * (2 * t - 1); }
template <class C>
__device__ __forceinline__ uint32_t v_use(uint32_t t) { return C::kNS * (2 * t + 2); }

__device__ __forceinline__ void record_error(int *err, int code) { atomicCAS(err, 0, code); }

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
  return r;
}

// One 5-D box -> shared memory, completing on an mbarrier.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, uint32_t bar, int x, int y, int z, int u, int w,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(w), "r"(bar), "l"(policy)
      : "memory");
}

// 32 TMEM lanes x N columns per warp (thread i <- lane base + i), N = 16 or 32.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[N]) {
  uint32_t r[N];
  if constexpr (N == 32) {
    tmem_ld32(addr, r);
  } else {
    static_assert(N == 16, "16 or 32 columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t addr, const float (&v)[N]) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __float_as_uint(v[i]);
  if constexpr (N == 32) {
    tmem_st32(addr, r);
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
  }
}

// Warp transpose-reduce: v[k] is this lane's value of column k; returns the
// max (or sum) over the 32 lanes of column lane % N.  Clobbers v.
template <bool kMax, int N>
__device__ __forceinline__ float reduce_columns(float (&v)[N], int lane) {
#pragma unroll
  for (int off = N / 2; off >= 1; off >>= 1) {
    const bool upper = (lane & off) != 0;
#pragma unroll
    for (int k = 0; k < off; ++k) {
      const float send = upper ? v[k] : v[k + off];
      const float keep = upper ? v[k + off] : v[k];
      const float recv = __shfl_xor_sync(0xffffffffu, send, off);
      v[k] = kMax ? fmaxf(keep, recv) : keep + recv;
    }
  }
  if constexpr (N == 16) {
    const float recv = __shfl_xor_sync(0xffffffffu, v[0], 16);
    v[0] = kMax ? fmaxf(v[0], recv) : v[0] + recv;
  }
  return v[0];
}

constexpr float kLowest = -3.402823466e38f;  // a column that has seen nothing yet
constexpr float kLag = 8.0f;                 // powers of two that a score may pass the reference maximum by
constexpr float kLn2 = 0.69314718055994530942f;

template <int kW, int kMaps, int kNC>
__global__ void __launch_bounds__(Config<kW, kMaps, kNC>::kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  using C = Config<kW, kMaps, kNC>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc &misc = *reinterpret_cast<Misc *>(smem + C::kOffMisc);
  const uint32_t s_slots = smem_u32(smem), s_q = s_slots + C::kOffQ, s_p = s_slots + C::kOffP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kProducer = C::kSoftmaxWarps, kMma = C::kSoftmaxWarps + 1;
  constexpr int kSoftmaxThreads = 32 * C::kSoftmaxWarps;

  if (warp == kMma) {
    tmem_alloc(smem_u32(&misc.tmem_base), C::kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_u32(&misc.full[i]), 1);
      mbar_init(smem_u32(&misc.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&misc.q_full[i]), 1);
      mbar_init(smem_u32(&misc.q_empty[i]), 1);
      mbar_init(smem_u32(&misc.s_full[i]), 1);
      mbar_init(smem_u32(&misc.p_full[i]), C::kSoftmaxWarps);
      mbar_init(smem_u32(&misc.o_done[i]), 1);
      misc.bad[i] = 0;
    }
    mbar_init(smem_u32(&misc.fin), 1);
    misc.abort = 0;
    fence_mbar_init();
  }
  // Query rows that no copy fills (a group that does not divide the columns) stay zero.
  for (int i = threadIdx.x; i < C::kQBufs * C::kQBytes / 16; i += C::kThreads)
    st_shared_v4(s_q + 16 * i, 0, 0, 0, 0);
  fence_proxy_async_smem();
  grid_dep_wait();
  grid_dep_launch();

  // What each request's rows see, and its positions.
  for (int b = threadIdx.x; b < p.num_reqs; b += C::kThreads) {
    const int q0 = p.qo_indptr[b], q1 = p.qo_indptr[b + 1];
    int lo = INT32_MAX, hi = 0, cost = 0;
    if (q0 < 0 || q1 < q0 || q1 > p.num_rows || q1 - q0 > p.max_qlen) {
      record_error(p.err, MLA_DEV_BAD_INDPTR);
    } else if (q1 > q0) {
      for (int r0 = q0; r0 < q1; r0 += 4) {
        int n[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) n[k] = r0 + k < q1 ? p.row_len[r0 + k] : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (n[k] > p.max_len) {
            record_error(p.err, MLA_DEV_LEN_BOUND);
            n[k] = p.max_len;
          }
          if (n[k] > 0) {
            hi = max(hi, n[k]);
            lo = min(lo, p.window > 0 ? max(0, n[k] - p.window) : 0);
          }
        }
      }
      const int tiles = hi > 0 ? (hi + kTile - 1) / kTile - lo / kTile : 0;
      cost = blocks_of(p, q1 - q0) * p.num_kv_heads * (tiles + kOverhead);
    }
    misc.lo[b] = hi > 0 ? lo : 0;
    misc.hi[b] = hi;
    misc.start[b + 1] = cost;
  }
  if (threadIdx.x == 0) misc.start[0] = 0;
  __syncthreads();
  if (warp == 0) {  // running sum, in place
    int carry = 0;
    for (int base = 0; base < p.num_reqs; base += 32) {
      const int b = base + lane;
      int x = b < p.num_reqs ? misc.start[b + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < p.num_reqs) misc.start[b + 1] = carry + x;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = misc.tmem_base;
  const int total = misc.start[p.num_reqs];
  const int chunks = max(1, min(static_cast<int>(gridDim.x), total / kMinChunk));
  const int chunk = static_cast<int>(blockIdx.x);
  auto cut = [&](int c) { return static_cast<int>(static_cast<long long>(c) * total / chunks); };
  auto chunk_of = [&](int x) { return static_cast<int>((static_cast<long long>(x + 1) * chunks - 1) / total); };
  const int pos_a = chunk < chunks ? cut(chunk) : total, pos_e = chunk < chunks ? cut(chunk + 1) : total;
  volatile int *abort_flag = &misc.abort;
  const long long budget = p.wait_budget;
  auto fail = [&]() {
    *abort_flag = 1;
    record_error(p.err, MLA_DEV_WAIT_TIMEOUT);
  };
  auto full_bar = [&](uint32_t use) { return smem_u32(&misc.full[use % C::kSlots]); };
  auto full_par = [&](uint32_t use) { return (use / C::kSlots) & 1u; };

  if (warp == kProducer) {
    // ======================================================== copies
    const uint64_t pol_kv = l2_policy_evict_first();
    const uint64_t pol_q = l2_policy_evict_last();
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int P = p.page_size, pages = kTile / P;
    const uint32_t page_bytes = static_cast<uint32_t>(P) * 128 * C::kCW;
    uint32_t armed = 0, armed_par = 0;  // the latest copy into each slot
    uint32_t q_armed = 0, q_armed_par = 0;
    bool ok = true;
    // page of this lane: row group, or the one behind the cache (zeros) if the id is bad
    auto load_tile = [&](const CUtensorMap *tm, uint32_t use, int group8, bool mine, int n_pages, int g) {
#pragma unroll
      for (int s = 0; s < C::kNS; ++s) {
        const uint32_t u = use + s, slot = u % C::kSlots;
        if (lane == 0 && ok && !mbar_wait(smem_u32(&misc.empty[slot]), ((u / C::kSlots) & 1u) ^ 1u, abort_flag, budget)) {
          fail();
          ok = false;
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) return;
        const uint32_t bar = smem_u32(&misc.full[slot]);
        if (lane == 0) mbar_arrive_expect_tx(bar, page_bytes * n_pages);
        __syncwarp();
        if (mine)
          tma_load_5d(s_slots + slot * C::kSlotBytes + lane * page_bytes, tm, bar, 0, 0, s * C::kCW, group8, g, pol_kv);
        armed |= 1u << slot;
        armed_par = (armed_par & ~(1u << slot)) | (((u / C::kSlots) & 1u) << slot);
      }
    };
    Walk walk(p, misc, pos_a, pos_e);
    Part w;
    uint32_t t = 0, kq = 0;
    int prev_group = 0, prev_pages = 0, prev_g = 0;
    bool prev_mine = false;
    while (ok && walk.next(w)) {
      if (w.e == w.a) continue;
      const int32_t *ids = p.subpage_table + static_cast<int64_t>(w.b) * p.subpage_stride;
      const int page_lo = w.lo / P, page_hi = (w.hi + P - 1) / P;
      auto id_of = [&](int tile) {
        const int page = (w.tile0 + tile) * pages + lane;
        return lane < pages && page >= page_lo && page < page_hi ? ids[page] : -1;
      };
      int id = id_of(w.a);
      // Q of this part
      const uint32_t qb = kq % C::kQBufs;
      if (lane == 0 && !mbar_wait(smem_u32(&misc.q_empty[qb]), ((kq / C::kQBufs) & 1u) ^ 1u, abort_flag, budget)) {
        fail();
        ok = false;
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      {
        const uint32_t bar = smem_u32(&misc.q_full[qb]);
        const int rows = p.head_blocks == 1 ? p.rows_per_block : 1;
        if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(kW * p.heads_per_block * rows * 128));
        __syncwarp();
        const int row = w.q0 + (p.head_blocks == 1 ? w.rb * rows : w.rb / p.head_blocks);
        const int head = p.head_blocks == 1 ? 0 : (w.rb % p.head_blocks) * p.heads_per_block;
        if (lane < kW)
          tma_load_5d(s_q + qb * C::kQBytes + lane * C::kQChunkBytes, &tm_q, bar, 0, head, row, lane, w.g, pol_q);
        q_armed |= 1u << qb;
        q_armed_par = (q_armed_par & ~(1u << qb)) | (((kq / C::kQBufs) & 1u) << qb);
        ++kq;
      }
      for (int i = w.a; i < w.e && ok; ++i, ++t) {
        const int first = (w.tile0 + i) * pages;
        const int p0 = max(page_lo, first), p1 = min(page_hi, first + pages);
        const int page = first + lane;
        const bool mine = page >= p0 && page < p1;
        int group8 = p.page_groups;
        if (mine) {
          if (id < 0 || (static_cast<int64_t>(id) + 1) * (P / 8) > p.page_groups) record_error(p.err, MLA_DEV_BAD_SUBPAGE);
          else group8 = id * (P / 8);
        }
        if (i + 1 < w.e) id = id_of(i + 1);
        load_tile(&tm_k, k_use<C>(t), group8, mine, p1 - p0, w.g);
        if (t > 0 && ok) load_tile(&tm_v, v_use<C>(t - 1), prev_group, prev_mine, prev_pages, prev_g);
        prev_group = group8;
        prev_mine = mine;
        prev_pages = p1 - p0;
        prev_g = w.g;
      }
    }
    if (ok && t > 0) load_tile(&tm_v, v_use<C>(t - 1), prev_group, prev_mine, prev_pages, prev_g);
    if (lane == 0 && (!ok || *abort_flag)) {
      // copies in flight land before the memory is given up
      const volatile int never = 0;
      for (int s = 0; s < C::kSlots; ++s)
        if (armed & (1u << s)) mbar_wait(smem_u32(&misc.full[s]), (armed_par >> s) & 1u, &never, p.drain_budget);
      for (int s = 0; s < C::kQBufs; ++s)
        if (q_armed & (1u << s)) mbar_wait(smem_u32(&misc.q_full[s]), (q_armed_par >> s) & 1u, &never, p.drain_budget);
    }
  } else if (warp == kMma) {
    // ======================================================== products
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, C::kNR, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(kW < 2 ? 64 : 128, kNC, 1, 1);
      const uint64_t d_k = sdesc_sw128(s_slots, 0, C::kCW * 1024);        // tokens: groups of 8
      const uint64_t d_v = sdesc_sw128(s_slots, 1024, C::kCW * 1024);     // dims: chunks; tokens: groups of 8
      const uint64_t d_q = sdesc_sw128(s_q, 0, 1024);
      const uint64_t d_p = sdesc_sw128(s_p, 1024, 1024);
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t par) {
        if (ok && !mbar_wait(bar, par, abort_flag, budget)) {
          fail();
          ok = false;
        }
        return ok;
      };
      int prev_k0 = 0, prev_k1 = 0;
      bool prev_first = false;
      auto pv = [&](uint32_t t) {
        if (!wait(smem_u32(&misc.p_full[t & 1u]), (t >> 1) & 1u)) return;
        const uint32_t use = v_use<C>(t);
#pragma unroll
        for (int s = 0; s < C::kNS; ++s)
          if (!wait(full_bar(use + s), full_par(use + s))) return;
        tc_fence_after();
        const uint64_t dp = d_p + (t & 1u) * (C::kPBytes >> 4);
#pragma unroll
        for (int s = 0; s < C::kBlocks; ++s) {
          const uint64_t dv = d_v + ((use + s) % C::kSlots) * (C::kSlotBytes >> 4);
          const uint32_t o = tmem + kNC * (2 + s);
          for (int k = prev_k0; k < prev_k1; ++k) {
            const uint64_t a = dv + k * (2 * C::kCW * 1024 >> 4), b = dp + k * (2048 >> 4);
            if (prev_first && k == prev_k0) umma_bf16_ss_first(o, a, b, idesc_pv);
            else umma_bf16_ss_acc(o, a, b, idesc_pv);
          }
          umma_commit(smem_u32(&misc.empty[(use + s) % C::kSlots]));
        }
        umma_commit(smem_u32(&misc.o_done[t & 1u]));
      };
      Walk walk(p, misc, pos_a, pos_e);
      Part w;
      uint32_t t = 0, kq = 0;
      while (ok && walk.next(w)) {
        if (w.e == w.a) continue;
        const uint32_t qb = kq % C::kQBufs;
        if (!wait(smem_u32(&misc.q_full[qb]), (kq / C::kQBufs) & 1u)) break;
        for (int i = w.a; i < w.e && ok; ++i, ++t) {
          const uint32_t use = k_use<C>(t);
          const uint32_t s_t = tmem + (t & 1u) * kNC;
#pragma unroll
          for (int s = 0; s < C::kNS; ++s) {
            if (!wait(full_bar(use + s), full_par(use + s))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < C::kCW; ++c) {
              const int chunk_i = s * C::kCW + c;             // of the token's row of keys
              const int map = chunk_i / (kW / kMaps);
              const bool fresh = chunk_i % (kW / kMaps) == 0;  // first chunk of its map
              const uint64_t a = d_k + ((use + s) % C::kSlots) * (C::kSlotBytes >> 4) + c * (1024 >> 4);
              const uint64_t b = d_q + qb * (C::kQBytes >> 4) + chunk_i * (C::kQChunkBytes >> 4);
              const uint32_t d = s_t + map * C::kNR;
              if (fresh) umma_bf16_ss_first(d, a, b, idesc_qk);
              else umma_bf16_ss_acc(d, a, b, idesc_qk);
              umma_bf16_ss_acc(d, a + 2, b + 2, idesc_qk);
              umma_bf16_ss_acc(d, a + 4, b + 4, idesc_qk);
              umma_bf16_ss_acc(d, a + 6, b + 6, idesc_qk);
            }
            umma_commit(smem_u32(&misc.empty[(use + s) % C::kSlots]));
          }
          if (!ok) break;
          if (i + 1 == w.e) umma_commit(smem_u32(&misc.q_empty[qb]));
          umma_commit(smem_u32(&misc.s_full[t & 1u]));
          if (t > 0) pv(t - 1);
          const int tok = (w.tile0 + i) * kTile;
          prev_k0 = max(w.lo - tok, 0) / 16;
          prev_k1 = (min(w.hi - tok, kTile) + 15) / 16;
          prev_first = i == w.a;
        }
        ++kq;
      }
      if (ok && t > 0) pv(t - 1);
      umma_commit(smem_u32(&misc.fin));
      const volatile int never = 0;
      mbar_wait(smem_u32(&misc.fin), 0, &never, p.drain_budget);
    }
    __syncwarp();
  } else {
    // ======================================================== softmax
    constexpr int N = C::kCols;
    const int grp = warp >> 2, wq = warp & 3;
    const int col0 = grp * N;                      // first column of this group of warps
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    const int row = wq * 32 + lane;                // token of the tile; lane of TMEM
    const uint32_t grp_bar = 1 + grp, all_bar = 3;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t par) {
      if (ok && !mbar_wait(bar, par, abort_flag, budget)) {
        fail();
        ok = false;
      }
    };
    uint32_t t = 0;
    int n_part = 0;
    Meta meta{0, 0, 0, -1};
    Walk walk(p, misc, pos_a, pos_e);
    Part w;
    while (walk.next(w)) {
      // what this lane's column sees
      int my_lo = 0, my_hi = 0, ct, ch;
      const int my_col = col0 + lane % N;
      const bool valid = column_row(p, w.rb, my_col % C::kNR, w.qlen, ct, ch);
      if (valid) {
        my_hi = min(max(p.row_len[w.q0 + ct], 0), p.max_len);
        my_lo = p.window > 0 ? max(0, my_hi - p.window) : 0;
      }
      if (wq == 0 && lane < N) {
        misc.col_lo[my_col] = my_lo;
        misc.col_hi[my_col] = my_hi;
      }
      named_bar_sync(all_bar, kSoftmaxThreads);
      if (threadIdx.x == 0) misc.stop[n_part & 1] = *abort_flag;
      named_bar_sync(all_bar, kSoftmaxThreads);
      if (misc.stop[n_part & 1]) break;
      ++n_part;
      // tokens that this group's columns all see (all_lo .. all_hi - 1), and
      // that all columns see that see anything (edge_lo .. edge_hi - 1)
      int all_lo = valid ? my_lo : 0, all_hi = valid ? my_hi : INT32_MAX;
      int edge_lo = 0, edge_hi = INT32_MAX;
      for (int c = lane; c < kNC; c += 32)
        if (misc.col_hi[c] > 0) {
          edge_lo = max(edge_lo, misc.col_lo[c]);
          edge_hi = min(edge_hi, misc.col_hi[c]);
        }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
        all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
        edge_lo = max(edge_lo, __shfl_xor_sync(0xffffffffu, edge_lo, o));
        edge_hi = min(edge_hi, __shfl_xor_sync(0xffffffffu, edge_hi, o));
      }
      float m[N], sum[N];
#pragma unroll
      for (int c = 0; c < N; ++c) {
        m[c] = kLowest;
        sum[c] = 0.0f;
      }
      for (int i = w.a; i < w.e; ++i, ++t) {
        const uint32_t sb = t & 1u;
        const int tok0 = (w.tile0 + i) * kTile, tok = tok0 + row;
        wait(smem_u32(&misc.s_full[sb]), (t >> 1) & 1u);
        tc_fence_after();
        float x[N];
        tmem_load<N>(tmem + lane_addr + sb * kNC + col0, x);
        const bool masked = tok0 < all_lo || tok0 + kTile > all_hi;
        float top = -INFINITY;
        if (!masked) {
#pragma unroll
          for (int c = 0; c < N; ++c) {
            x[c] *= p.scale_log2;
            top = fmaxf(top, x[c] - m[c]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const int lo = __shfl_sync(0xffffffffu, my_lo, c), hi = __shfl_sync(0xffffffffu, my_hi, c);
            x[c] = tok >= lo && tok < hi ? x[c] * p.scale_log2 : -INFINITY;
            top = fmaxf(top, x[c] - m[c]);
          }
        }
        if (named_bar_red_or(grp_bar, 128, top > kLag)) {
          float v[N];
#pragma unroll
          for (int c = 0; c < N; ++c) v[c] = x[c];
          const float r = reduce_columns<true, N>(v, lane);
          if (lane < N) misc.red[grp][wq][lane] = r;
          named_bar_sync(grp_bar, 128);
          float f[N];
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const float best = fmaxf(fmaxf(misc.red[grp][0][c], misc.red[grp][1][c]), fmaxf(misc.red[grp][2][c], misc.red[grp][3][c]));
            const float now = fmaxf(m[c], best);
            f[c] = fast_exp2(m[c] - now);
            m[c] = now;
            sum[c] *= f[c];
          }
          if (i > w.a) {
            wait(smem_u32(&misc.o_done[sb ^ 1u]), ((t - 1) >> 1) & 1u);
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < C::kBlocks; ++s) {
              float o[N];
              tmem_load<N>(tmem + lane_addr + kNC * (2 + s) + col0, o);
#pragma unroll
              for (int c = 0; c < N; ++c) o[c] *= f[c];
              tmem_store<N>(tmem + lane_addr + kNC * (2 + s) + col0, o);
            }
          }
        }
        uint32_t pk[N / 2];
#pragma unroll
        for (int c = 0; c < N; c += 2) {
          const float p0 = fast_exp2(x[c] - m[c]), p1 = fast_exp2(x[c + 1] - m[c + 1]);
          sum[c] += p0;
          sum[c + 1] += p1;
          pk[c / 2] = pack_bf16(p0, p1);
        }
        if (t >= 2) wait(smem_u32(&misc.o_done[sb]), ((t - 2) >> 1) & 1u);  // P of tile t - 2 has been read
        const uint32_t prow = s_p + sb * C::kPBytes + row * 128;
#pragma unroll
        for (int j = 0; j < N / 8; ++j)
          st_shared_v4(prow + (((col0 / 8 + j) ^ (row & 7)) * 16), pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        if (grp == 0 && (tok0 < edge_lo || tok0 + kTile > edge_hi)) {
          const bool dead = tok < w.lo || tok >= w.hi;
          const bool mixed = !dead && (tok < edge_lo || tok >= edge_hi);
          if (__any_sync(0xffffffffu, dead || mixed)) {
            const uint32_t use = v_use<C>(t);
#pragma unroll
            for (int s = 0; s < C::kNS; ++s) wait(full_bar(use + s), full_par(use + s));
            bool zero = dead;
            auto piece = [&](int s, int c, int j) {
              return s_slots + ((use + s) % C::kSlots) * C::kSlotBytes + (row >> 3) * (C::kCW * 1024) + c * 1024 +
                     (row & 7) * 128 + j * 16;
            };
            if (mixed) {
              bool odd = false;
              for (int s = 0; s < C::kNS; ++s)
                for (int c = 0; c < C::kCW; ++c)
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const uint4 v = ld_shared_v4(piece(s, c, j));
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                      odd |= (u[k] & 0x7f80u) == 0x7f80u || (u[k] & 0x7f800000u) == 0x7f800000u;
                  }
              if (odd) {
                zero = true;
                for (int c = 0; c < kNC; ++c)
                  if (tok >= misc.col_lo[c] && tok < misc.col_hi[c]) atomicOr(&misc.bad[c / N], 1u << (c % N));
              }
            }
            if (zero)
              for (int s = 0; s < C::kNS; ++s)
                for (int c = 0; c < C::kCW; ++c)
#pragma unroll
                  for (int j = 0; j < 8; ++j) st_shared_v4(piece(s, c, j), 0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&misc.p_full[sb]));
      }

      // ---- the part's result
      if (w.e > w.a) wait(smem_u32(&misc.o_done[(t - 1) & 1u]), ((t - 1) >> 1) & 1u);
      {
        float v[N];
#pragma unroll
        for (int c = 0; c < N; ++c) v[c] = sum[c];
        const float r = reduce_columns<false, N>(v, lane);
        if (lane < N) misc.red[grp][wq][lane] = r;
      }
      if (wq == 0) {
#pragma unroll
        for (int c = 0; c < N; ++c)
          if (lane == c) misc.stat_m[col0 + c] = m[c];
      }
      named_bar_sync(grp_bar, 128);
      if (wq == 0 && lane < N)
        misc.stat_l[col0 + lane] = misc.red[grp][0][lane] + misc.red[grp][1][lane] + misc.red[grp][2][lane] + misc.red[grp][3][lane];
      named_bar_sync(all_bar, kSoftmaxThreads);
      tc_fence_after();
      const bool whole = w.a == 0 && w.e == w.n;
      const unsigned bad0 = misc.bad[0], bad1 = misc.bad[1];
      auto is_bad = [&](int c) { return ((c < N ? bad0 >> c : bad1 >> (c - N)) & 1u) != 0; };
      // dim of this thread in block s of O^T: an M = 64 result has its rows in lanes 0-15 of each warp
      const bool has_dim = kW >= 2 || lane < 16;
      const int dim = kW >= 2 ? row : wq * 16 + lane;
      if (!whole) {
        const int64_t rec = static_cast<int64_t>(chunk) * 2 + (w.a == 0 ? 1 : 0);
        if (wq == 0 && lane < N) {
          p.part_stat[rec * 2 * kNC + col0 + lane] = misc.stat_m[col0 + lane];
          p.part_stat[rec * 2 * kNC + kNC + col0 + lane] = misc.stat_l[col0 + lane];
        }
        float *po = p.part_o + rec * kNC * C::kDv;
#pragma unroll
        for (int s = 0; s < C::kBlocks; ++s) {
          float o[N];
          tmem_load<N>(tmem + lane_addr + kNC * (2 + s) + col0, o);
          if (has_dim)
#pragma unroll
            for (int c = 0; c < N; ++c)
              po[(col0 + c) * C::kDv + 128 * s + dim] = is_bad(col0 + c) ? __int_as_float(0x7fffffff) : o[c];
        }
        if (w.a == 0) meta = Meta{w.b, w.g, w.rb, chunk_of(w.start + kOverhead + w.n - 1)};
      } else if (kMaps == 1) {
        if (wq == 0 && valid && lane < N) {
          const float l = misc.stat_l[my_col];
          p.lse[(static_cast<int64_t>(w.q0) + ct) * p.num_heads + w.g * p.group + ch] =
              l == 0.0f ? -INFINITY : (misc.stat_m[my_col] + log2f(l)) * kLn2;
        }
#pragma unroll
        for (int s = 0; s < C::kBlocks; ++s) {
          float o[N];
          tmem_load<N>(tmem + lane_addr + kNC * (2 + s) + col0, o);
#pragma unroll
          for (int c = 0; c < N; ++c) {
            int rt, rh;
            if (column_row(p, w.rb, col0 + c, w.qlen, rt, rh) && has_dim) {
              const float l = misc.stat_l[col0 + c];
              const float y = l == 0.0f ? 0.0f : (is_bad(col0 + c) ? __int_as_float(0x7fffffff) : o[c] / l);
              p.out[((static_cast<int64_t>(w.q0) + rt) * p.num_heads + w.g * p.group + rh) * C::kDv + 128 * s + dim] =
                  __float2bfloat16_rn(y);
            }
          }
        }
      } else {
        // 16 rows of both maps per group of warps
        constexpr int R = 16;
        const int r0 = grp * R;
        if (wq == 0 && valid && lane < N) {
          const float l = misc.stat_l[my_col];
          p.lse[((static_cast<int64_t>(w.q0) + ct) * p.num_heads + w.g * p.group + ch) * 2 + my_col / C::kNR] =
              l == 0.0f ? -INFINITY : (misc.stat_m[my_col] + log2f(l)) * kLn2;
        }
        float y[C::kBlocks][R], sq[R];
#pragma unroll
        for (int c = 0; c < R; ++c) sq[c] = 0.0f;
#pragma unroll
        for (int s = 0; s < C::kBlocks; ++s) {
          float o[R];
          tmem_load<R>(tmem + lane_addr + kNC * (2 + s) + r0, y[s]);
          tmem_load<R>(tmem + lane_addr + kNC * (2 + s) + C::kNR + r0, o);
#pragma unroll
          for (int c = 0; c < R; ++c) {
            int rt, rh;
            const bool there = column_row(p, w.rb, r0 + c, w.qlen, rt, rh);
            const float lam = there ? p.lambda[w.g * p.group + rh] : 0.0f;
            const float l0 = misc.stat_l[r0 + c], l1 = misc.stat_l[C::kNR + r0 + c];
            const float u0 = l0 == 0.0f ? 0.0f : y[s][c] / l0, u1 = l1 == 0.0f ? 0.0f : o[c] / l1;
            y[s][c] = is_bad(r0 + c) ? __int_as_float(0x7fffffff) : u0 - lam * u1;
            sq[c] += y[s][c] * y[s][c];
          }
        }
        float norm[R];
#pragma unroll
        for (int c = 0; c < R; ++c) norm[c] = 1.0f;
        if (p.gain != nullptr) {
          const float r = reduce_columns<false, R>(sq, lane);
          named_bar_sync(grp_bar, 128);
          if (lane < R) misc.red[grp][wq][lane] = r;
          named_bar_sync(grp_bar, 128);
#pragma unroll
          for (int c = 0; c < R; ++c) {
            const float total_sq = misc.red[grp][0][c] + misc.red[grp][1][c] + misc.red[grp][2][c] + misc.red[grp][3][c];
            norm[c] = rsqrtf(total_sq * (1.0f / C::kDv) + p.eps);
          }
        }
#pragma unroll
        for (int s = 0; s < C::kBlocks; ++s) {
          const float gain = p.gain != nullptr ? p.gain[128 * s + dim] : 1.0f;
#pragma unroll
          for (int c = 0; c < R; ++c) {
            int rt, rh;
            if (column_row(p, w.rb, r0 + c, w.qlen, rt, rh)) {
              const float z = misc.stat_l[r0 + c] == 0.0f ? 0.0f : y[s][c] * norm[c] * gain;
              p.out[((static_cast<int64_t>(w.q0) + rt) * p.num_heads + w.g * p.group + rh) * C::kDv + 128 * s + dim] =
                  __float2bfloat16_rn(z);
            }
          }
        }
      }
      tc_fence_before();
      named_bar_sync(all_bar, kSoftmaxThreads);  // statistics and flags have been read
      if (threadIdx.x < 2) misc.bad[threadIdx.x] = 0;
    }
    if (threadIdx.x == 0) p.meta[chunk] = meta;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) tmem_dealloc(tmem, C::kTmemCols);
}

}  // namespace grouped
}  // namespace mla
