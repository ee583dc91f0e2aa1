// mla_grouped.cuh -- the decode kernel of grouped-query and differential
// attention over a paged K/V cache, and what its launcher and its merge share
// with it.
//
// For every row (verify row t of request b, query head of group g) and map m:
//   s_j = sm_scale <q_m, k_{j,g,m}>,  o_m = sum_j softmax(s)_j v_{j,g}
// with an online base-2 softmax.  The rows of a group (heads x verify rows) go
// over their keys and values together, so the cache is read once per group:
// R flops a byte for R rows, so memory decides (282 flops a byte is the ridge)
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
//    that one box brings a page (32 tokens of a larger one: what lies outside a
//    window or behind the end is not read) as [8 rows][chunk][row][128 bytes]:
//    the same uniform strides for pages of 8 as of 128, read by both products as
//    they are (128-byte swizzle).
//  * Copies through a ring of slots of at most 32 KB (two chunks) for the keys
//    and one for the values, which wait for the softmax; a warp copies into each,
//    a warp issues each product, and the stream of tiles runs on from part to part.
//  * Balanced split: a unit (request, group, row block) is kOverhead positions
//    and then its tiles; the positions of all units, laid end to end, are cut
//    into equal chunks, one per SM, or per two that have a group's row blocks between
//    them (a few short units: a chunk each).  A chunk holds at most two units that it
//    does not hold whole: its first and its last.  So there are two partial
//    records per SM, whatever the batch, and the merge looks at 152 chunks.
//  * Softmax: a thread has one token and the 16 columns of its group of warps (32
//    of 64), in registers.  The reference maximum moves only when a score
//    passes it by 2^8; sums are float32 per thread and column.  A probability goes
//    to the product as two bf16 terms (2^-16 of itself), the second as further
//    columns of N, which cost the tensor cores nothing up to N = 64.
//  * Tokens that no row sees are neither loaded (whole pages) nor multiplied:
//    their values in shared memory are set to zero.  A token that some rows see
//    is looked at, and a value in it that is not finite is zeroed too and
//    spoils the rows that see it (0 x NaN would spoil the others).
//  * Every wait is bounded; one that runs out records MLA_DEV_WAIT_TIMEOUT, all
//    roles end, copies in flight land, TMEM is freed.  Neither the part at hand
//    nor a unit with such a part is stored: its rows are left as they were.
//
// Measured (one call among others on fresh inputs; in brackets calls in a graph, by
// box): 32 requests of 1,024-8,192 tokens, 8 key heads of 128, 96.5 us (593 MB: 6.1
// TB/s, 0.91 of a copy's rate) [92-94]; 4 x 131,072, 4 key heads, 64 rows 169.5 us
// (1.07 GB: 0.94) [167-170]; 40 requests of 8 groups with two maps of 64 134 us (839
// MB: 0.93) [129-133]; ragged ones with heads of 64 89 us (470 MB: 0.78) [80-88]. A
// tile of 16 columns takes its softmax about 900 cycles, its products 400 and 420,
// beside 2,800 for its copy; of 64 columns the softmax 1,500 (two warps a scheduler:
// exp2 512, the rest instructions and spills). What every call adds: 4 us until the
// first copies (offsets, row lengths, sum, page ids in turn), 1 of epilogue, 1-4 of
// merge.
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
constexpr int kMaxReqs = 512;     // requests of one launch (tabulated in shared memory)
constexpr int kOverhead = 2;      // positions a unit counts beside its tiles (1: ragged heads of 64 79 -> 82 us; 3, 4: no change)
constexpr int kMinChunk = 4;      // positions a chunk has at least (6: two requests of two tiles 8.0 -> 12.3 us)
constexpr int kMaxCtas = 152;

// Tiles up to which units are not cut, when there are no more units than SMs: a
// tile more takes 0.3-0.6 us, parts and their merge 2 to 4 (units of 4 tiles of 128
// dims 13.3 -> 9.4 us for 16 requests, of 8 tiles 15.8 -> 12.6 for 16, 9.8 -> 10.0
// for one; of 256 dims 4 tiles 12.7 -> 10.4, 8 tiles 12.7 -> 15.1).
__host__ __device__ constexpr int whole_tiles(int W) { return W == 4 ? 4 : 8; }

// A unit that is cut across chunks: written by the chunk with its first tile.
struct Meta {
  int q0, qlen, g, rb;
  int last;  // CTA that has its last tile; -1: no such unit starts in this one's chunk
  int step;  // from a CTA with a part to the next
  int pad[2];
};

struct Params {
  const int32_t *qo_indptr, *row_len, *subpage_table;
  __nv_bfloat16 *out;
  float *lse;
  const float *lambda, *gain;
  float eps;
  float *part_o;     // [CTA][2][NC][64 W] unnormalised outputs
  float *part_stat;  // [CTA][2][2][NC] base-2 maxima, sums (-1: a wait gave up)
  Meta *meta;        // [CTA]
  int *err;
  long long wait_budget, drain_budget;
  float scale_log2;
  int first_req;  // of the call, where it takes several launches
  int num_reqs, num_rows, num_heads, num_kv_heads, group, max_qlen, max_len, window;
  int subpage_stride, page_shift, page_groups;  // pages of 2^page_shift; page_groups: num_cache_rows / 8
  int box_shift;        // a copy's box has 2^box_shift tokens: a page, or 32 of a larger one
  int rows_per_block;   // verify rows of a row block (group <= NR)
  int heads_per_block;  // query heads of a row block: group, or NR if group > NR
  int one_block;        // every request has one row block
  int few;              // no more units than CTAs
  int may_twin;         // a request may have several row blocks
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
  static constexpr int kPN = 2 * kNC;               // columns of P^T: both terms
  static constexpr int kPAtoms = kPN <= 64 ? 1 : 2; // of 64 columns
  static constexpr int kPBytes = kPAtoms * kTile * 128;
  static constexpr int kMiscBytes = 16 * 1024;
  static constexpr int kPBufs = kW == 4 && kNR == 64 ? 1 : 2;  // where two leave no room for a key and a value tile
  static constexpr int kFit = (232448 - 1024 - kMiscBytes - kQBufs * kQBytes - kPBufs * kPBytes) / kSlotBytes;
  static constexpr int kSlots = kFit > 10 ? 10 : kFit;
  static constexpr int kKSlots = kSlots / 2, kVSlots = kSlots - kKSlots;  // values wait for the softmax
  static constexpr int kCols = kNC < 64 ? 16 : 32;  // columns of a group of four softmax warps
  static constexpr int kGroups = kNC / kCols;
  static constexpr int kSoftmaxWarps = 4 * kGroups;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
  static constexpr int kBlocks = kW < 2 ? 1 : kW / 2;  // blocks of O^T: 128 dims each (64 if W = 1)
  static constexpr int kTmemO = 2 * kNC;             // behind the two S^T: blocks of kPN columns
  static constexpr int kTmemUsed = kTmemO + kPN * kBlocks;
  static constexpr int kTmemCols = kTmemUsed <= 64 ? 64 : (kTmemUsed <= 128 ? 128 : (kTmemUsed <= 256 ? 256 : 512));
  static constexpr int kOffQ = kSlots * kSlotBytes;
  static constexpr int kOffP = kOffQ + kQBufs * kQBytes;
  static constexpr int kOffMisc = kOffP + kPBufs * kPBytes;
  static constexpr int kSmem = kOffMisc + kMiscBytes + 1024;
  static_assert(kTmemUsed <= 512 && kNR % 16 == 0 && kKSlots >= kNS && kSmem <= 232448, "configuration");
};

// Row blocks of the CTAs of a chunk: of two, one has the even and one the odd ones.
__device__ __forceinline__ int rounds_of(const Params &p, int qlen, int twin) {
  return p.one_block ? 1 : (blocks_of(p, qlen) + twin) >> twin;
}

// The first unit that a chunk meets: its request, group and round of row blocks,
// its position, its positions, and the request's rounds.
struct Place {
  int b, g, rb, s, per, blocks;
};

// Tiles of a request's units, from the tokens that its rows see.
__device__ __forceinline__ int tiles_of(const int4 &req) {
  return req.y > req.x ? (req.y + kTile - 1) / kTile - req.x / kTile : 0;
}

// A part: the tiles a .. e - 1 (of n) of a unit that lie in this chunk.
struct Part {
  int b, g, rb;   // request, group, row block
  int q0, qlen;
  int lo, hi;     // tokens the request sees
  int tile0;      // tile index of the unit's tile 0
  int a, e, n;
  int start;      // position of the unit
};

struct Misc;

// Goes over a chunk's parts in order.  The issuing roles have one each; the
// softmax warps' is in shared memory (in registers it made them spill).
struct Walk {
  int pos_a, pos_e;  // the chunk
  int b, g, rb, s, per, blocks, tiles;
  int4 req;
  __device__ __forceinline__ void begin(const Misc &m, int a, int e);
  template <bool kTwin>  // there may be several row blocks
  __device__ __forceinline__ bool next(const Params &p, const Misc &m, Part &o);
};

// What the softmax warps share about a part's columns.
struct Columns {
  alignas(16) float stat_m[64], stat_l[64], inv[64];
  alignas(16) int lo[64], hi[64];  // tokens that a column sees
  int row[64];         // its row of out (row * H + head), -1: none
  float lam[64];
  unsigned bad[2];     // columns of a group of warps that see a value that is not finite
  Part part;           // the part itself
  int more;            // there is one
  int stop;            // the role ends here (a wait ran out)
};

struct Misc {
  uint64_t full[10], empty[10];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2], fin[2];
  uint32_t tmem_base;
  int abort;
  uint32_t armed[10], q_armed[2];         // 1 + the parity of the last use of a slot (or Q buffer) that a copy was issued for
  int start[kMaxReqs + 1];                // positions before request b
  int4 req[kMaxReqs];                     // tokens that some row of the request sees (x .. y - 1), first row, rows
  Walk walk;                              // the softmax warps'
  Place place;                            // where this chunk begins
  int whole;                              // a chunk is a unit: one position each
  int twin;                               // 1: two CTAs share a chunk, each with its row blocks
  alignas(16) float red[2][4][32];        // [group of warps][warp][column]
  Columns cols[2];                        // of the even and odd parts
};
static_assert(sizeof(Misc) <= 16 * 1024, "misc");

__device__ __forceinline__ void Walk::begin(const Misc &m, int a, int e) {
  pos_a = a;
  pos_e = e;
  b = m.place.b;
  g = m.place.g;
  rb = m.place.rb;
  s = m.place.s;
  per = m.place.per;
  blocks = m.place.blocks;
  req = m.req[b];
  tiles = tiles_of(req);
}

template <bool kTwin>
__device__ __forceinline__ bool Walk::next(const Params &p, const Misc &m, Part &o) {
  const int twin = kTwin && p.may_twin ? m.twin : 0;
  while (s < pos_e) {
    const int first = s + kOverhead, n = tiles;
    const int a = m.whole ? 0 : max(pos_a - first, 0), e = m.whole ? n : min(pos_e - first, n);
    int block = kTwin ? rb : 0;
    bool take = n > 0 ? e > a : s >= pos_a;
    if (twin) {
      block = 2 * rb + static_cast<int>(blockIdx.x & 1);
      take = take && block < blocks_of(p, req.w);
    }
    if (take) o = Part{b, g, block, req.z, req.w, req.x, req.y, req.x / kTile, n == 0 ? 0 : a, n == 0 ? 0 : e, n, s};
    s += per;
    if (++rb == blocks) {
      rb = 0;
      if (++g == p.num_kv_heads && s < pos_e) {  // the next request that has rows
        g = 0;
        do ++b;
        while (m.start[b + 1] <= s);
        req = m.req[b];
        blocks = kTwin ? rounds_of(p, req.w, twin) : 1;
        tiles = tiles_of(req);
        per = m.whole ? 1 : tiles + kOverhead;
      }
    }
    if (take) return true;
  }
  return false;
}

// Slot of the u-th use of the keys' ring, or of the values' ring behind it (each
// in order of its own copies and products), and the parity of that use.
template <class C>
__device__ __forceinline__ uint32_t k_slot(uint32_t u) { return u % C::kKSlots; }
template <class C>
__device__ __forceinline__ uint32_t v_slot(uint32_t u) { return C::kKSlots + u % C::kVSlots; }
template <class C>
__device__ __forceinline__ uint32_t k_par(uint32_t u) { return (u / C::kKSlots) & 1u; }
template <class C>
__device__ __forceinline__ uint32_t v_par(uint32_t u) { return (u / C::kVSlots) & 1u; }

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

__device__ __forceinline__ bool elect_one() {
  uint32_t y;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(y));
  return y != 0;
}
// D(tmem) = A B^T, or += if acc.
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
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

// Stores of threads for which `there` holds (a predicate: 16 branches in a row
// cost 120 cycles each).
__device__ __forceinline__ void store_if(bool there, float *p, float v) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q st.global.f32 [%0], %1;\n\t}" ::"l"(p), "f"(v),
               "r"(static_cast<uint32_t>(there))
               : "memory");
}
__device__ __forceinline__ void store_if(bool there, __nv_bfloat16 *p, float v) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q st.global.b16 [%0], %1;\n\t}" ::"l"(p),
               "h"(*reinterpret_cast<const uint16_t *>(&h)), "r"(static_cast<uint32_t>(there))
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

// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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
  // warps behind the softmax: copies of K and Q, copies of V, products with K, products with V
  constexpr int kCopyK = C::kSoftmaxWarps, kCopyV = kCopyK + 1, kMmaK = kCopyK + 2, kMmaV = kCopyK + 3;
  constexpr int kSoftmaxThreads = 32 * C::kSoftmaxWarps;
  constexpr bool kTwin = kNC == 64;  // fewer columns hold all rows of a group

  if (warp == kMmaK) {
    tmem_alloc(smem_u32(&misc.tmem_base), C::kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_u32(&misc.full[i]), 1);
      mbar_init(smem_u32(&misc.empty[i]), 1);
      misc.armed[i] = 0;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&misc.q_full[i]), 1);
      mbar_init(smem_u32(&misc.q_empty[i]), 1);
      mbar_init(smem_u32(&misc.s_full[i]), 1);
      mbar_init(smem_u32(&misc.p_full[i]), C::kSoftmaxWarps);
      mbar_init(smem_u32(&misc.o_done[i]), 1);
      mbar_init(smem_u32(&misc.fin[i]), 1);
      misc.q_armed[i] = 0;
    }
    misc.abort = 0;
    misc.place = Place{0, 0, 0, INT32_MAX, 0, 0};  // a chunk without positions
    fence_mbar_init();
  }
  // Query rows that no copy fills (a group that does not divide the columns) stay zero.
  for (int i = threadIdx.x; i < C::kQBufs * C::kQBytes / 16; i += C::kThreads)
    st_shared_v4(s_q + 16 * i, 0, 0, 0, 0);
  fence_proxy_async_smem();
  grid_dep_wait();
  grid_dep_launch();

  // What each request's rows see, and its positions.
  bool low = true;  // units are not worth a cut
  for (int b = threadIdx.x; b < p.num_reqs; b += C::kThreads) {
    // the first row lengths where a batch of equal requests has them, read beside the offsets
    int ahead[4];
    const int64_t guess = static_cast<int64_t>(p.first_req + b) * p.max_qlen;
#pragma unroll
    for (int k = 0; k < 4; ++k) ahead[k] = k < p.max_qlen && guess + k < p.num_rows ? p.row_len[guess + k] : 0;
    const int q0 = p.qo_indptr[b], q1 = p.qo_indptr[b + 1];
    int lo = INT32_MAX, hi = 0, cost = 0;  // of the rows that see anything
    if (q0 < 0 || q1 < q0 || q1 > p.num_rows || q1 - q0 > p.max_qlen) {
      record_error(p.err, MLA_DEV_BAD_INDPTR);
    } else if (q1 > q0) {
      for (int r0 = q0; r0 < q1; r0 += 4) {
        int n[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) n[k] = r0 + k >= q1 ? 0 : (q0 == guess && r0 == q0 ? ahead[k] : p.row_len[r0 + k]);
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
      if (hi == 0) lo = 0;
      const int tiles = tiles_of(make_int4(lo, hi, 0, 0));
      low &= tiles <= whole_tiles(kW);
      cost = (p.one_block ? 1 : blocks_of(p, q1 - q0)) * p.num_kv_heads * (tiles + kOverhead);
    }
    misc.req[b] = make_int4(lo, hi, q0, cost > 0 ? q1 - q0 : 0);
    misc.start[b + 1] = cost;
  }
  if (threadIdx.x == 0) misc.start[0] = 0;
  const bool whole = __syncthreads_and(low) != 0 && p.few;
  if (warp == 0) {
    int twin = 0, carry = 0;
    // Row blocks of a group read the same keys and values.  Two CTAs share a chunk, one
    // with the even and one with the odd blocks, where these are about as many (the odd
    // block of a request leaves one idle): they go over the tokens together, and the
    // second read is L2's.  16 requests of 16,384 tokens, 128 rows of 4 groups of 128 dims
    // 172 -> 126 us, of two maps 324 -> 232; at 1.25 instead of 1.1 64 requests of 3-8 x 16
    // rows 146 -> 139, but 24 ragged ones of 1-8 x 16 78 -> 87.
    if (kTwin && p.may_twin) {
      float single = 0.0f, pairs = 0.0f;
      for (int b = lane; b < p.num_reqs; b += 32) {
        const int4 req = misc.req[b];
        const int blocks = blocks_of(p, req.w), positions = req.w > 0 ? tiles_of(req) + kOverhead : 0;
        single += static_cast<float>(blocks) * positions;
        pairs += static_cast<float>((blocks + 1) / 2) * positions;
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        single += __shfl_xor_sync(0xffffffffu, single, o);
        pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
      }
      twin = !whole && 2.0f * pairs <= 1.1f * single;
      if (lane == 0) misc.twin = twin;
    }
    // running sum, in place
    for (int base = 0; base < p.num_reqs; base += 32) {
      const int b = base + lane;
      int x = b < p.num_reqs ? misc.start[b + 1] : 0;
      if (whole && x > 0) x = blocks_of(p, misc.req[b].w) * p.num_kv_heads;
      if (twin && x > 0) x = rounds_of(p, misc.req[b].w, 1) * p.num_kv_heads * (tiles_of(misc.req[b]) + kOverhead);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < p.num_reqs) misc.start[b + 1] = carry + x;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  // chunks 0 .. rest - 1 have size + 1 positions, the others size
  const unsigned total = misc.start[p.num_reqs];
  const int twin = kTwin && p.may_twin ? misc.twin : 0;
  const unsigned chunks = max(1u, min(gridDim.x >> twin, whole ? total : total / kMinChunk)), size = total / chunks, rest = total - size * chunks;
  const unsigned chunk = blockIdx.x >> twin;
  auto cut = [&](unsigned c) { return static_cast<int>(c * size + min(c, rest)); };
  auto chunk_of = [&](int x) {
    const unsigned big = rest * (size + 1), u = static_cast<unsigned>(x);
    return static_cast<int>(u < big ? u / (size + 1) : rest + (u - big) / size);
  };
  const int pos_a = chunk < chunks ? cut(chunk) : total, pos_e = chunk < chunks ? cut(chunk + 1) : total;
  if (threadIdx.x == 0) misc.whole = whole;
  for (int b = threadIdx.x; b < p.num_reqs; b += C::kThreads) {
    const int from = misc.start[b];
    if (from <= pos_a && pos_a < misc.start[b + 1]) {  // one request at most
      const int4 req = misc.req[b];
      const int per = whole ? 1 : tiles_of(req) + kOverhead, blocks = rounds_of(p, req.w, twin);
      const int j = (pos_a - from) / per, g = blocks == 1 ? j : j / blocks;
      misc.place = Place{b, g, j - g * blocks, from + j * per, per, blocks};
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = misc.tmem_base;
  volatile int *abort_flag = &misc.abort;
  const long long budget = p.wait_budget;
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t par) {
    if (ok && !mbar_wait(bar, par, abort_flag, budget)) {
      *abort_flag = 1;
      record_error(p.err, MLA_DEV_WAIT_TIMEOUT);
      ok = false;
    }
    return ok;
  };
  auto full_bar = [&](uint32_t slot) { return smem_u32(&misc.full[slot]); };
  auto empty_bar = [&](uint32_t slot) { return smem_u32(&misc.empty[slot]); };

  if (warp == kCopyK || warp == kCopyV) {
    // ======================================================== copies
    const bool keys = warp == kCopyK;
    const CUtensorMap *tm = keys ? &tm_k : &tm_v;
    const uint64_t pol_kv = l2_policy_evict_first(), pol_q = l2_policy_evict_last();
    if (lane == 0) {
      tma_prefetch_desc(tm);
      if (keys) tma_prefetch_desc(&tm_q);
    }
    // boxes of a tile, row groups of a page, boxes of a page
    const int shift = p.box_shift, boxes = kTile >> shift, groups = 1 << (p.page_shift - 3), split = p.page_shift - shift;
    const uint32_t box_bytes = (128u * C::kCW) << shift;
    Walk walk;
    walk.begin(misc, pos_a, pos_e);
    Part w;
    uint32_t t = 0, kq = 0;
    while (ok && walk.next<kTwin>(p, misc, w)) {
      if (w.e == w.a) continue;
      // a lane holds a box of the tile, and reads the next tile's page id ahead of the waits
      const int32_t *ids = p.subpage_table + static_cast<int64_t>(w.b) * p.subpage_stride;
      const int box_lo = w.lo >> shift, box_hi = ((w.hi - 1) >> shift) + 1;
      auto id_of = [&](int tile) {
        const int box = (w.tile0 + tile) * boxes + lane;
        return lane < boxes && box >= box_lo && box < box_hi ? ids[box >> split] : -1;
      };
      int id = id_of(w.a);
      if (keys) {
        const uint32_t qb = kq % C::kQBufs;
        if (lane == 0) wait(smem_u32(&misc.q_empty[qb]), ((kq / C::kQBufs) & 1u) ^ 1u);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        const uint32_t bar = smem_u32(&misc.q_full[qb]);
        const int rows = p.head_blocks == 1 ? p.rows_per_block : 1;
        if (lane == 0) {
          misc.q_armed[qb] = 1 + ((kq / C::kQBufs) & 1u);
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(kW * p.heads_per_block * rows * 128));
        }
        __syncwarp();
        const int row = w.q0 + (p.head_blocks == 1 ? w.rb * rows : w.rb / p.head_blocks);
        const int head = p.head_blocks == 1 ? 0 : (w.rb % p.head_blocks) * p.heads_per_block;
        if (lane < kW)
          tma_load_5d(s_q + qb * C::kQBytes + lane * C::kQChunkBytes, &tm_q, bar, 0, head, row, lane, w.g, pol_q);
        ++kq;
      }
      for (int i = w.a; i < w.e && ok; ++i, ++t) {
        const int first = (w.tile0 + i) * boxes;
        const int b0 = max(box_lo, first), b1 = min(box_hi, first + boxes);
        const bool mine = first + lane >= b0 && first + lane < b1;
        int group8 = p.page_groups;  // behind the cache: zeros
        if (mine) {
          if (id < 0 || (static_cast<int64_t>(id) + 1) * groups > p.page_groups) record_error(p.err, MLA_DEV_BAD_SUBPAGE);
          else group8 = id * groups + (((first + lane) & ((1 << split) - 1)) << (shift - 3));
        }
        if (i + 1 < w.e) id = id_of(i + 1);
#pragma unroll
        for (int s = 0; s < C::kNS; ++s) {
          const uint32_t use = C::kNS * t + s;
          const uint32_t slot = keys ? k_slot<C>(use) : v_slot<C>(use), par = keys ? k_par<C>(use) : v_par<C>(use);
          if (lane == 0) wait(empty_bar(slot), par ^ 1u);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          if (lane == 0) {
            misc.armed[slot] = 1 + par;
            mbar_arrive_expect_tx(full_bar(slot), box_bytes * (b1 - b0));
          }
          __syncwarp();
          if (mine)
            tma_load_5d(s_slots + slot * C::kSlotBytes + lane * box_bytes, tm, full_bar(slot), 0, 0, s * C::kCW, group8, w.g,
                        pol_kv);
        }
      }
    }
    __syncwarp();
  } else if (warp == kMmaK) {
    // ======================================================== S^T = K Q^T
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, C::kNR, 0, 0);
      const uint64_t d_k = sdesc_sw128(s_slots, 0, C::kCW * 1024);  // tokens: groups of 8
      const uint64_t d_q = sdesc_sw128(s_q, 0, 1024);
      Walk walk;
      walk.begin(misc, pos_a, pos_e);
      Part w;
      uint32_t t = 0, kq = 0;
      while (ok && walk.next<kTwin>(p, misc, w)) {
        if (w.e == w.a) continue;
        const uint32_t qb = kq % C::kQBufs;
        if (!wait(smem_u32(&misc.q_full[qb]), (kq / C::kQBufs) & 1u)) break;
        ++kq;
        for (int i = w.a; i < w.e; ++i, ++t) {
          // S^T of tile t - 2 has been read
          if (t >= 2 && !wait(smem_u32(&misc.p_full[t & 1u]), ((t - 2) >> 1) & 1u)) break;
#pragma unroll
          for (int s = 0; s < C::kNS; ++s) {
            const uint32_t use = C::kNS * t + s, slot = k_slot<C>(use);
            if (!wait(full_bar(slot), k_par<C>(use))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < C::kCW; ++c) {
              const int ci = s * C::kCW + c;  // chunk of the token's row of keys
              const uint64_t a = d_k + slot * (C::kSlotBytes >> 4) + c * (1024 >> 4);
              const uint64_t b = d_q + qb * (C::kQBytes >> 4) + ci * (C::kQChunkBytes >> 4);
              const uint32_t d = tmem + (t & 1u) * kNC + ci / (kW / kMaps) * C::kNR;
              umma(d, a, b, idesc, ci % (kW / kMaps) != 0);
              umma(d, a + 2, b + 2, idesc, 1);
              umma(d, a + 4, b + 4, idesc, 1);
              umma(d, a + 6, b + 6, idesc, 1);
            }
            umma_commit(empty_bar(slot));
          }
          if (!ok) break;
          if (i + 1 == w.e) umma_commit(smem_u32(&misc.q_empty[qb]));
          umma_commit(smem_u32(&misc.s_full[t & 1u]));
        }
      }
      umma_commit(smem_u32(&misc.fin[0]));
      const volatile int never = 0;
      mbar_wait(smem_u32(&misc.fin[0]), 0, &never, p.drain_budget);
    }
    __syncwarp();
  } else if (warp == kMmaV) {
    // ======================================================== O^T += V^T P^T
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_bf16_f32(kW < 2 ? 64 : 128, C::kPN, 1, 1);
      const uint64_t d_v = sdesc_sw128(s_slots, 1024, C::kCW * 1024);      // dims: chunks; tokens: groups of 8
      const uint64_t d_p = sdesc_sw128(s_p, C::kPBytes / C::kPAtoms, 1024);  // columns: atoms of 64
      Walk walk;
      walk.begin(misc, pos_a, pos_e);
      Part w;
      uint32_t t = 0;
      while (ok && walk.next<kTwin>(p, misc, w)) {
        for (int i = w.a; i < w.e; ++i, ++t) {
          if (!wait(smem_u32(&misc.p_full[t & 1u]), (t >> 1) & 1u)) break;
          const int tok = (w.tile0 + i) * kTile;
          const int k0 = max(w.lo - tok, 0) / 16, k1 = (min(w.hi - tok, kTile) + 15) / 16;
          const uint64_t dp = d_p + (t % C::kPBufs) * (C::kPBytes >> 4);
#pragma unroll
          for (int s = 0; s < C::kBlocks; ++s) {
            const uint32_t use = C::kNS * t + s, slot = v_slot<C>(use);
            if (!wait(full_bar(slot), v_par<C>(use))) break;
            tc_fence_after();
            const uint64_t dv = d_v + slot * (C::kSlotBytes >> 4);
            const uint32_t o = tmem + C::kTmemO + C::kPN * s;
            if (k1 - k0 == kTile / 16) {
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                umma(o, dv + k * (2 * C::kCW * 1024 >> 4), dp + k * (2048 >> 4), idesc, k > 0 || i > w.a);
            } else {
              for (int k = k0; k < k1; ++k)
                umma(o, dv + k * (2 * C::kCW * 1024 >> 4), dp + k * (2048 >> 4), idesc, k > k0 || i > w.a);
            }
            umma_commit(empty_bar(slot));
          }
          if (!ok) break;
          umma_commit(smem_u32(&misc.o_done[t & 1u]));
        }
      }
      umma_commit(smem_u32(&misc.fin[1]));
      const volatile int never = 0;
      mbar_wait(smem_u32(&misc.fin[1]), 0, &never, p.drain_budget);
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
    uint32_t t = 0;
    Meta meta{0, 0, 0, 0, -1, 1, {}};
    const int my_col = col0 + lane % N;
    bool valid = false, gave_up = false;
    int my_lo = 0, my_hi = 0, ct = 0, ch = 0, cur_b = -1, cur_rb = -1;
    if (threadIdx.x == 0) {
      misc.walk.begin(misc, pos_a, pos_e);
      misc.cols[0].more = misc.walk.next<kTwin>(p, misc, misc.cols[0].part);
    }
    named_bar_sync(all_bar, kSoftmaxThreads);
    for (int n_part = 0;; ++n_part) {
      Columns &cols = misc.cols[n_part & 1];
      if (!cols.more) break;
      const Part &w = cols.part;
      // what this lane's column sees; the groups of a request see the same
      if (w.b != cur_b || w.rb != cur_rb) {
        cur_b = w.b;
        cur_rb = w.rb;
        valid = column_row(p, w.rb, my_col % C::kNR, w.qlen, ct, ch);
        my_hi = valid ? min(max(p.row_len[w.q0 + ct], 0), p.max_len) : 0;
        my_lo = p.window > 0 ? max(0, my_hi - p.window) : 0;
      }
      if (wq == 0 && lane < N) {
        cols.lo[my_col] = my_lo;
        cols.hi[my_col] = my_hi;
        cols.row[my_col] = valid ? (w.q0 + ct) * p.num_heads + w.g * p.group + ch : -1;
        if (kMaps == 2) cols.lam[my_col] = valid ? p.lambda[w.g * p.group + ch] : 0.0f;
      }
      // The even parts have one buffer and the odd parts the other: a part's is
      // written again only behind the next part's barrier here.
      if (threadIdx.x == 0) {
        cols.bad[0] = cols.bad[1] = 0;
        cols.stop = *abort_flag;
      }
      named_bar_sync(all_bar, kSoftmaxThreads);
      gave_up = cols.stop;
      if (gave_up) break;
      // tokens that this group's columns all see (all_lo .. all_hi - 1), and
      // that all columns see that see anything (edge_lo .. edge_hi - 1)
      int all_lo = valid ? my_lo : 0, all_hi = valid ? my_hi : INT32_MAX;
      int edge_lo = 0, edge_hi = INT32_MAX;
      for (int c = lane; c < kNC; c += 32)
        if (cols.hi[c] > 0) {
          edge_lo = max(edge_lo, cols.lo[c]);
          edge_hi = min(edge_hi, cols.hi[c]);
        }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
        all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
        edge_lo = max(edge_lo, __shfl_xor_sync(0xffffffffu, edge_lo, o));
        edge_hi = min(edge_hi, __shfl_xor_sync(0xffffffffu, edge_hi, o));
      }
      uint64_t less[N / 2], sum[N / 2];  // minus the reference maximum, and this thread's sum, of two columns each
#pragma unroll
      for (int c = 0; c < N / 2; ++c) {
        less[c] = pair(-kLowest, -kLowest);
        sum[c] = 0;
      }
      const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), minus2 = pair(-1.0f, -1.0f);
      for (int i = w.a; i < w.e; ++i, ++t) {
        const uint32_t sb = t & 1u;
        const int tok0 = (w.tile0 + i) * kTile, tok = tok0 + row;
        wait(smem_u32(&misc.s_full[sb]), (t >> 1) & 1u);
        tc_fence_after();
        float x[N];  // scores, base 2, less the reference maximum
        const uint32_t s_addr = tmem + lane_addr + sb * kNC + col0;
        tmem_load<N>(s_addr, x);
        uint32_t sees = 0xffffffffu;  // columns that see this thread's token
        if (tok0 < all_lo || tok0 + kTile > all_hi) {
          sees = 0;
#pragma unroll
          for (int c = 0; c < N; c += 4) {
            const int4 lo = *reinterpret_cast<const int4 *>(cols.lo + col0 + c), hi = *reinterpret_cast<const int4 *>(cols.hi + col0 + c);
            sees |= (tok >= lo.x && tok < hi.x ? 1u << c : 0u) | (tok >= lo.y && tok < hi.y ? 2u << c : 0u) |
                    (tok >= lo.z && tok < hi.z ? 4u << c : 0u) | (tok >= lo.w && tok < hi.w ? 8u << c : 0u);
          }
        }
        auto relate = [&](float &top) {
#pragma unroll
          for (int c = 0; c < N; c += 2) {
            unpair(fma2(pair(x[c], x[c + 1]), scale2, less[c / 2]), x[c], x[c + 1]);
            top = fmaxf(top, fmaxf(x[c], x[c + 1]));
          }
        };
        auto hide = [&]() {  // what a column does not see is minus infinity
          if (sees == 0xffffffffu) return;
#pragma unroll
          for (int c = 0; c < N; ++c) x[c] = (sees >> c) & 1u ? x[c] : -INFINITY;
        };
        float top = -INFINITY;
        const bool rescale = i > w.a;  // there are outputs already
        hide();
        bool move = true;
        if (rescale) {
          relate(top);
          move = named_bar_red_or(grp_bar, 128, top > kLag);
          if (move) {
            tmem_load<N>(s_addr, x);
            hide();
          }
        }
        if (move) {
          float v[N];
#pragma unroll
          for (int c = 0; c < N; ++c) v[c] = x[c] * p.scale_log2;
          const float r = reduce_columns<true, N>(v, lane);
          if (lane < N) misc.red[grp][wq][lane] = r;
          named_bar_sync(grp_bar, 128);
          if (rescale) {
            wait(smem_u32(&misc.o_done[sb ^ 1u]), ((t - 1) >> 1) & 1u);
            tc_fence_after();
          }
#pragma unroll
          for (int h = 0; h < N; h += 16) {
            float f[16];
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              float l[2], now[2];
              unpair(less[(h + c) / 2], l[0], l[1]);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int at = h + c + k;
                const float best = fmaxf(fmaxf(misc.red[grp][0][at], misc.red[grp][1][at]),
                                         fmaxf(misc.red[grp][2][at], misc.red[grp][3][at]));
                now[k] = fmaxf(-l[k], best);
                f[c + k] = fast_exp2(-l[k] - now[k]);
              }
              less[(h + c) / 2] = pair(-now[0], -now[1]);
              float s0, s1;
              unpair(sum[(h + c) / 2], s0, s1);
              sum[(h + c) / 2] = pair(s0 * f[c], s1 * f[c + 1]);
            }
            if (rescale)
#pragma unroll
              for (int s = 0; s < 2 * C::kBlocks; ++s) {  // both terms of every block
                const uint32_t addr = tmem + lane_addr + C::kTmemO + kNC * s + col0 + h;
                float o[16];
                tmem_load<16>(addr, o);
#pragma unroll
                for (int c = 0; c < 16; ++c) o[c] *= f[c];
                tmem_store<16>(addr, o);
              }
          }
          relate(top);
        }
        // a probability as two bf16 terms: its rounding, and the rounding of what that left
        uint32_t hi[N / 2], lo[N / 2];
#pragma unroll
        for (int c = 0; c < N; c += 2) {
          const uint64_t pp = pair(fast_exp2(x[c]), fast_exp2(x[c + 1]));
          sum[c / 2] = add2(sum[c / 2], pp);
          float p0, p1;
          unpair(pp, p0, p1);
          const uint32_t u = pack_bf16(p0, p1);
          unpair(fma2(pair(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)), minus2, pp), p0, p1);
          hi[c / 2] = u;
          lo[c / 2] = pack_bf16(p0, p1);
        }
        // the P^T that this one overwrites has been read
        if (t >= C::kPBufs) wait(smem_u32(&misc.o_done[(t - C::kPBufs) & 1u]), ((t - C::kPBufs) >> 1) & 1u);
        const uint32_t prow = s_p + (t % C::kPBufs) * C::kPBytes + row * 128;
#pragma unroll
        for (int j = 0; j < N / 8; ++j) {
          st_shared_v4(prow + (((col0 / 8 + j) ^ (row & 7)) * 16), hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
          // the second terms: columns kNC on, of this atom of 64 or the next
          const int at = (kNC + col0) / 8 + j;
          st_shared_v4(prow + at / 8 * (kTile * 128) + (((at % 8) ^ (row & 7)) * 16), lo[4 * j], lo[4 * j + 1], lo[4 * j + 2],
                       lo[4 * j + 3]);
        }
        if (grp == 0 && (tok0 < edge_lo || tok0 + kTile > edge_hi)) {
          const bool unseen = tok < w.lo || tok >= w.hi;
          // of these only the ones in a step of 16 that the product takes
          const bool dead = unseen && (tok | 15) >= w.lo && (tok & ~15) < w.hi;
          const bool mixed = !unseen && (tok < edge_lo || tok >= edge_hi);
          if (__any_sync(0xffffffffu, dead || mixed)) {
            const uint32_t use = C::kNS * t;
            // the slots' last values have been read: until then the parity could be theirs
            if (t > 0) wait(smem_u32(&misc.o_done[sb ^ 1u]), ((t - 1) >> 1) & 1u);
#pragma unroll
            for (int s = 0; s < C::kNS; ++s) wait(full_bar(v_slot<C>(use + s)), v_par<C>(use + s));
            bool zero = dead;
            auto piece = [&](int s, int c, int j) {  // lanes in different columns of 16 bytes: no bank twice
              return s_slots + v_slot<C>(use + s) * C::kSlotBytes + (row >> 3) * (C::kCW * 1024) + c * 1024 +
                     (row & 7) * 128 + ((j + lane) & 7) * 16;
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
                  if (tok >= cols.lo[c] && tok < cols.hi[c]) atomicOr(&cols.bad[c / N], 1u << (c % N));
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
      if (threadIdx.x == 0) {  // the next part, beside the last product; read behind this result's barrier
        Columns &then = misc.cols[(n_part + 1) & 1];
        then.more = misc.walk.next<kTwin>(p, misc, then.part);
      }
      if (w.e > w.a) wait(smem_u32(&misc.o_done[(t - 1) & 1u]), ((t - 1) >> 1) & 1u);
      {
        float v[N];
#pragma unroll
        for (int c = 0; c < N; c += 2) unpair(sum[c / 2], v[c], v[c + 1]);
        const float r = reduce_columns<false, N>(v, lane);
        if (lane < N) misc.red[grp][wq][lane] = r;
      }
      if (wq == 0 && lane == 0) {
#pragma unroll
        for (int c = 0; c < N; c += 2) {
          float l0, l1;
          unpair(less[c / 2], l0, l1);
          *reinterpret_cast<float2 *>(cols.stat_m + col0 + c) = make_float2(-l0, -l1);
        }
      }
      named_bar_sync(grp_bar, 128);
      if (wq == 0 && lane < N) {
        const float l = misc.red[grp][0][lane] + misc.red[grp][1][lane] + misc.red[grp][2][lane] + misc.red[grp][3][lane];
        const bool bad = (cols.bad[grp] >> lane) & 1u;
        cols.stat_l[my_col] = l;
        // 0: the row saw nothing, and what its column of O^T holds is not looked at
        cols.inv[my_col] = l == 0.0f ? 0.0f : (bad ? __int_as_float(0x7fffffff) : 1.0f / l);
      }
      // A part that any of these threads gave up on is not stored, nor are those behind it: what a
      // wait guarded is stale, and the warps whose own waits ended multiplied it like the rest.
      gave_up = named_bar_red_or(all_bar, kSoftmaxThreads, !ok);
      if (gave_up) break;
      tc_fence_after();
      const bool whole = w.a == 0 && w.e == w.n;
      if (whole && valid && wq == 0 && lane < N) {
        const int64_t at = static_cast<int64_t>(cols.row[my_col]) * kMaps + my_col / C::kNR;
        const float l = cols.stat_l[my_col];
        p.lse[at] = l == 0.0f ? -INFINITY : (cols.stat_m[my_col] + log2f(l)) * kLn2;
      }
      // dim of this thread in block s of O^T: an M = 64 result has its rows in lanes 0-15 of each warp
      const bool has_dim = kW >= 2 || lane < 16;
      const int dim = kW >= 2 ? row : wq * 16 + lane;
      // columns c .. c + 15 of block s: the sum of both terms.  Where the first is infinite the
      // second is not looked at: a probability's second term may be zero or negative, and its
      // product with an infinite value is not that value's.
      auto load_o = [&](int s, int c, float (&o)[16]) {
        float u[16];
        const uint32_t addr = tmem + lane_addr + C::kTmemO + C::kPN * s + c;
        tmem_load<16>(addr, o);
        tmem_load<16>(addr + kNC, u);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = fabsf(o[k]) == INFINITY ? o[k] : o[k] + u[k];
      };
      if (!whole) {
        const int64_t rec = static_cast<int64_t>(blockIdx.x) * 2 + (w.a == 0 ? 1 : 0);
        if (wq == 0 && lane < N) {
          p.part_stat[rec * 2 * kNC + my_col] = cols.stat_m[my_col];
          p.part_stat[rec * 2 * kNC + kNC + my_col] = cols.stat_l[my_col];
        }
        float *po = p.part_o + rec * kNC * C::kDv;
#pragma unroll
        for (int s = 0; s < C::kBlocks; ++s)
#pragma unroll
          for (int h = 0; h < N; h += 16) {
            float o[16];
            load_o(s, col0 + h, o);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float y = cols.inv[col0 + h + c];
              store_if(has_dim && cols.row[col0 + h + c] >= 0, po + (col0 + h + c) * C::kDv + 128 * s + dim,
                       isnan(y) ? y : o[c]);
            }
          }
        if (w.a == 0) {
          const int twin = kTwin && p.may_twin ? misc.twin : 0, last = chunk_of(w.start + kOverhead + w.n - 1);
          meta = Meta{w.q0, w.qlen, w.g, w.rb, (last << twin) + static_cast<int>(blockIdx.x & twin), 1 + twin, {}};
        }
      } else if (kMaps == 1) {
#pragma unroll
        for (int s = 0; s < C::kBlocks; ++s)
#pragma unroll
          for (int h = 0; h < N; h += 16) {
            float o[16];
            load_o(s, col0 + h, o);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int at = cols.row[col0 + h + c];
              const float by = cols.inv[col0 + h + c];
              store_if(at >= 0 && has_dim, p.out + static_cast<int64_t>(at) * C::kDv + 128 * s + dim,
                       by == 0.0f ? 0.0f : o[c] * by);
            }
          }
      } else if (grp * 16 < C::kNR) {
        // 16 rows of both maps per group of warps, of the first half of them
        constexpr int R = 16;
        const int r0 = grp * R;
        float y[C::kBlocks][R], sq[R];
#pragma unroll
        for (int c = 0; c < R; ++c) sq[c] = 0.0f;
#pragma unroll
        for (int s = 0; s < C::kBlocks; ++s) {
          float o[R];
          load_o(s, r0, y[s]);
          load_o(s, C::kNR + r0, o);
#pragma unroll
          for (int c = 0; c < R; ++c) {
            const float i0 = cols.inv[r0 + c], i1 = cols.inv[C::kNR + r0 + c];
            y[s][c] = (i0 == 0.0f ? 0.0f : y[s][c] * i0) - cols.lam[r0 + c] * (i1 == 0.0f ? 0.0f : o[c] * i1);
            sq[c] += y[s][c] * y[s][c];
          }
        }
        float norm[R];
#pragma unroll
        for (int c = 0; c < R; ++c) norm[c] = 1.0f;
        if (p.gain != nullptr) {
          const float r = reduce_columns<false, R>(sq, lane);
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
            const int at = cols.row[r0 + c];
            store_if(at >= 0, p.out + static_cast<int64_t>(at) * C::kDv + 128 * s + dim,
                     cols.inv[r0 + c] == 0.0f ? 0.0f : y[s][c] * norm[c] * gain);
          }
        }
      }
      tc_fence_before();
    }
    if (threadIdx.x == 0) p.meta[blockIdx.x] = meta;
    // a unit that reaches into this chunk is not merged: a negative sum tells
    if (gave_up && wq == 0 && lane < N) p.part_stat[(static_cast<int64_t>(blockIdx.x) * 2 * 2 + 1) * kNC + my_col] = -1.0f;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaK) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0 && misc.abort) {
    // copies in flight land before the memory is given up
    const volatile int never = 0;
    for (int i = 0; i < C::kSlots; ++i)
      if (misc.armed[i]) mbar_wait(smem_u32(&misc.full[i]), misc.armed[i] - 1, &never, p.drain_budget);
    for (int i = 0; i < C::kQBufs; ++i)
      if (misc.q_armed[i]) mbar_wait(smem_u32(&misc.q_full[i]), misc.q_armed[i] - 1, &never, p.drain_budget);
  }
}

// The launches of a call: W chunks a token, nc columns (mla_grouped_plain.cu,
// mla_grouped_differential.cu).
mla_status launch_grouped(int W, int nc, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const Params &p,
                          int grid, bool merge, cudaStream_t stream);
mla_status launch_differential(int W, int nc, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const Params &p,
                               int grid, bool merge, cudaStream_t stream);

}  // namespace grouped
}  // namespace mla
