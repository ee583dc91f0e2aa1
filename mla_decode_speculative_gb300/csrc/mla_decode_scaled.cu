// mla_decode_scaled.cu -- absorbed-form MLA decode / causal verify over a paged
// e4m3 cache with one scale per block of G cache rows
// (mla_decode_verify_scaled).
//
// For query row r = (verify row t, head h) of request b and its visible tokens
// j < row_len[t], token j in cache row n with scale a_j = kv_scales[n / G]:
//   s_j = sm_scale * a_j * <q[r], code_j>, out = sum softmax(s)_j a_j code_j[0:512],
//   lse = ln sum e^{s_j}.
//
// Both products run on the 8-bit codes as they lie in the cache
// (tcgen05 kind::f8f6f4), nothing is expanded to 16 bits:
//  * q is split exactly: each row is scaled by a power of two so that its
//    largest element lies in [128, 256); q1 = e4m3(q), and what is left, at
//    most half a step of q1, has no more than four significant bits, so
//    q2 = e4m3(32 (q - q1)) holds it (elements below 2^-14 of the row's
//    largest keep an absolute 2^-22 of it).  s = (q1 + q2 / 32) . code.
//  * a probability times its token's scale is written as two e5m2 terms, the
//    second the rounded remainder of the first: at most 2^-7 of itself off,
//    over a range of 2^28 below the row's largest (e4m3 terms would lose the
//    many small weights beside one large one).  The sums of the weights before
//    and after this rounding correct the row's mean, so one visible token, or
//    equal ones, come out exact.
//  * The scale joins the score,
//      w_j = 2^(s_j log2e + log2 a_j - m),  l = sum w_j / a_j,  out = sum w_j code_j / l,
//    so the running reference m bounds the weights whatever the scales are.
//    log2 a_j and 1 / a_j come from a warp of their own, once per token.
//
// Work: (row view, request, block of up to 64 query rows) units in 96-token
// tiles.  The tiles of all units plus a few overhead positions per unit
// (part_cost), end to end, are cut into one equal chunk per CTA (one CTA per
// SM), never more than S chunks per unit; a chunk's part of a unit is one of its
// split-K segments (S = 1: whole units, by the chunk their first tile lies in).
// Every CTA sums up the positions for itself and its producer walks on from its
// chunk's first unit, so nothing is tabulated and any number of units fits.
//
// Operands.  q1 and q2 of 16 rows share a quarter of the 128 TMEM lanes (lane
// 32 w + i: q1 of row 16 w + i, lane 32 w + 16 + i: its q2), 144 columns, as
// the A operand of S[128, 96 tok] = Q . K^T: with A in TMEM no query is held
// in shared memory, which takes four whole tiles instead.  A tile is four
// 128-dim chunks [96 tok x 128 B] (128-byte swizzle) and the rope chunk
// [96 tok x 64 B] (64-byte swizzle): the B operand of S = Q K^T as it lies, and
// of O^T[4 x 128 dims, 64 rows] += V^T P^T the A operand in the other major.
// P^T, the B operand there, is 32-token blocks [64 rows x 32 B] (32-byte
// swizzle): the first term's blocks replace the tile's rope chunk, which S has
// used by then, the second term's have 6 KB of their own.
// TMEM: Q 0-143, O^T 144-399, S 400-495; 96 tokens is the widest S that the
// columns left by Q and O^T hold.
//
// Warps.  0-7: queries into TMEM, softmax, epilogue; two groups of four take
// turns with the tiles, so one group's loads and exponentials run beside the
// other's (all eight on each tile: 2665 cycles a tile, in turns 2390).  8: work
// and TMA.  9: S = Q K^T, 10: O^T += V^T P^T, an elected thread each, so that
// neither waits for the other's barriers.  11: the tiles' scales.  S and the
// second term of P^T have one buffer each: tile g + 1's S is issued when tile
// g's has been read, its second term is written when tile g's products are done.
//
// What bounds it.  An instruction of 128 x N x 32 takes 53-63 cycles for N up to
// 96 and 64 at N = 128 (measured), a tile's 18 + 24 about 2500 if nothing
// overlapped; the steady state is 2390 cycles a tile, 1.25 us, against 1.24 us for
// the SM's share of the HBM rate (55 KB at 6.76 TB/s / 152).  16 requests of
// 131,072 tokens take 255 us (4.7 TB/s) and run at the power limit.  Short calls
// are latency: about 10 us from the call's start to the first S (lengths and
// split 1.8, finding the part 1.9, its queries 1.4 and their two terms 2.3), 3 us
// from the last tile to the partial output, then the merge kernel; 32 requests of
// 1,024 to 8,192 tokens take 39 us, 13 of them at the HBM rate.  The loops are
// kept small: the instruction cache holds about 32 KB for four loops that run at
// once.
//
// Every wait is bounded; one that runs out records MLA_DEV_WAIT_TIMEOUT, all
// roles drain without skipping a barrier, TMEM is freed and the kernel returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "mla_internal.h"
#include "mla_ptx.cuh"

namespace mla {
namespace {

constexpr int kTile = 96;          // tokens of a tile
constexpr int kStages = 4;         // tiles in shared memory
constexpr int kRows = 64;          // query rows of a unit
constexpr int kAtom = 1024;                       // 128 dims of eight tokens
constexpr int kGroup = 4 * kAtom;                 // 512 dims of eight tokens
constexpr int kRopeOff = kTile / 8 * kGroup;      // rope chunk, then the first term of P^T
constexpr int kStageBytes = kTile * 576;
constexpr int kQPitch = 1152 + 16;  // a query row there: rows a quarter of the banks apart
constexpr int kPBlock = kRows * 32;               // 32 tokens of one term of P^T
constexpr int kOffP2 = kStages * kStageBytes;     // second term of P^T
constexpr int kOffMisc = kOffP2 + 3 * kPBlock;
constexpr int kSoftWarps = 8, kSoftThreads = 256;
constexpr int kGroupWarps = 4, kGroupThreads = 128;  // two groups take turns with the tiles
constexpr int kTmaWarp = 8, kQkWarp = 9, kPvWarp = 10, kScaleWarp = 11;
constexpr int kThreads = 384;
constexpr uint32_t kTmemQ = 0, kTmemO = 144, kTmemS = 400, kTmemCols = 512;
constexpr int kWorkRing = 3;
constexpr float kThreshold = 3.0f;   // the reference moves when a weight exceeds 2^3 of it
constexpr float kTop = 11.0f;        // a weight at the reference is held as 2^11: at most 2^14 < 57344
constexpr float kInvTop = 4.8828125e-4f;  // 2^-kTop
constexpr float kLn2 = 0.69314718055994530942f;
constexpr uint32_t kBarSoft = 1;     // named barriers: the softmax warps, and 2, 3 their groups

// A part of a unit, as the producer publishes it.
struct Part {
  int stop;                 // 1: no more work
  int b;                    // view * B + request
  int rb, seg, fill_hi;     // slots seg + 1 .. fill_hi - 1 of the unit get no part: mark them empty
                            // seg -1: the unit's only part, which writes the outputs itself
  int q_row, row_base, n_rows;
  int seg_lo, seg_hi, n_tiles;
};

struct Misc {
  uint64_t full[kStages], empty[kStages];
  uint64_t s_free, p2_full, q_here, q_read, q_full, fin_qk, fin_pv;
  // by the tile's parity, so by softmax group: a group looks at every other tile,
  // and one barrier's phases look alike two tiles apart
  uint64_t s_full[2], p1_full[2], o_done[2], turn[2], sc_full[2], sc_free[2];
  uint64_t work_full[kWorkRing], work_empty[kWorkRing];
  uint32_t tmem_base;
  int abort;
  int stop[2];
  int first_vb, first_pos;  // the chunk's first (view, request) and its first position
  alignas(16) float sc[2][kTile], lg[2][kTile], rc[2][kTile];  // a tile's scales, their logarithms and reciprocals
  Part part[kWorkRing];
  float ref[kRows];         // running reference of each row (log2 units)
  float red[2][kRows];      // sums of the setup, the queries' maxima, the rows' sums
  // What a group's new references scale O^T by.  Between the parts' tiles: [0] the rows' lost weights,
  // [1] what the epilogue scales O^T by (group 1 writes it again only after group 0's first tile).
  alignas(16) float alpha[2][kRows];
};
constexpr int kSmemBytes = kOffMisc + static_cast<int>(sizeof(Misc)) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kStageBytes % 1024 == 0 && kRopeOff % 1024 == 0 && kOffP2 % 1024 == 0, "swizzle-atom alignment");
static_assert(kRows * kQPitch <= 2 * kStageBytes, "the first part's queries fit two stages");
static_assert(3 * kPBlock <= kTile * 64, "a term of P^T fits the rope chunk");
static_assert(2 * (kThreads / 32) <= 2 * kRows, "the setup's sums fit red");

struct Params {
  const __nv_bfloat16 *q;
  const float *scales;
  const int32_t *qo_indptr, *row_len, *subpage_table;
  __nv_bfloat16 *segm_out;
  float *segm_max, *segm_sum;
  __nv_bfloat16 *out;
  float *lse;
  int *err;
  int64_t num_cache_rows;
  long long wait_budget, drain_budget;
  float score_scale;        // sm_scale * log2(e)
  int subpage_stride, page_size, log_g, num_heads, num_segments, row_blocks, num_reqs, num_views, max_qlen, num_rows,
      max_len, q_aligned;
};

__device__ __forceinline__ void note(int *err, int code) { atomicCAS(err, 0, code); }

// A scale's logarithm (within 2^-22 of it, so a weight within 2^-15) and reciprocal (within an ulp): with
// log2f and a division the loop of the warp that makes them costs the others 2% in the instruction cache.
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D (+)= A . B^T, kind::f8f6f4; A in TMEM / in shared memory.
__device__ __forceinline__ void mma8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// One lane of a converged warp.  The compiler knows that a branch on this has a
// single thread, and keeps descriptors in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t y;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(y));
  return y != 0;
}
// Shared-memory matrix descriptor (fields as sdesc_sw128's); layout: 2 = 128-,
// 4 = 64-, 6 = 32-byte swizzle; sbo: bytes from one 8-row group to the next.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t sbo, uint64_t layout) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) |
         (layout << 61);
}
// Instruction descriptor: D f32; A e4m3; B e4m3 (0) or e5m2 (1); A's major-ness.
__host__ __device__ constexpr uint32_t idesc_f8(int n, int b_fmt, int a_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_fmt) << 10) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

// 32 lanes x 16 columns (thread i: lane base + i), without the wait.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two floats at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, y;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 y, a, b;\n\t"
      "mov.b64 {%0, %1}, y;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, y;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 y, a, b;\n\t"
      "mov.b64 {%0, %1}, y;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, c, y;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 y, a, b, c;\n\tmov.b64 {%0, %1}, y;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}

// A wait that did not pass at once, kept out of line: the kernel's loops have to
// stay small enough for the instruction caches.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, int *abort, long long budget, int *err) {
  if (mbar_wait(bar, parity, abort, budget)) return true;
  *const_cast<volatile int *>(abort) = 1;
  note(err, MLA_DEV_WAIT_TIMEOUT);
  return false;
}

__device__ __forceinline__ void load8(const float *ptr, float (&v)[8]) {  // 16-byte aligned
  const float4 lo = reinterpret_cast<const float4 *>(ptr)[0], hi = reinterpret_cast<const float4 *>(ptr)[1];
  v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
  v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
}

// A thread's 48 scores (six runs of eight tokens, 16 apart) to weights against
// the reference: the sums (rc: the tokens' 1 / scale), and the weights' two e5m2
// terms.  A weight goes through f16 (2^-12 of itself): there e5m2 is the upper
// byte, so a term's value is its codes moved up and the remainder is exact.
// kWide: a run has one scale.
template <bool kWide>
__device__ __forceinline__ void weigh(const float2 (&x)[24], const float *rc, float ref, float &l_t, float &w_sum,
                                      float &w_lost, uint32_t (&p1)[12], uint32_t (&p2)[12]) {
  float w_t = 0.0f, l_w = 0.0f;
  float2 l_2 = make_float2(0.0f, 0.0f);
  __half2 lost = __float2half2_rn(0.0f);
  const float2 neg = make_float2(-ref, -ref);
#pragma unroll
  for (int q = 0; q < 6; ++q) {
    float2 run = make_float2(0.0f, 0.0f);
    float r[8];
    if (kWide) r[0] = rc[16 * q];
    else load8(rc + 16 * q, r);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float2 d = add2(x[4 * q + u], neg);
      const float2 e = make_float2(ex2(d.x), ex2(d.y));
      run = add2(run, e);
      if (!kWide) l_2 = fma2(e, make_float2(r[2 * u], r[2 * u + 1]), l_2);
      const __half2 w = __floats2half2_rn(e.x, e.y);
      const uint32_t c1 = __nv_cvt_halfraw2_to_fp8x2(w, __NV_SATFINITE, __NV_E5M2);
      const uint32_t v1 = __byte_perm(c1, 0, 0x1404);
      const __half2 rest = __hsub2(w, *reinterpret_cast<const __half2 *>(&v1));
      const uint32_t c2 = __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E5M2);
      const uint32_t v2 = __byte_perm(c2, 0, 0x1404);
      lost = __hadd2(lost, __hsub2(rest, *reinterpret_cast<const __half2 *>(&v2)));
      p1[2 * q + u / 2] = (u & 1) ? __byte_perm(p1[2 * q + u / 2], c1, 0x5410) : c1;
      p2[2 * q + u / 2] = (u & 1) ? __byte_perm(p2[2 * q + u / 2], c2, 0x5410) : c2;
    }
    const float both = run.x + run.y;
    if (kWide) l_w = fmaf(both, r[0], l_w);
    w_t += both;
  }
  l_t = (kWide ? l_w : l_2.x + l_2.y) * kInvTop;
  w_sum += w_t;
  w_lost += __low2float(lost) + __high2float(lost);
}

__device__ __forceinline__ void ld_global_32(const uint4 *ptr, uint4 &a, uint4 &b) {  // 32-byte aligned
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(ptr)
               : "memory");
}
__device__ __forceinline__ void copy_to_smem(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void prefetch_l2(const void *ptr, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(ptr), "r"(bytes) : "memory");
}

// ---- work

// Longest visible length of a request's rows in a view; 0 when its qo_indptr
// entries are inconsistent.
__device__ __forceinline__ int request_len(const Params &p, int v, int b, int &qlen) {
  const int q0 = p.qo_indptr[b], q1 = p.qo_indptr[b + 1];
  qlen = 0;
  if (q0 < 0 || q1 < q0 || q1 > p.num_rows || q1 - q0 > p.max_qlen) return 0;
  qlen = q1 - q0;
  const int32_t *rl = p.row_len + static_cast<int64_t>(v) * p.num_rows;
  int len = 0;
  for (int t0 = q0; t0 < q1; t0 += 8) {
    int l[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) l[k] = t0 + k < q1 ? rl[t0 + k] : 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) len = max(len, min(max(l[k], 0), p.max_len));
  }
  return len;
}
// What a part costs besides its tiles (queries, sums, epilogue), in tiles, by the
// request's query rows: the second part of a CTA takes 11.7 us at 64 rows and 7.6
// at 12 to 36, a tile 1.3 to 1.6.  With one for all, 8 against 6 is 42.2 against
// 43.4 us for 32 requests of 64 rows, but 85.2 against 83.6 for 64 of 12 to 36.
__host__ __device__ __forceinline__ int part_cost(int rows) { return 4 + (rows < kRows ? rows : kRows) / 16; }
// Positions of a (view, request): for each of its row blocks a part's cost and
// its tiles, nothing when no row sees a token.
__device__ __forceinline__ int positions(const Params &p, int vb, int &tiles) {
  int qlen;
  const int len = request_len(p, vb / p.num_reqs, vb % p.num_reqs, qlen);
  tiles = (len + kTile - 1) / kTile;
  const int rows = qlen * p.num_heads;
  return tiles > 0 ? (rows + kRows - 1) / kRows * (tiles + part_cost(rows)) : 0;
}

struct Split {
  int total, n_chunks, chunk, lo, hi;  // positions; this CTA's chunk [lo, hi)
};
__device__ __forceinline__ int chunk_of(const Split &s, int x) {
  return static_cast<int>((static_cast<long long>(x + 1) * s.n_chunks - 1) / s.total);
}

// The whole CTA: total positions, the chunk of this CTA, and the (view,
// request) in which it starts (misc.first_vb, misc.first_pos).
__device__ Split make_split(const Params &p, Misc &misc) {
  const int n_vb = p.num_views * p.num_reqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  int *warp_sum = reinterpret_cast<int *>(misc.red), *warp_max = warp_sum + kWarps;
  int mine = 0, pos = 0, t_max = 0;
  for (int vb = tid; vb < n_vb; vb += kThreads) {
    int t;
    pos = positions(p, vb, t);
    mine += pos;
    t_max = max(t_max, t);
  }
  const int sum = __reduce_add_sync(0xffffffffu, mine);
  t_max = __reduce_max_sync(0xffffffffu, t_max);
  if (lane == 0) {
    warp_sum[warp] = sum;
    warp_max[warp] = t_max;
  }
  __syncthreads();
  Split s;
  s.total = 0;
  t_max = 0;
  int before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    s.total += warp_sum[w];
    t_max = max(t_max, warp_max[w]);
  }
  // chunks of at least `need` tiles meet a unit at most S times
  const int S = p.num_segments, need = S > 1 ? max((t_max + S - 2) / (S - 1), 1) : 1;
  s.n_chunks = s.total > 0 ? min(static_cast<int>(gridDim.x), max(s.total / need, 1)) : 1;
  s.chunk = blockIdx.x;
  s.lo = static_cast<int>(static_cast<long long>(s.chunk) * s.total / s.n_chunks);
  s.hi = static_cast<int>(static_cast<long long>(s.chunk + 1) * s.total / s.n_chunks);
  if (s.chunk == s.n_chunks - 1) s.hi = s.total + 1;  // units without tiles at the very end
  // the one with first position < lo <= end, or the very first: by one scan when
  // every thread has one (view, request), else by scans of kThreads
  int carry = 0;
  for (int v0 = 0; v0 < n_vb && s.chunk < s.n_chunks; v0 += kThreads) {
    const int vb = v0 + tid;
    if (n_vb > kThreads) {
      int t;
      pos = vb < n_vb ? positions(p, vb, t) : 0;
      const int part = __reduce_add_sync(0xffffffffu, pos);
      __syncthreads();
      if (lane == 0) warp_sum[warp] = part;
      __syncthreads();
      before = carry;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        carry += warp_sum[w];
      }
    }
    int x = vb < n_vb ? pos : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int end = before + x, start = end - (vb < n_vb ? pos : 0);
    if (vb < n_vb && end >= s.lo && (vb == 0 || start < s.lo)) {
      misc.first_vb = vb;
      misc.first_pos = start;
    }
  }
  return s;
}

template <bool kWide>
__global__ void __launch_bounds__(kThreads, 1)
    mla_decode_scaled_kernel(const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_r,
                             const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc &misc = *reinterpret_cast<Misc *>(smem + kOffMisc);
  const uint32_t s_base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.num_segments, P = p.page_size;

  if (warp == kQkWarp) {
    tmem_alloc(smem_u32(&misc.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&misc.full[i]), 1);
      mbar_init(smem_u32(&misc.empty[i]), 1);
    }
    mbar_init(smem_u32(&misc.s_free), kGroupWarps);
    mbar_init(smem_u32(&misc.p2_full), kGroupWarps);
    mbar_init(smem_u32(&misc.q_here), 1);
    mbar_init(smem_u32(&misc.q_read), 1);
    mbar_init(smem_u32(&misc.q_full), kSoftWarps);
    mbar_init(smem_u32(&misc.fin_qk), 1);
    mbar_init(smem_u32(&misc.fin_pv), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&misc.s_full[i]), 1);
      mbar_init(smem_u32(&misc.p1_full[i]), kGroupWarps);
      mbar_init(smem_u32(&misc.o_done[i]), 1);
      mbar_init(smem_u32(&misc.turn[i]), kGroupWarps);
      mbar_init(smem_u32(&misc.sc_full[i]), 1);
      mbar_init(smem_u32(&misc.sc_free[i]), kGroupWarps);
    }
    for (int i = 0; i < kWorkRing; ++i) {
      mbar_init(smem_u32(&misc.work_full[i]), 1);
      mbar_init(smem_u32(&misc.work_empty[i]), kSoftWarps + 3);
    }
    misc.abort = 0;
    misc.first_vb = misc.first_pos = 0;
    fence_mbar_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_r);
  }
  grid_dep_wait();
  grid_dep_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Split split = make_split(p, misc);
  __syncthreads();
  const uint32_t tmem = misc.tmem_base;
  volatile int *abort_flag = &misc.abort;
  const long long budget = p.wait_budget;
  bool ok = true;
  auto wait = [&](const uint64_t &bar, uint32_t parity) {
    if (ok && !mbar_try_wait(smem_u32(&bar), parity & 1u))
      ok = wait_long(smem_u32(&bar), parity & 1u, &misc.abort, budget, p.err);
    return ok;
  };

  if (warp == kTmaWarp) {
    // ================================================ work and tile copies
    const uint64_t policy = l2_policy_evict_first();
    const int run = min(P, 32), lg_p = 31 - __clz(P);  // rope rows of a copy: one page, or 32 of one
    // A lane's copy of a tile: 512 dims of eight tokens, or the rope dims of `run` tokens.
    const bool is_v = lane < kTile / 8;
    const int c_tok = is_v ? 8 * lane : (lane - kTile / 8) * run;
    const uint32_t c_dst = s_base + (is_v ? lane * kGroup : kRopeOff + c_tok * 64);
    bool q_staged = false;  // the first part's queries are in the third and fourth stage
    uint32_t armed = 0, armed_par = 0;  // stages with a copy possibly in flight (for the exit path)
    uint32_t g = 0;
    int vb = misc.first_vb, rb = 0, pos = misc.first_pos, u_pos = pos;
    int tiles = 0, len = 0, q0 = 0, qlen = 0, my_len = 0, loaded = -1;
    bool clipped = false, bad = false;
    const int n_vb = p.num_views * p.num_reqs;
    for (uint32_t k = 0;; ++k) {
      Part &e = misc.part[k % kWorkRing];
      if (lane == 0) wait(misc.work_empty[k % kWorkRing], (k / kWorkRing) ^ 1u);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      bool found = false;
      int t_lo = 0, t_hi = 0, seg = -1, fill_hi = S, unit_len = 0;
      while (ok && split.chunk < split.n_chunks && vb < n_vb) {
        const int v = vb / p.num_reqs, b = vb - v * p.num_reqs;
        if (loaded != vb) {  // the request's rows: lane t holds the length of row t (t < 32)
          q0 = p.qo_indptr[b];
          const int q1 = p.qo_indptr[b + 1];
          bad = q0 < 0 || q1 < q0 || q1 > p.num_rows || q1 - q0 > p.max_qlen;
          qlen = bad ? 0 : q1 - q0;
          const int32_t *rl = p.row_len + static_cast<int64_t>(v) * p.num_rows + q0;
          my_len = lane < qlen ? rl[lane] : 0;
          len = 0;
          clipped = false;
          for (int t = lane; t < qlen; t += 32) {
            const int l = t == lane ? my_len : rl[t];
            clipped |= l > p.max_len;
            len = max(len, min(max(l, 0), p.max_len));
          }
          len = __reduce_max_sync(0xffffffffu, len);
          clipped = __any_sync(0xffffffffu, clipped);
          tiles = (len + kTile - 1) / kTile;
          loaded = vb;
          if (lane == 0 && bad) note(p.err, MLA_DEV_BAD_INDPTR);
          if (lane == 0 && clipped) note(p.err, MLA_DEV_LEN_BOUND);
          // row blocks that end before the chunk
          if (tiles > 0 && u_pos < split.lo) {
            rb = (split.lo - u_pos) / (tiles + part_cost(qlen * p.num_heads));
            u_pos += rb * (tiles + part_cost(qlen * p.num_heads));
          }
        }
        const int blocks = (qlen * p.num_heads + kRows - 1) / kRows;
        if (rb >= blocks) {
          ++vb;
          rb = 0;
          continue;
        }
        if (u_pos >= split.hi) break;
        const int here = u_pos, start = here + (tiles > 0 ? part_cost(qlen * p.num_heads) : 0), end = start + tiles;
        if (start >= split.hi) break;
        u_pos = end;
        const int this_rb = rb++;
        if (tiles == 0) {
          if (here < split.lo) continue;
        } else if (S == 1) {
          if (start < split.lo) continue;
          t_hi = tiles;
        } else {
          const int lo = max(split.lo, start), hi = min(split.hi, end);
          if (lo >= hi) continue;
          t_lo = lo - start;
          t_hi = hi - start;
          if (t_lo > 0 || t_hi < tiles) seg = split.chunk - chunk_of(split, start);
          fill_hi = end <= split.hi ? S : seg + 1;
        }
        found = true;
        const int row_begin = this_rb * kRows;
        const int n_rows = min(kRows, qlen * p.num_heads - row_begin);
        unit_len = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = lane + 32 * h, t = (row_begin + c) / p.num_heads;
          int l = __shfl_sync(0xffffffffu, my_len, t < 32 ? t : 0);
          if (t >= 32 && c < n_rows) l = p.row_len[static_cast<int64_t>(v) * p.num_rows + q0 + t];
          if (c < n_rows) unit_len = max(unit_len, min(max(l, 0), p.max_len));
        }
        // a token that only other units' rows see is not in this unit's tiles: its code may be a NaN
        unit_len = __reduce_max_sync(0xffffffffu, unit_len);
        t_hi = min(t_hi, (unit_len + kTile - 1) / kTile);
        t_lo = min(t_lo, t_hi);
        if (lane == 0) {
          e.stop = 0;
          e.b = vb;
          e.rb = this_rb;
          e.seg = seg;
          e.fill_hi = fill_hi;
          e.q_row = q0 * p.num_heads + row_begin;
          e.row_base = (v * p.num_rows + q0) * p.num_heads + row_begin;
          e.n_rows = n_rows;
          e.seg_lo = t_lo * kTile;
          e.seg_hi = min(t_hi * kTile, unit_len);
          e.n_tiles = t_hi - t_lo;
          const __nv_bfloat16 *q = p.q + static_cast<int64_t>(e.q_row) * 576;
          if (t_hi > t_lo) prefetch_l2(q, n_rows * 1152);
        }
        if (k == 0) q_staged = t_hi > t_lo;
        break;
      }
      __syncwarp();
      if (!found) {
        if (lane == 0) {
          e.stop = 1;
          mbar_arrive(smem_u32(&misc.work_full[k % kWorkRing]));
        }
        break;
      }
      if (lane == 0) mbar_arrive(smem_u32(&misc.work_full[k % kWorkRing]));
      if (t_hi == t_lo) continue;
      const int seg_lo = t_lo * kTile, seg_hi = min(t_hi * kTile, unit_len);
      const int32_t *pages = p.subpage_table + static_cast<int64_t>(vb) * p.subpage_stride;
      const int last_page = (seg_hi - 1) >> lg_p;
      int win = seg_lo >> lg_p;         // lane l holds the id of page win + l
      int32_t win_id = win + lane <= last_page ? pages[win + lane] : -1;
#pragma unroll 1
      for (int tok0 = seg_lo; tok0 < seg_hi; tok0 += kTile, ++g) {
        const int n_valid = min(kTile, seg_hi - tok0);
        const uint32_t st = g % kStages;
        if ((tok0 + n_valid - 1) >> lg_p >= win + 32) {
          win = tok0 >> lg_p;
          win_id = win + lane <= last_page ? pages[win + lane] : -1;
        }
        if (q_staged && g == 2 && !__all_sync(0xffffffffu, wait(misc.q_read, 0))) break;
        if (!__all_sync(0xffffffffu, wait(misc.empty[st], (g / kStages) ^ 1u))) break;
        const uint32_t bar = smem_u32(&misc.full[st]);
        if (lane == 0) mbar_arrive_expect_tx(bar, ((n_valid + 7) & -8) * 512 + ((n_valid + run - 1) & -run) * 64);
        __syncwarp();
        const bool mine = c_tok < n_valid;
        const int t = tok0 + c_tok;
        const int32_t id = __shfl_sync(0xffffffffu, win_id, mine ? (t >> lg_p) - win : 0);
        if (mine) {
          int32_t row = static_cast<int32_t>(p.num_cache_rows);  // past the last row: zeros
          if (id < 0 || (static_cast<int64_t>(id) + 1) << lg_p > p.num_cache_rows) note(p.err, MLA_DEV_BAD_SUBPAGE);
          else row = (id << lg_p) + (t & (P - 1));
          if (is_v) tma_load_3d(c_dst + st * kStageBytes, &tm_v, bar, 0, row, 0, policy);
          else tma_load_2d(c_dst + st * kStageBytes, &tm_r, bar, 512, row, policy);
        }
        armed |= 1u << st;
        armed_par = (armed_par & ~(1u << st)) | (((g / kStages) & 1u) << st);
      }
      ok = __all_sync(0xffffffffu, ok) != 0;
    }
    if (lane == 0 && (!ok || *abort_flag)) {  // let the copies land before the memory is released
      const volatile int never = 0;
      for (int st = 0; st < kStages; ++st)
        if (armed & (1u << st)) mbar_wait(smem_u32(&misc.full[st]), (armed_par >> st) & 1u, &never, p.drain_budget);
    }
  } else if (warp == kQkWarp) {
    // ================================================ S = Q K^T
    if (elect_one()) {
      constexpr uint32_t id_qk = idesc_f8(kTile, 0, 0);
      const uint64_t d_k = sdesc(s_base, kGroup, 2), d_rope = sdesc(s_base + kRopeOff, 512, 4);
      uint32_t g = 0, kq = 0;
      for (uint32_t k = 0; wait(misc.work_full[k % kWorkRing], k / kWorkRing); ++k) {
        const Part &e = misc.part[k % kWorkRing];
        if (e.stop) break;
        const int n_tiles = e.n_tiles;
        mbar_arrive(smem_u32(&misc.work_empty[k % kWorkRing]));
        if (n_tiles > 0 && !wait(misc.q_full, kq++)) break;
        for (int i = 0; i < n_tiles && ok; ++i, ++g) {
          const uint32_t st = g % kStages;
          if (!wait(misc.full[st], g / kStages)) break;
          if (g > 0 && !wait(misc.s_free, g - 1)) break;
          tc_fence_after();
          const uint64_t off = static_cast<uint64_t>(st) * (kStageBytes >> 4);
#pragma unroll 1
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma8_ts(tmem + kTmemS, tmem + kTmemQ + 32 * c + 8 * i, d_k + off + c * (kAtom >> 4) + 2 * i, id_qk,
                      (c | i) > 0);
          mma8_ts(tmem + kTmemS, tmem + kTmemQ + 128, d_rope + off, id_qk, 1u);
          mma8_ts(tmem + kTmemS, tmem + kTmemQ + 136, d_rope + off + 2, id_qk, 1u);
          umma_commit(smem_u32(&misc.s_full[g & 1u]));
        }
      }
      umma_commit(smem_u32(&misc.fin_qk));  // every product issued so far has retired
      const volatile int never = 0;
      mbar_wait(smem_u32(&misc.fin_qk), 0, &never, p.drain_budget);
    }
  } else if (warp == kPvWarp) {
    // ================================================ O^T += V^T P^T
    if (elect_one()) {
      constexpr uint32_t id_pv = idesc_f8(kRows, 1, 1);
      // V^T: a 128-byte row holds all of M, so only the step between 8-token groups counts
      const uint64_t d_v = sdesc(s_base, kGroup, 2) | (static_cast<uint64_t>(kAtom >> 4) << 16);
      const uint64_t d_p1 = sdesc(s_base + kRopeOff, 256, 6), d_p2 = sdesc(s_base + kOffP2, 256, 6);
      uint32_t g = 0;
      for (uint32_t k = 0; wait(misc.work_full[k % kWorkRing], k / kWorkRing); ++k) {
        const Part &e = misc.part[k % kWorkRing];
        if (e.stop) break;
        const int n_tiles = e.n_tiles, tokens = e.seg_hi - e.seg_lo;
        mbar_arrive(smem_u32(&misc.work_empty[k % kWorkRing]));
        for (int i = 0; i < n_tiles && ok; ++i, ++g) {
          const uint32_t st = g % kStages;
          const uint64_t off = static_cast<uint64_t>(st) * (kStageBytes >> 4);
          const int n32 = (min(kTile, tokens - i * kTile) + 31) / 32;
          // The first term's products need not wait for the second term, whose buffer the tile
          // before has until its own are done.
#pragma unroll 1
          for (int term = 0; term < 2; ++term) {
            if (!wait(term == 0 ? misc.p1_full[g & 1u] : misc.p2_full, term == 0 ? g >> 1 : g)) break;
            tc_fence_after();
            uint64_t dv = d_v + off, dp = term == 0 ? d_p1 + off : d_p2;
#pragma unroll 1
            for (int kk = 0; kk < n32; ++kk, dv += 4 * kGroup >> 4, dp += kPBlock >> 4) {
#pragma unroll
              for (int blk = 0; blk < 4; ++blk)
                mma8_ss(tmem + kTmemO + blk * kRows, dv + blk * (kAtom >> 4), dp, id_pv, (term | kk | i) > 0);
            }
          }
          if (!ok) break;
          umma_commit(smem_u32(&misc.o_done[g & 1u]));
          umma_commit(smem_u32(&misc.empty[st]));
        }
      }
      umma_commit(smem_u32(&misc.fin_pv));
      const volatile int never = 0;
      mbar_wait(smem_u32(&misc.fin_pv), 0, &never, p.drain_budget);
    }
  } else if (warp == kScaleWarp) {
    // ================================================ the tiles' scales
    uint32_t g = 0;
    for (uint32_t k = 0;; ++k) {
      const uint32_t ws = k % kWorkRing;
      wait(misc.work_full[ws], k / kWorkRing);
      if (!__all_sync(0xffffffffu, ok) || misc.part[ws].stop) break;
      const Part &e = misc.part[ws];
      const int seg_lo = e.seg_lo, seg_hi = e.seg_hi, n_tiles = e.n_tiles;
      const int32_t *pages = p.subpage_table + static_cast<int64_t>(e.b) * p.subpage_stride;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&misc.work_empty[ws]));
      // scale of token t, one tile ahead of its use; a page outside the cache is zeros
      const int lg_p = 31 - __clz(P);
      auto load = [&](int t) {
        float a = 1.0f;
        if (t < seg_hi) {
          const int id = pages[t >> lg_p];
          if (id >= 0 && (static_cast<int64_t>(id) + 1) << lg_p <= p.num_cache_rows)
            a = p.scales[((id << lg_p) + (t & (P - 1))) >> p.log_g];
        }
        return fminf(fmaxf(a, 7.888609052210118e-31f), 1.329227995784916e36f);  // within [2^-100, 2^120]
      };
      float a[3];
#pragma unroll
      for (int j = 0; j < 3; ++j) a[j] = load(seg_lo + lane + 32 * j);
#pragma unroll 1
      for (int i = 0; i < n_tiles; ++i, ++g) {
        float next[3];
#pragma unroll
        for (int j = 0; j < 3; ++j) next[j] = load(seg_lo + (i + 1) * kTile + lane + 32 * j);
        wait(misc.sc_free[g & 1u], (g >> 1) ^ 1u);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          misc.sc[g & 1u][lane + 32 * j] = a[j];
          misc.lg[g & 1u][lane + 32 * j] = lg2(a[j]);
          misc.rc[g & 1u][lane + 32 * j] = rcp(a[j]);
          a[j] = next[j];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&misc.sc_full[g & 1u]));
      }
    }
  } else {
    // ================================================ queries, softmax, epilogue
    const int wq = warp & 3, h = warp >> 2, term = lane >> 4;
    const int row = 16 * wq + (lane & 15);       // this thread's query row
    const uint32_t bar_group = kBarSoft + 1 + h;
    const uint32_t lanes = static_cast<uint32_t>(32 * wq) << 16;
    const bool owner = h == 0 && term == 0;      // of the row's statistics
    const float w_mine = term ? 0.03125f : 1.0f, w_other = term ? 1.0f : 0.03125f;
    uint32_t g0 = 0;                             // tiles of the parts before
    float q_scale = 1.0f;                        // q = q_scale * (q1 + q2 / 32)
    bool spoilt = false;                        // the query row is not finite

    // A part's queries into TMEM.  Thread: 144 dims of its row, from
    // 288 h + 144 term; both terms of them, one of which goes to the partner lane.
    // A CTA's first queries are copied to the stages that its tiles reach last:
    // read from global memory, 32 sectors an instruction and behind the first
    // tiles' copies, they took 3 us more (32 requests of 64 rows: 42.9 -> 39.3 us).
    // Those of a later part, in L2 by then, are read directly: its tiles are
    // on their way into all stages.
    auto load_queries = [&](const Part &e, bool first) {
      const bool live = row < e.n_rows;
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (static_cast<int64_t>(e.q_row) + row) * 576) + 36 * h +
                         18 * term;
      uint4 v[18];
#pragma unroll
      for (int i = 0; i < 18; ++i) v[i] = make_uint4(0, 0, 0, 0);
      if (first) {
        // a bulk copy per row: eight from each warp, since one warp takes 50 cycles for each
        const uint32_t bar = smem_u32(&misc.q_here);
        if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, e.n_rows * 1152);
        const int r = 8 * warp + lane;
        if (lane < 8 && r < e.n_rows)
          copy_to_smem(s_base + 2 * kStageBytes + r * kQPitch, p.q + (static_cast<int64_t>(e.q_row) + r) * 576, 1152,
                       bar);
        __syncwarp();
        if (!wait(misc.q_here, 0) && threadIdx.x == 0) {  // the copies land before the memory is released
          const volatile int never = 0;
          mbar_wait(bar, 0, &never, p.drain_budget);
        }
        const uint32_t at = s_base + 2 * kStageBytes + row * kQPitch + 576 * h + 288 * term;
        if (live) {
#pragma unroll
          for (int i = 0; i < 18; ++i) v[i] = ld_shared_v4(at + 16 * i);
        }
      } else if (live && p.q_aligned) {
#pragma unroll
        for (int i = 0; i < 18; i += 2) ld_global_32(src + i, v[i], v[i + 1]);
      } else if (live) {
#pragma unroll
        for (int i = 0; i < 18; ++i) v[i] = src[i];
      }
      uint32_t most = 0;  // two elements at a time: magnitudes compare as their bits, NaN on top
#pragma unroll
      for (int i = 0; i < 18; ++i) {
        const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; j += 2) most = __vimax3_u16x2(most, u[j] & 0x7fff7fffu, u[j + 1] & 0x7fff7fffu);
      }
      uint32_t top = max(most & 0xffffu, most >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
      if (term == 0) misc.red[h][row] = __uint_as_float(top);
      named_bar_sync(kBarSoft, kSoftThreads);
      if (first && threadIdx.x == 0) mbar_arrive(smem_u32(&misc.q_read));
      top = max(__float_as_uint(misc.red[0][row]), __float_as_uint(misc.red[1][row]));
      const bool finite = top < 0x7f80u;  // otherwise zeros, and the row is spoilt
      const int ex = finite ? max(static_cast<int>(top >> 7), 27) : 127;  // exponent + 127, at least 2^-100
      const float mult = __uint_as_float(static_cast<uint32_t>(127 + 127 + 7 - ex) << 23);
      const uint32_t keep = finite ? 0xffff0000u : 0u;
      q_scale = __uint_as_float(static_cast<uint32_t>(ex - 7) << 23);
      spoilt = !finite;
#pragma unroll 1
      for (int c0 = 0; c0 < 9; c0 += 3) {  // 48 dims; the code of 144 at once would crowd out the tiles'
#pragma unroll
        for (int c = 0; c < 3; ++c) {  // 16 dims: four words of each term
          uint32_t t1[4], t2[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 &u = v[2 * c + (j >> 1)];
            const uint32_t w[2] = {(j & 1) ? u.z : u.x, (j & 1) ? u.w : u.y};
            uint32_t code[2][2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              // in f16, exact but for elements below 2^-21 of the row's largest
              const float2 y = mul2(make_float2(__uint_as_float((w[s] << 16) & keep), __uint_as_float(w[s] & keep)),
                                    make_float2(mult, mult));
              const __half2 yh = __floats2half2_rn(y.x, y.y);
              code[0][s] = __nv_cvt_halfraw2_to_fp8x2(yh, __NV_SATFINITE, __NV_E4M3);
              const __half2 first = __half2(__nv_cvt_fp8x2_to_halfraw2(code[0][s], __NV_E4M3));
              const __half2 rest = __hmul2(__hsub2(yh, first), __float2half2_rn(32.0f));
              code[1][s] = __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E4M3);
            }
            t1[j] = __byte_perm(code[0][0], code[0][1], 0x5410);
            t2[j] = __byte_perm(code[1][0], code[1][1], 0x5410);
          }
          uint32_t got[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) got[j] = __shfl_xor_sync(0xffffffffu, term ? t1[j] : t2[j], 16);
          const uint32_t col = tmem + kTmemQ + lanes + 72 * h + 4 * (c0 + c);
          tmem_st4(col, term ? got[0] : t1[0], term ? got[1] : t1[1], term ? got[2] : t1[2], term ? got[3] : t1[3]);
          tmem_st4(col + 36, term ? t2[0] : got[0], term ? t2[1] : got[1], term ? t2[2] : got[2],
                   term ? t2[3] : got[3]);
        }
#pragma unroll
        for (int i = 0; i < 12; ++i) v[i] = v[i + 6];
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&misc.q_full));
    };
    // The softmax warps' shared decision whether part k is to be done.
    auto next_part = [&](uint32_t k) {
      wait(misc.work_full[k % kWorkRing], k / kWorkRing);
      named_bar_sync(kBarSoft, kSoftThreads);
      if (threadIdx.x == 0) misc.stop[k & 1u] = *abort_flag != 0 || misc.part[k % kWorkRing].stop;
      named_bar_sync(kBarSoft, kSoftThreads);
      return misc.stop[k & 1u] == 0;
    };

    // Part k's queries go into TMEM before part k - 1's O^T is written out, so
    // that S of the next part overlaps that part's last PV and its epilogue.
    struct Done {
      int b, rb, seg, n_rows, n_tiles;
      int64_t row_base;
    } last{};
    for (uint32_t k = 0;; ++k) {
      const bool more = next_part(k);
      const Part &e = misc.part[k % kWorkRing];
      const bool was_ok = ok;
      if (more && e.n_tiles > 0) load_queries(e, k == 0);
      if (k > 0) {
        if (last.n_tiles > 0) {
          wait(misc.o_done[(g0 - 1) & 1u], (g0 - 1) >> 1);
          tc_fence_after();
          const int n_cols = last.n_rows - 32 * h;  // rows of the unit among this warp's 32 columns
#pragma unroll 1
          for (int blk = 0; blk < 4 && n_cols > 0; ++blk) {
            uint32_t ov[32];
            tmem_ld32(tmem + lanes + kTmemO + blk * kRows + 32 * h, ov);
            if (!ok || !was_ok || *abort_flag != 0) continue;
            const int dim = blk * 128 + 32 * wq + lane;
            const float4 *factor = reinterpret_cast<const float4 *>(&misc.alpha[1][32 * h]);
            // O^T scaled; a factor of 0 is a row without a token
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 f = factor[j];
              ov[4 * j] = __float_as_uint(f.x != 0.0f ? __uint_as_float(ov[4 * j]) * f.x : 0.0f);
              ov[4 * j + 1] = __float_as_uint(f.y != 0.0f ? __uint_as_float(ov[4 * j + 1]) * f.y : 0.0f);
              ov[4 * j + 2] = __float_as_uint(f.z != 0.0f ? __uint_as_float(ov[4 * j + 2]) * f.z : 0.0f);
              ov[4 * j + 3] = __float_as_uint(f.w != 0.0f ? __uint_as_float(ov[4 * j + 3]) * f.w : 0.0f);
            }
            if (last.seg < 0) {
              __nv_bfloat16 *o = p.out + (last.row_base + 32 * h) * 512 + dim;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j < n_cols) o[static_cast<int64_t>(j) * 512] = __float2bfloat16_rn(__uint_as_float(ov[j]));
            } else {
              // partial block [8 row octets][512 dims][8 rows]: one 16-byte store per octet
              const int64_t block = (static_cast<int64_t>(last.b) * p.row_blocks + last.rb) * S + last.seg;
              uint4 *o = reinterpret_cast<uint4 *>(p.segm_out + block * (512 * kRows)) + 4 * h * 512 + dim;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (8 * q >= n_cols) break;
                uint32_t w4[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  w4[u] = pack_bf16(__uint_as_float(ov[8 * q + 2 * u]), __uint_as_float(ov[8 * q + 2 * u + 1]));
                o[q * 512] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
              }
            }
          }
          tc_fence_before();
        } else if (last.seg < 0 && ok) {  // no row sees a token
          uint4 *o = reinterpret_cast<uint4 *>(p.out + last.row_base * 512);
          for (int c = threadIdx.x; c < last.n_rows * 64; c += kSoftThreads) o[c] = make_uint4(0, 0, 0, 0);
        }
      }
      if (!more) break;
      // All eight warps have read their columns of O^T.  The first product of this part overwrites them
      // all, and waits only for the group that has the part's first tile.
      if (k > 0) named_bar_sync(kBarSoft, kSoftThreads);

      const int n_rows = e.n_rows, n_tiles = e.n_tiles, seg_lo = e.seg_lo, seg_hi = e.seg_hi;
      const int len = row < n_rows ? min(max(p.row_len[(e.row_base + row) / p.num_heads], 0), p.max_len) : 0;
      const bool active = 16 * wq < n_rows;  // rows of the unit in this warp's quarter
      const float mult = q_scale * p.score_scale;
      float m_ref = -INFINITY, l = 0.0f, w_sum = 0.0f, w_lost = 0.0f;  // sums in units of 2^m_ref

      // group h takes every other tile; a thread: runs of eight tokens, from 8 term on, 16 apart
#pragma unroll 1
      for (int i = static_cast<int>((g0 ^ h) & 1u); i < n_tiles; i += 2) {
        const uint32_t g = g0 + i;
        const int tok0 = seg_lo + i * kTile, n_valid = min(kTile, seg_hi - tok0);
        const uint32_t stage = s_base + (g % kStages) * kStageBytes;
        const float *sc = misc.sc[h] + 8 * term, *lg = misc.lg[h] + 8 * term, *rc = misc.rc[h] + 8 * term;
        float2 x[24];
        float top = -INFINITY;
        wait(misc.s_full[h], g >> 1);
        tc_fence_after();
        if (active) {
          uint32_t v[96];
#pragma unroll
          for (int c = 0; c < 6; ++c) tmem_ld16(tmem + kTmemS + lanes + 16 * c, v + 16 * c);
          wait(misc.sc_full[h], g >> 1);  // long there: tested while the loads run
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&misc.s_free));
          // lane i has q1 . k of the tile, lane i + 16 q2 . k: each adds up half of them, to scores in
          // log2 units plus the scale's logarithm
          const float2 w_a = make_float2(w_mine, w_mine), w_b = make_float2(w_other, w_other);
#pragma unroll
          for (int q = 0; q < 6; ++q) {
            float s8[8], g8[8];
            if (kWide) {
              s8[0] = sc[16 * q];
              g8[0] = lg[16 * q];
            } else {
              load8(sc + 16 * q, s8);
              load8(lg + 16 * q, g8);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int a = 16 * q + 2 * u, b = a + 8;
              const float2 mine = make_float2(__uint_as_float(term ? v[b] : v[a]),
                                              __uint_as_float(term ? v[b + 1] : v[a + 1]));
              const uint32_t give0 = term ? v[a] : v[b], give1 = term ? v[a + 1] : v[b + 1];
              const float2 other = make_float2(__shfl_xor_sync(0xffffffffu, __uint_as_float(give0), 16),
                                               __shfl_xor_sync(0xffffffffu, __uint_as_float(give1), 16));
              const float2 dot = fma2(mine, w_a, mul2(other, w_b));
              const int i0 = kWide ? 0 : 2 * u, i1 = kWide ? 0 : 2 * u + 1;
              x[4 * q + u] =
                  fma2(dot, mul2(make_float2(s8[i0], s8[i1]), make_float2(mult, mult)), make_float2(g8[i0], g8[i1]));
            }
          }
          const int seen = min(n_valid, len - tok0) - 8 * term;  // tokens this row sees, counted from 8 term
          if (__any_sync(0xffffffffu, seen < 88)) {
#pragma unroll
            for (int j = 0; j < 24; ++j) {
              const int tok = 16 * (j / 4) + 2 * (j % 4);
              if (tok >= seen) x[j].x = -INFINITY;
              if (tok + 1 >= seen) x[j].y = -INFINITY;
            }
          }
#pragma unroll
          for (int j = 0; j < 24; ++j) top = max3(top, x[j].x, x[j].y);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&misc.s_free));
        }
        // The reference as the tile before left it; it moves when a weight exceeds 2^3 of it.
        if (i > 0) wait(misc.turn[(g - 1) & 1u], (g - 1) >> 1);
        const float ref = i > 0 ? misc.ref[row] : -INFINITY;
        const bool move = top > ref + kThreshold;
        const float m_new = move ? top : ref;
        if (term == 0) misc.ref[row] = m_new;
        const bool rescale = named_bar_red_or(bar_group, kGroupThreads, move) && i > 0;
        if (lane == 0) mbar_arrive(smem_u32(&misc.turn[h]));
        if (rescale && term == 0) misc.alpha[h][row] = move ? ex2(ref - top) : 1.0f;  // 0 when ref is -inf
        if (m_ref != m_new) {
          const float c = m_ref == -INFINITY ? 0.0f : ex2(m_ref - m_new);
          l *= c;
          w_sum *= c;
          w_lost *= c;
          m_ref = m_new;
        }
        uint32_t p1[12], p2[12];
        float l_tile = 0.0f;
        if (active) weigh<kWide>(x, rc, m_ref == -INFINITY ? 0.0f : m_ref - kTop, l_tile, w_sum, w_lost, p1, p2);
        l += l_tile;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&misc.sc_free[h]));
        // 32-token blocks [64 rows x 32 B] of each term, the 16-byte halves swapped in every other four rows
        const uint32_t at = row * 32 + ((row >> 2) & 1) * 16 + 8 * term;
        if (active) {
#pragma unroll
          for (int q = 0; q < 6; ++q)
            st_shared_v2(stage + kRopeOff + (q >> 1) * kPBlock + (at ^ ((q & 1) * 16)), p1[2 * q], p1[2 * q + 1]);
          if (l_tile != l_tile) {
            // A NaN code: the rows that see its token are NaN by their sums, and it must not meet the
            // zero weights of the others.  (Or a score beyond float32, which spoils its own row only.)
            wait(misc.full[g % kStages], g / kStages);  // long there: what the copies wrote, to this thread
#pragma unroll 1
            for (int t = 0; t < 48; ++t) {
              const int b = t >> 3;  // 16-token block
              uint32_t code;
              asm volatile("ld.shared.u8 %0, [%1];"
                           : "=r"(code)
                           : "r"(stage + kRopeOff + (b >> 1) * kPBlock + (at ^ ((b & 1) * 16)) + (t & 7))
                           : "memory");
              if ((code & 0x7fu) > 0x7cu)
                for (int c = 0; c < 128; ++c) {
                  const int tok = 16 * b + 8 * term + (t & 7);
                  const uint32_t word = stage + (tok >> 3) * kGroup + (c >> 5) * kAtom + (tok & 7) * 128 + (c & 31) * 4;
                  uint32_t v;
                  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(word) : "memory");
                  const uint32_t nan = __vcmpeq4(v & 0x7f7f7f7fu, 0x7f7f7f7fu);
                  if (nan) asm volatile("st.shared.u32 [%0], %1;" ::"r"(word), "r"(v & ~nan) : "memory");
                }
            }
          }
        }
        // rows of the last 32-token step past the part's end hold anything: zeros
        const int behind = ((n_valid + 31) & ~31) - n_valid;
        for (int c = threadIdx.x & (kGroupThreads - 1); c < behind * 32; c += kGroupThreads) {
          const int tok = n_valid + (c >> 5), chunk = (c & 31) >> 3;
          st_shared_v4(stage + (tok >> 3) * kGroup + chunk * kAtom + (tok & 7) * 128 + (c & 7) * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        if (rescale) {
          wait(misc.o_done[(g - 1) & 1u], (g - 1) >> 1);  // O^T at rest
          named_bar_sync(bar_group, kGroupThreads);        // every row's alpha is there
          tc_fence_after();
#pragma unroll 1
          for (int blk = 0; blk < 8; ++blk) {
            const uint32_t taddr = tmem + lanes + kTmemO + 32 * blk;
            const float4 *alpha = reinterpret_cast<const float4 *>(&misc.alpha[h][32 * (blk & 1)]);
            uint32_t ov[32];
            tmem_ld32(taddr, ov);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 a = alpha[j];
              ov[4 * j] = __float_as_uint(__uint_as_float(ov[4 * j]) * a.x);
              ov[4 * j + 1] = __float_as_uint(__uint_as_float(ov[4 * j + 1]) * a.y);
              ov[4 * j + 2] = __float_as_uint(__uint_as_float(ov[4 * j + 2]) * a.z);
              ov[4 * j + 3] = __float_as_uint(__uint_as_float(ov[4 * j + 3]) * a.w);
            }
            tmem_st32(taddr, ov);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&misc.p1_full[h]));
        if (g > 0) wait(misc.o_done[(g - 1) & 1u], (g - 1) >> 1);  // the tile before has left the second term's buffer
        if (active) {
#pragma unroll
          for (int q = 0; q < 6; ++q)
            st_shared_v2(s_base + kOffP2 + (q >> 1) * kPBlock + (at ^ ((q & 1) * 16)), p2[2 * q], p2[2 * q + 1]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&misc.p2_full));
      }
      g0 += n_tiles;

      // the rows' sums over the four threads that share one
      named_bar_sync(kBarSoft, kSoftThreads);  // both groups' last references are there
      const float m_row = n_tiles > 0 ? misc.ref[row] : -INFINITY;
      const float c_row = m_ref == -INFINITY ? 0.0f : ex2(m_ref - m_row);
      l *= c_row;
      w_sum *= c_row;
      w_lost *= c_row;
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      w_sum += __shfl_xor_sync(0xffffffffu, w_sum, 16);
      w_lost += __shfl_xor_sync(0xffffffffu, w_lost, 16);
      if (h == 1 && term == 0) {
        misc.red[0][row] = l;
        misc.red[1][row] = w_sum;
        misc.alpha[0][row] = w_lost;
      }
      named_bar_sync(kBarSoft, kSoftThreads);
      if (owner) {
        l += misc.red[0][row];
        w_sum += misc.red[1][row];
        w_lost += misc.alpha[0][row];
        if (spoilt && l > 0.0f) l = NAN;
        const bool none = l == 0.0f;
        const float fix = w_sum / (w_sum - w_lost);
        misc.alpha[1][row] = none ? 0.0f : (e.seg < 0 ? fix * kInvTop / l : fix * kInvTop);
        if (ok && row < n_rows) {
          const int64_t r = static_cast<int64_t>(e.row_base) + row;
          if (e.seg < 0) {
            p.lse[r] = none ? -INFINITY : (m_row + log2f(l)) * kLn2;
            if (S > 1) p.segm_sum[r * S] = -1.0f;  // for the merge: written
          } else {
            // a NaN row keeps a finite maximum, so that the merge looks at its sum
            p.segm_max[r * S + e.seg] = none ? -INFINITY : (m_row == -INFINITY ? 0.0f : m_row);
            p.segm_sum[r * S + e.seg] = l;
            for (int s = e.seg + 1; s < e.fill_hi; ++s) {
              p.segm_max[r * S + s] = -INFINITY;
              p.segm_sum[r * S + s] = 0.0f;
            }
          }
        }
      }
      last = {e.b, e.rb, e.seg, n_rows, n_tiles, static_cast<int64_t>(e.row_base)};
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&misc.work_empty[k % kWorkRing]));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

std::atomic<bool> g_attr_set[2][64];  // [kWide][device]
std::atomic<int> g_num_sms[64];

}  // namespace

mla_status launch_decode_scaled(const DecodeLaunch &d, const float *kv_scales, int scale_block, cudaStream_t stream) {
  const mla_decode_args &a = *d.a;
  const uint32_t run = a.page_size < 32 ? a.page_size : 32;
  CUtensorMap tm_v, tm_r;
  mla_status st = make_tmap_tile3d(&tm_v, a.kv_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1,
                                   static_cast<uint64_t>(a.num_cache_rows), 8, CU_TENSOR_MAP_SWIZZLE_128B, 128, 4);
  if (st == MLA_OK)
    st = make_tmap_2d(&tm_r, a.kv_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 576, static_cast<uint64_t>(a.num_cache_rows),
                      64, run, CU_TENSOR_MAP_SWIZZLE_64B);
  if (st != MLA_OK) return st;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  // Scale blocks of eight rows or more: a thread's runs of eight tokens have one scale each, which saves
  // three loads from shared memory a token (64 requests at G = 8: 79.4 us against 82.9 by token, 32 of 64
  // rows at G = 64: 39.0 against 40.9, 16 x 131,072 tokens at G = 32: 258 against 264).
  const bool wide = scale_block >= 8;
  auto kern = wide ? mla_decode_scaled_kernel<true> : mla_decode_scaled_kernel<false>;
  if (!g_attr_set[wide][dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(decode_scaled smem)");
    g_attr_set[wide][dev].store(true, std::memory_order_relaxed);
  }
  int num_sms = g_num_sms[dev].load(std::memory_order_relaxed);
  if (num_sms == 0) {
    e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(SM count)");
    g_num_sms[dev].store(num_sms, std::memory_order_relaxed);
  }
  Params p{};
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.scales = kv_scales;
  p.q_aligned = reinterpret_cast<uintptr_t>(a.q) % 32 == 0;
  p.qo_indptr = a.qo_indptr;
  p.row_len = a.row_len;
  p.subpage_table = a.subpage_table;
  p.segm_out = reinterpret_cast<__nv_bfloat16 *>(d.segm_out);
  p.segm_max = d.segm_max;
  p.segm_sum = d.segm_sum;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.err = d.err;
  p.num_cache_rows = a.num_cache_rows;
  constexpr long long kDefaultBudget = 4000000000LL;  // ~2 s of SM clock
  p.wait_budget = a.wait_cycles > 0 ? static_cast<long long>(a.wait_cycles) : kDefaultBudget;
  p.drain_budget = kDefaultBudget;
  p.score_scale = static_cast<float>(static_cast<double>(a.sm_scale) * 1.4426950408889634);
  p.subpage_stride = a.subpage_stride;
  p.page_size = a.page_size;
  p.log_g = __builtin_ctz(static_cast<unsigned>(scale_block));
  p.num_heads = a.num_heads;
  p.num_segments = a.num_segments;
  p.row_blocks = (a.max_qlen * a.num_heads + kRows - 1) / kRows;
  p.num_reqs = a.num_reqs;
  p.num_views = a.num_views > 1 ? a.num_views : 1;
  p.max_qlen = a.max_qlen;
  p.num_rows = a.num_rows;
  p.max_len = a.subpage_stride * a.page_size;
  // positions (a unit's tiles and its cost) are counted in int32, at the static bound
  const int64_t units = static_cast<int64_t>(a.num_reqs) * p.num_views * p.row_blocks;
  if (units * ((p.max_len + kTile - 1) / kTile + part_cost(kRows)) > INT32_MAX) {
    set_error("mla_decode_verify_scaled: %lld row blocks of up to %d tokens overflow int32 positions", (long long)units,
              p.max_len);
    return MLA_ERR_UNSUPPORTED;
  }
  const int64_t items = units * a.num_segments;
  const unsigned grid = static_cast<unsigned>(items < num_sms ? items : num_sms);
  e = launch_pdl(kern, dim3(grid), dim3(kThreads), kSmemBytes, stream, tm_v, tm_r, p);
  return e == cudaSuccess ? MLA_OK : cuda_fail(e, "decode_scaled launch");
}

}  // namespace mla
