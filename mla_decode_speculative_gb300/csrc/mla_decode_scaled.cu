// mla_decode_scaled.cu -- absorbed-form MLA decode / causal verify over a paged
// e4m3 cache with one scale per block of G cache rows
// (mla_decode_verify_scaled).
//
// For query row r = (verify row t, head h) of request b and its visible tokens
// j < row_len[t], token j in cache row n with scale a_j = kv_scales[n / G]:
//   s_j = sm_scale * a_j * <q[r], code_j>, out = sum softmax(s)_j a_j code_j[0:512],
//   lse = ln sum e^{s_j}.
// One warp per (view, row, head): lane l holds dims 18 l .. 18 l + 17 of q, an
// online softmax runs over the tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_internal.h"

namespace mla {
namespace {

struct ScaledParams {
  const __nv_bfloat16 *q;
  const uint8_t *cache;
  const float *scales;
  const int32_t *qo_indptr, *row_len, *subpage_table;
  __nv_bfloat16 *out;
  float *lse;
  int *err;
  int64_t num_cache_rows;
  float scale_log2;
  int log_g, page_size, subpage_stride, num_reqs, num_rows, num_heads, num_views, max_qlen;
};

__device__ __forceinline__ float code_value(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half *>(&h));
}

__global__ void __launch_bounds__(256) decode_scaled_rows(const ScaledParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t items = static_cast<int64_t>(p.num_views) * p.num_rows * p.num_heads;
  const int total = p.qo_indptr[p.num_reqs];
  if (p.qo_indptr[0] != 0 || total < 0 || total > p.num_rows) {
    if (threadIdx.x == 0) atomicCAS(p.err, 0, MLA_DEV_BAD_INDPTR);
    return;
  }
  for (int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; item < items;
       item += (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5) {
    const int64_t vr = item / p.num_heads;
    const int v = static_cast<int>(vr / p.num_rows), r = static_cast<int>(vr % p.num_rows);
    if (r >= total) continue;
    int lo = 0, hi = p.num_reqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.qo_indptr[mid] <= r) lo = mid;
      else hi = mid;
    }
    if (p.qo_indptr[lo + 1] <= r || p.qo_indptr[lo + 1] - p.qo_indptr[lo] > p.max_qlen) {
      if (lane == 0) atomicCAS(p.err, 0, MLA_DEV_BAD_INDPTR);
      continue;
    }
    const int h = static_cast<int>(item % p.num_heads);
    int n = p.row_len[vr];
    const int64_t bound = static_cast<int64_t>(p.subpage_stride) * p.page_size;
    if (n > bound) {
      if (lane == 0) atomicCAS(p.err, 0, MLA_DEV_LEN_BOUND);
      n = static_cast<int>(bound);
    }
    const int32_t *pages = p.subpage_table + (static_cast<int64_t>(v) * p.num_reqs + lo) * p.subpage_stride;
    float q[18], acc[18];
    const __nv_bfloat16 *qr = p.q + (static_cast<int64_t>(r) * p.num_heads + h) * 576;
#pragma unroll
    for (int i = 0; i < 18; ++i) {
      q[i] = __bfloat162float(qr[lane + 32 * i]);
      acc[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f, lost = 0.0f;  // l + lost: many small weights under a large one
    for (int j = 0; j < n; ++j) {
      const int id = pages[j / p.page_size];
      const int64_t row = static_cast<int64_t>(id) * p.page_size + j % p.page_size;
      float k[18], a = 0.0f;
      if (id < 0 || (static_cast<int64_t>(id) + 1) * p.page_size > p.num_cache_rows) {
        if (lane == 0) atomicCAS(p.err, 0, MLA_DEV_BAD_SUBPAGE);
#pragma unroll
        for (int i = 0; i < 18; ++i) k[i] = 0.0f;
      } else {
        a = fmaxf(p.scales[row >> p.log_g], 7.888609052210118e-31f);  // 2^-100 at least
#pragma unroll
        for (int i = 0; i < 18; ++i) k[i] = code_value(p.cache[row * 576 + lane + 32 * i]);
      }
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 18; ++i) s += q[i] * k[i];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float x = s * a * p.scale_log2;
      if (x > m) {
        const float c = exp2f(m - x);
        l *= c;
        lost *= c;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] *= c;
        m = x;
      }
      const float e = exp2f(x - m);
      const float y = e + lost, sum = l + y;
      lost = y - (sum - l);
      l = sum;
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] += e * a * k[i];
    }
    const float inv = l > 0.0f ? 1.0f / l : (n > 0 ? l : 0.0f);
    __nv_bfloat16 *o = p.out + (vr * p.num_heads + h) * 512;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[lane + 32 * i] = __float2bfloat16_rn(acc[i] * inv);
    if (lane == 0) p.lse[vr * p.num_heads + h] = n > 0 ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
  }
}

}  // namespace

mla_status launch_decode_scaled(const DecodeLaunch &d, const float *kv_scales, int scale_block, cudaStream_t stream) {
  const mla_decode_args &a = *d.a;
  ScaledParams p{};
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.cache = static_cast<const uint8_t *>(a.kv_cache);
  p.scales = kv_scales;
  p.qo_indptr = a.qo_indptr;
  p.row_len = a.row_len;
  p.subpage_table = a.subpage_table;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.err = d.err;
  p.num_cache_rows = a.num_cache_rows;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.sm_scale) * 1.4426950408889634);
  p.log_g = __builtin_ctz(static_cast<unsigned>(scale_block));
  p.page_size = a.page_size;
  p.subpage_stride = a.subpage_stride;
  p.num_reqs = a.num_reqs;
  p.num_rows = a.num_rows;
  p.num_heads = a.num_heads;
  p.num_views = a.num_views > 1 ? a.num_views : 1;
  p.max_qlen = a.max_qlen;
  const int64_t items = static_cast<int64_t>(p.num_views) * a.num_rows * a.num_heads;
  const int64_t ctas = (items + 7) / 8;
  const cudaError_t e = launch_pdl(decode_scaled_rows, dim3(static_cast<unsigned>(ctas < 65536 ? ctas : 65536)), dim3(256),
                                   0, stream, p);
  return e == cudaSuccess ? MLA_OK : cuda_fail(e, "decode_scaled launch");
}

}  // namespace mla
