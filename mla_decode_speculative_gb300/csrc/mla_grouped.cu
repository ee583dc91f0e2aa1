// mla_grouped.cu -- grouped-query and differential decode / causal verify over
// a paged K/V cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_internal.h"

namespace mla {
namespace {

struct Params {
  mla_grouped_args a;
  const float *lambda, *gain;
  float eps;
  int maps, group;
  int *err;
};

// One block per (row, head); the 256 threads go over the tokens in turn.
__global__ void __launch_bounds__(256) grouped_simple(const __grid_constant__ Params p) {
  grid_dep_wait();
  grid_dep_launch();
  const mla_grouped_args &a = p.a;
  const int r = blockIdx.x, h = blockIdx.y, g = h / p.group, D = a.head_dim, Dv = p.maps * D;
  __shared__ float q[512], part[256], o[2][512], red[8];
  int b = -1;
  for (int i = 0; i < a.num_reqs; ++i)
    if (a.qo_indptr[i] <= r && r < a.qo_indptr[i + 1]) b = i;
  if (b < 0) return;
  const int q0 = a.qo_indptr[b], q1 = a.qo_indptr[b + 1];
  if (q0 < 0 || q1 > a.num_rows || q1 - q0 > a.max_qlen) {
    if (threadIdx.x == 0) atomicCAS(p.err, 0, MLA_DEV_BAD_INDPTR);
    return;
  }
  const int bound = a.subpage_stride * a.page_size;
  int n = a.row_len[r];
  if (n > bound) {
    if (threadIdx.x == 0) atomicCAS(p.err, 0, MLA_DEV_LEN_BOUND);
    n = bound;
  }
  const int lo = a.window > 0 && n > a.window ? n - a.window : 0;
  const __nv_bfloat16 *Q = static_cast<const __nv_bfloat16 *>(a.q) + r * a.q_row + h * Dv;
  const __nv_bfloat16 *K = static_cast<const __nv_bfloat16 *>(a.k_cache), *V = static_cast<const __nv_bfloat16 *>(a.v_cache);
  for (int d = threadIdx.x; d < Dv; d += 256) q[d] = __bfloat162float(Q[d]);
  for (int m = 0; m < p.maps; ++m) {
    float top = -INFINITY, total = 0.0f, acc[2] = {0.0f, 0.0f};
    for (int j0 = lo; j0 < n; j0 += 256) {
      __syncthreads();
      const int j = j0 + threadIdx.x;
      float s = -INFINITY;
      int64_t row = -1;
      if (j < n) {
        const int id = a.subpage_table[static_cast<int64_t>(b) * a.subpage_stride + j / a.page_size];
        if (id < 0 || (id + 1LL) * a.page_size > a.num_cache_rows) atomicCAS(p.err, 0, MLA_DEV_BAD_SUBPAGE);
        else row = static_cast<int64_t>(id) * a.page_size + j % a.page_size;
        s = 0.0f;
        if (row >= 0)
          for (int d = 0; d < D; ++d) s += q[m * D + d] * __bfloat162float(K[row * a.k_row + g * Dv + m * D + d]);
        s *= a.sm_scale;
      }
      float t = s;
      for (int x = 16; x > 0; x >>= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, x));
      if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = t;
      __syncthreads();
      float best = top;
      for (int x = 0; x < 8; ++x) best = fmaxf(best, red[x]);
      const float shrink = top == -INFINITY ? 0.0f : expf(top - best);
      part[threadIdx.x] = j < n ? (best == -INFINITY ? s - s : expf(s - best)) : 0.0f;
      __syncthreads();
      total *= shrink;
      acc[0] *= shrink;
      acc[1] *= shrink;
      const int take = min(256, n - j0);
      for (int i = 0; i < take; ++i) {
        const int id = a.subpage_table[static_cast<int64_t>(b) * a.subpage_stride + (j0 + i) / a.page_size];
        const bool bad = id < 0 || (id + 1LL) * a.page_size > a.num_cache_rows;
        const int64_t vr = static_cast<int64_t>(id) * a.page_size + (j0 + i) % a.page_size;
        total += part[i];
        for (int k = 0; k < 2; ++k) {
          const int d = threadIdx.x + 256 * k;
          if (d < Dv && !bad) acc[k] += part[i] * __bfloat162float(V[vr * a.v_row + g * Dv + d]);
        }
      }
      top = best;
    }
    for (int k = 0; k < 2; ++k) {
      const int d = threadIdx.x + 256 * k;
      if (d < Dv) o[m][d] = lo < n ? acc[k] / total : 0.0f;
    }
    if (threadIdx.x == 0) a.lse[(static_cast<int64_t>(r) * a.num_heads + h) * p.maps + m] = lo < n ? top + logf(total) : -INFINITY;
  }
  __syncthreads();
  const float lam = p.maps == 2 ? p.lambda[h] : 0.0f;
  float square = 0.0f;
  for (int d = 0; d < Dv; ++d) {
    const float y = p.maps == 2 ? o[0][d] - lam * o[1][d] : o[0][d];
    square += y * y;
  }
  const float norm = p.gain != nullptr ? rsqrtf(square / Dv + p.eps) : 1.0f;
  for (int d = threadIdx.x; d < Dv; d += 256) {
    const float y = p.maps == 2 ? o[0][d] - lam * o[1][d] : o[0][d];
    static_cast<__nv_bfloat16 *>(a.out)[(static_cast<int64_t>(r) * a.num_heads + h) * Dv + d] =
        __float2bfloat16_rn(p.gain != nullptr ? y * norm * p.gain[d] : y);
  }
}

bool sizes_ok(const mla_grouped_args &a, bool differential) {
  return a.num_heads >= 1 && a.num_kv_heads >= 1 && a.num_heads % a.num_kv_heads == 0 && a.max_qlen >= 1 &&
         (a.head_dim == 64 || a.head_dim == 128 || (a.head_dim == 256 && !differential));
}

mla_status check(const char *what, const mla_grouped_args *a, bool differential) {
  if (a == nullptr) {
    set_error("%s: null argument struct", what);
    return MLA_ERR_INVALID_ARG;
  }
  if (a->num_reqs < 1 || a->num_rows < 1 || a->num_heads < 1 || a->num_kv_heads < 1 || a->max_qlen < 1 ||
      a->subpage_stride < 1 || a->num_cache_rows < 1) {
    set_error("%s: B=%d T=%d H=%d Hkv=%d max_qlen=%d subpage_stride=%d rows=%lld must be >= 1", what, a->num_reqs,
              a->num_rows, a->num_heads, a->num_kv_heads, a->max_qlen, a->subpage_stride,
              (long long)a->num_cache_rows);
    return MLA_ERR_INVALID_ARG;
  }
  if (a->num_heads % a->num_kv_heads != 0) {
    set_error("%s: %d heads do not divide into %d groups", what, a->num_heads, a->num_kv_heads);
    return MLA_ERR_INVALID_ARG;
  }
  if (!sizes_ok(*a, differential)) {
    set_error("%s: head_dim %d unsupported (64, 128%s)", what, a->head_dim, differential ? "" : " or 256");
    return MLA_ERR_UNSUPPORTED;
  }
  if (a->page_size < 8 || a->page_size > 128 || (a->page_size & (a->page_size - 1)) != 0) {
    set_error("%s: page_size %d unsupported (power of two in [8, 128])", what, a->page_size);
    return MLA_ERR_UNSUPPORTED;
  }
  if (static_cast<int64_t>(a->subpage_stride) * a->page_size > INT32_MAX - 1024 || a->num_cache_rows > INT32_MAX ||
      static_cast<int64_t>(a->num_rows) * a->num_heads > INT32_MAX / 2 ||
      static_cast<int64_t>(a->max_qlen) * a->num_heads > INT32_MAX / 2) {
    set_error("%s: sizes overflow int32 indexing", what);
    return MLA_ERR_INVALID_ARG;
  }
  if (a->max_qlen > a->num_rows) {
    set_error("%s: max_qlen %d above the row capacity %d", what, a->max_qlen, a->num_rows);
    return MLA_ERR_INVALID_ARG;
  }
  if (a->window < 0 || a->wait_cycles < 0 || !(a->sm_scale > 0.0f) || a->sm_scale > 1e30f) {
    set_error("%s: window %d and wait_cycles must be >= 0, sm_scale %g positive", what, a->window, a->sm_scale);
    return MLA_ERR_INVALID_ARG;
  }
  if (a->q == nullptr || a->k_cache == nullptr || a->v_cache == nullptr || a->qo_indptr == nullptr ||
      a->row_len == nullptr || a->subpage_table == nullptr || a->out == nullptr || a->lse == nullptr) {
    set_error("%s: null device pointer", what);
    return MLA_ERR_INVALID_ARG;
  }
  for (const void *ptr : {a->q, a->k_cache, a->v_cache, static_cast<const void *>(a->out)})
    if (reinterpret_cast<uintptr_t>(ptr) % 16 != 0) {
      set_error("%s: q, k_cache, v_cache and out must be 16-byte aligned", what);
      return MLA_ERR_INVALID_ARG;
    }
  const int64_t row = static_cast<int64_t>(differential ? 2 : 1) * a->head_dim;
  if (a->q_row % 8 != 0 || a->k_row % 8 != 0 || a->v_row % 8 != 0 || a->q_row < row * a->num_heads ||
      a->k_row < row * a->num_kv_heads || a->v_row < row * a->num_kv_heads || a->q_row > (1LL << 34) ||
      a->k_row > (1LL << 34) || a->v_row > (1LL << 34)) {
    set_error("%s: rows must be a multiple of 8 elements apart and not overlap (q %lld, k %lld, v %lld)", what,
              (long long)a->q_row, (long long)a->k_row, (long long)a->v_row);
    return MLA_ERR_INVALID_ARG;
  }
  if (a->num_cache_rows % 8 != 0) {
    set_error("%s: %lld cache rows are not a multiple of 8", what, (long long)a->num_cache_rows);
    return MLA_ERR_INVALID_ARG;
  }
  return MLA_OK;
}

mla_status run(const char *what, const mla_grouped_args *a, bool differential, const float *lambda, const float *gain,
               float eps, void *workspace, size_t bytes, mla_stream_t stream) {
  const mla_status st = check(what, a, differential);
  if (st != MLA_OK) return st;
  if (differential && lambda == nullptr) {
    set_error("%s: null lambda", what);
    return MLA_ERR_INVALID_ARG;
  }
  if (gain != nullptr && !(eps >= 0.0f)) {
    set_error("%s: eps %g must be >= 0", what, eps);
    return MLA_ERR_INVALID_ARG;
  }
  const size_t need = mla_decode_grouped_workspace(a, differential);
  if (need > 0 && (workspace == nullptr || bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)) {
    set_error("%s: workspace of %zu bytes (256-byte aligned) needed, got %zu at %p", what, need, bytes, workspace);
    return MLA_ERR_WORKSPACE;
  }
  int *err = device_error_word();
  if (err == nullptr) return MLA_ERR_CUDA;
  Params p{*a, lambda, gain, eps, differential ? 2 : 1, a->num_heads / a->num_kv_heads, err};
  const cudaError_t e = launch_pdl(grouped_simple, dim3(a->num_rows, a->num_heads), dim3(256), 0,
                                   reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? MLA_OK : cuda_fail(e, "grouped launch");
}

}  // namespace
}  // namespace mla

extern "C" {

size_t mla_decode_grouped_workspace(const mla_grouped_args *a, int differential) {
  if (a == nullptr || !mla::sizes_ok(*a, differential != 0)) return 0;
  return 256;
}

mla_status mla_decode_grouped(const mla_grouped_args *a, void *workspace, size_t workspace_bytes, mla_stream_t stream) {
  return mla::run("mla_decode_grouped", a, false, nullptr, nullptr, 0.0f, workspace, workspace_bytes, stream);
}

mla_status mla_decode_differential(const mla_grouped_args *a, const float *lambda, const float *gain, float eps,
                                   void *workspace, size_t workspace_bytes, mla_stream_t stream) {
  return mla::run("mla_decode_differential", a, true, lambda, gain, eps, workspace, workspace_bytes, stream);
}

}  // extern "C"
