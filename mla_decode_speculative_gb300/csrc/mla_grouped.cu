// mla_grouped.cu -- grouped-query and differential decode / causal verify over
// a paged K/V cache: argument checks, tensor maps and the choice of the
// configuration.  The kernels are in mla_grouped.cuh and mla_grouped_launch.cuh.


#include "mla_grouped.cuh"

namespace mla {
namespace grouped {
namespace {

// Columns of the products: the fewest of 16, 32, 64 that hold a request's rows
// of a group (differential: 16 or 32 of each map).
int columns_of(const mla_grouped_args &a, bool differential) {
  const int64_t rows = static_cast<int64_t>(a.max_qlen) * (a.num_heads / a.num_kv_heads);
  if (differential) return rows <= 16 ? 32 : 64;
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
}

struct Layout {
  size_t part_o, part_stat, meta, total;
};
Layout layout_of(const mla_grouped_args &a, bool differential) {
  const size_t nc = columns_of(a, differential), dv = static_cast<size_t>(a.head_dim) * (differential ? 2 : 1);
  Layout l{};
  size_t off = 0;
  l.part_o = off;
  off += align256(kMaxCtas * 2 * nc * dv * sizeof(float));
  l.part_stat = off;
  off += align256(kMaxCtas * 2 * 2 * nc * sizeof(float));
  l.meta = off;
  off += align256(kMaxCtas * sizeof(Meta));
  l.total = off;
  return l;
}

// From a row of q to the next (of a single one whatever the caller's stride is).
int64_t q_stride(const mla_grouped_args &a, bool differential) {
  return a.num_rows > 1 ? a.q_row : static_cast<int64_t>(differential ? 2 : 1) * a.head_dim * a.num_heads;
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
  const int64_t q_row = q_stride(*a, differential);
  if (q_row % 8 != 0 || a->k_row % 8 != 0 || a->v_row % 8 != 0 || q_row < row * a->num_heads ||
      a->k_row < row * a->num_kv_heads || a->v_row < row * a->num_kv_heads || q_row > (1LL << 34) ||
      a->k_row > (1LL << 34) || a->v_row > (1LL << 34)) {
    set_error("%s: rows must be a multiple of 8 elements apart and not overlap (q %lld, k %lld, v %lld)", what,
              (long long)q_row, (long long)a->k_row, (long long)a->v_row);
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
  const Layout lay = layout_of(*a, differential);
  char *ws = static_cast<char *>(workspace);
  const int maps = differential ? 2 : 1, W = a->head_dim * maps / 64, nc = columns_of(*a, differential), nr = nc / maps;
  const int G = a->num_heads / a->num_kv_heads, P = a->page_size;
  Params p{};
  p.row_len = a->row_len;
  p.out = static_cast<__nv_bfloat16 *>(a->out);
  p.lse = a->lse;
  p.lambda = lambda;
  p.gain = gain;
  p.eps = eps;
  p.part_o = reinterpret_cast<float *>(ws + lay.part_o);
  p.part_stat = reinterpret_cast<float *>(ws + lay.part_stat);
  p.meta = reinterpret_cast<Meta *>(ws + lay.meta);
  p.err = err;
  p.wait_budget = a->wait_cycles > 0 ? a->wait_cycles : 4000000000LL;
  p.drain_budget = 4000000000LL;
  p.scale_log2 = a->sm_scale * 1.44269504088896340736f;
  p.num_rows = a->num_rows;
  p.num_heads = a->num_heads;
  p.num_kv_heads = a->num_kv_heads;
  p.group = G;
  p.max_qlen = a->max_qlen;
  p.max_len = a->subpage_stride * P;
  p.window = a->window;
  p.subpage_stride = a->subpage_stride;
  while ((8 << p.page_shift) < P) ++p.page_shift;
  p.page_shift += 3;
  p.box_shift = p.page_shift < 5 ? p.page_shift : 5;
  p.page_groups = static_cast<int>(a->num_cache_rows / 8);
  p.head_blocks = (G + nr - 1) / nr;
  p.heads_per_block = p.head_blocks == 1 ? G : nr;
  p.one_block = p.head_blocks == 1 && nr / G >= a->max_qlen;
  p.rows_per_block = p.head_blocks == 1 ? (nr / G < a->max_qlen ? nr / G : a->max_qlen) : 1;

  // Requests of one launch: as many as the kernel tabulates and as int32
  // positions hold at the static bound.
  const int64_t tiles = (static_cast<int64_t>(p.max_len) + kTile - 1) / kTile + (p.window > 0 ? 1 : 0);
  const int64_t blocks = p.head_blocks == 1 ? (a->max_qlen + p.rows_per_block - 1) / p.rows_per_block
                                            : static_cast<int64_t>(a->max_qlen) * p.head_blocks;
  const int64_t units = blocks * a->num_kv_heads, most = units * (tiles + kOverhead);
  if (units > INT32_MAX || most > INT32_MAX) {
    set_error("%s: one request of %d tokens and %d rows is too large", what, p.max_len, a->max_qlen);
    return MLA_ERR_UNSUPPORTED;
  }
  const int64_t by_range = INT32_MAX / most;
  const int reqs = static_cast<int>(by_range < kMaxReqs ? by_range : kMaxReqs);

  CUtensorMap tq, tk, tv;
  const uint64_t w64 = static_cast<uint64_t>(W), hkv = static_cast<uint64_t>(a->num_kv_heads), g64 = static_cast<uint64_t>(G);
  {
    const cuuint64_t dims[5] = {64, g64, static_cast<uint64_t>(a->num_rows), w64, hkv};
    const cuuint64_t strides[4] = {w64 * 128, static_cast<uint64_t>(q_stride(*a, differential)) * 2, 128, g64 * w64 * 128};
    const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(p.heads_per_block), static_cast<cuuint32_t>(p.rows_per_block), 1, 1};
    const mla_status s = make_tmap_5d(&tq, a->q, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (s != MLA_OK) return s;
  }
  for (int i = 0; i < 2; ++i) {
    const uint64_t row = static_cast<uint64_t>(i == 0 ? a->k_row : a->v_row) * 2;
    const cuuint64_t dims[5] = {64, 8, w64, static_cast<uint64_t>(p.page_groups), hkv};
    const cuuint64_t strides[4] = {row, 128, row * 8, w64 * 128};
    const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(W < 2 ? W : 2), 1u << (p.box_shift - 3), 1};
    // a fetch of 256 bytes would bring another group's 128 bytes of a token along
    const mla_status s = make_tmap_5d(i == 0 ? &tk : &tv, i == 0 ? a->k_cache : a->v_cache, dims, strides, box,
                                      CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
    if (s != MLA_OK) return s;
  }
  for (int b0 = 0; b0 < a->num_reqs; b0 += reqs) {
    p.num_reqs = a->num_reqs - b0 < reqs ? a->num_reqs - b0 : reqs;
    p.first_req = b0;
    p.qo_indptr = a->qo_indptr + b0;
    p.subpage_table = a->subpage_table + static_cast<int64_t>(b0) * a->subpage_stride;
    // no more CTAs than there are chunks at the static bound
    const int64_t all = units * p.num_reqs, want = most * p.num_reqs / kMinChunk > all ? most * p.num_reqs / kMinChunk : all;
    const int grid = static_cast<int>(want < kMaxCtas ? want : kMaxCtas);
    p.few = all <= grid;
    p.may_twin = blocks > 1 && grid > 1;
    const bool merge = grid > 1 && !(p.few && tiles <= whole_tiles(W));  // units may be cut
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const mla_status s =
        differential ? launch_differential(W, nc, tq, tk, tv, p, grid, merge, cs) : launch_grouped(W, nc, tq, tk, tv, p, grid, merge, cs);
    if (s != MLA_OK) return s;
  }
  return MLA_OK;
}

}  // namespace
}  // namespace grouped
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_decode_grouped_workspace(const mla_grouped_args *a, int differential) {
  if (a == nullptr || !grouped::sizes_ok(*a, differential != 0)) return 0;
  return grouped::layout_of(*a, differential != 0).total;
}

mla_status mla_decode_grouped(const mla_grouped_args *a, void *workspace, size_t workspace_bytes, mla_stream_t stream) {
  return grouped::run("mla_decode_grouped", a, false, nullptr, nullptr, 0.0f, workspace, workspace_bytes, stream);
}

mla_status mla_decode_differential(const mla_grouped_args *a, const float *lambda, const float *gain, float eps,
                                   void *workspace, size_t workspace_bytes, mla_stream_t stream) {
  return grouped::run("mla_decode_differential", a, true, lambda, gain, eps, workspace, workspace_bytes, stream);
}

}  // extern "C"
