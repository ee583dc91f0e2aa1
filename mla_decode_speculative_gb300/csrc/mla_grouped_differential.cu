// mla_grouped_differential.cu -- the configurations of differential attention:
// two keys of 64 or 128 values, 16 or 32 columns of each map.
#include "mla_grouped_launch.cuh"

namespace mla {
namespace grouped {

mla_status launch_differential(int W, int nc, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const Params &p,
                               int grid, bool merge, cudaStream_t stream) {
  if (W == 2) {
    if (nc == 32) return launch_as<2, 2, 32>(q, k, v, p, grid, merge, stream);
    return launch_as<2, 2, 64>(q, k, v, p, grid, merge, stream);
  }
  if (nc == 32) return launch_as<4, 2, 32>(q, k, v, p, grid, merge, stream);
  return launch_as<4, 2, 64>(q, k, v, p, grid, merge, stream);
}

}  // namespace grouped
}  // namespace mla
