// mla_grouped_plain.cu -- the configurations of grouped-query attention: heads
// of 64, 128 and 256 values, 16 to 64 columns.
#include "mla_grouped_launch.cuh"

namespace mla {
namespace grouped {

mla_status launch_grouped(int W, int nc, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const Params &p,
                          int grid, bool merge, cudaStream_t stream) {
  if (W == 1) {
    if (nc == 16) return launch_as<1, 1, 16>(q, k, v, p, grid, merge, stream);
    if (nc == 32) return launch_as<1, 1, 32>(q, k, v, p, grid, merge, stream);
    return launch_as<1, 1, 64>(q, k, v, p, grid, merge, stream);
  }
  if (W == 2) {
    if (nc == 16) return launch_as<2, 1, 16>(q, k, v, p, grid, merge, stream);
    if (nc == 32) return launch_as<2, 1, 32>(q, k, v, p, grid, merge, stream);
    return launch_as<2, 1, 64>(q, k, v, p, grid, merge, stream);
  }
  if (nc == 16) return launch_as<4, 1, 16>(q, k, v, p, grid, merge, stream);
  if (nc == 32) return launch_as<4, 1, 32>(q, k, v, p, grid, merge, stream);
  return launch_as<4, 1, 64>(q, k, v, p, grid, merge, stream);
}

}  // namespace grouped
}  // namespace mla
