// Row-tile attention kernels for head_dim = 128.
#include "tile_kernel.cuh"

namespace pagedattn {

cudaError_t launch_tile_d128(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                            cudaStream_t stream) {
  if (p.teams == 2) return launch_tile<128, 2>(tk, tv, p, stream);
  return launch_tile<128, 1>(tk, tv, p, stream);
}

}  // namespace pagedattn
