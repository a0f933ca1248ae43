// Row-tile attention kernels for head_dim = 256.
#include "tile_kernel.cuh"

namespace pagedattn {

cudaError_t launch_tile_d256(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                            cudaStream_t stream) {
  return launch_tile<256, 1>(tk, tv, p, stream);
}

}  // namespace pagedattn
