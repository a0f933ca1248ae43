// Row-tile attention kernel for head_dim = 64.
#include "tile_kernel.cuh"

namespace pagedattn {

cudaError_t launch_tile_d64(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                            cudaStream_t stream) {
  return launch_tile<64>(tk, tv, p, stream);
}

}  // namespace pagedattn
