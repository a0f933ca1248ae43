// Row-tile attention of drafted trees for head_dim = 256.
#include "tile_kernel.cuh"

namespace pagedattn {

cudaError_t launch_tile_tree_d256(const CUtensorMap& tk, const CUtensorMap& tv,
                                 const TileParams& p, cudaStream_t stream) {
  return launch_tile<256, 1, true>(tk, tv, p, stream);
}

}  // namespace pagedattn
