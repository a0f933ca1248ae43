// Row-tile attention of drafted trees for head_dim = 128.
#include "tile_kernel.cuh"

namespace pagedattn {

cudaError_t launch_tile_tree_d128(const CUtensorMap& tk, const CUtensorMap& tv,
                                 const TileParams& p, cudaStream_t stream) {
  if (p.teams == 2) return launch_tile<128, 2, true>(tk, tv, p, stream);
  return launch_tile<128, 1, true>(tk, tv, p, stream);
}

}  // namespace pagedattn
