// Row-tile attention kernels for head_dim = 64.
#include "tile_kernel.cuh"

namespace pagedattn {

cudaError_t launch_tile_d64(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                            cudaStream_t stream) {
  if (p.tree_mask != nullptr) return launch_tile_tree_d64(tk, tv, p, stream);
  if (p.teams == 2) return launch_tile<64, 2>(tk, tv, p, stream);
  return launch_tile<64, 1>(tk, tv, p, stream);
}

}  // namespace pagedattn
