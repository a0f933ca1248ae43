// Row-tile attention kernel for head_dim = 128.
#include "tile_kernel.cuh"

namespace pagedattn {

cudaError_t launch_tile_d128(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                            cudaStream_t stream) {
  return launch_tile<128>(tk, tv, p, stream);
}

}  // namespace pagedattn
