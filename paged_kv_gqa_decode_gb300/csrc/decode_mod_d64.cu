// Decode kernel instantiations with score options over bf16 caches for
// head_dim = 64 (block sizes 16 and 32, query groups up to 8 and up to 16).
#include "launch.h"

namespace pagedattn {

cudaError_t launch_decode_mod_d64(int block_size, bool g16, const CUtensorMap& tk,
                                  const CUtensorMap& tv, const DecodeParams& p, int grid,
                                  size_t smem, cudaStream_t stream) {
  return launch_for_dim<64, kKvBf16, false, true>(block_size, g16, tk, tv, p, grid, smem, stream);
}

}  // namespace pagedattn
