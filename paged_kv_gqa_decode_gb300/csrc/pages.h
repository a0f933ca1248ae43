// Compaction, forks and release of a cache's pages (see pages.cu).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace pagedattn {

// The caches as bytes: bf16 rows, or e4m3 rows with one float each.
struct CacheRows {
  uint8_t* k;       // [num_blocks, H_kv, BS, row_bytes]
  uint8_t* v;
  float* k_scale;   // [num_blocks, H_kv, BS] or null
  float* v_scale;
  int H_kv, BS, row_bytes;
  long long num_blocks;
};

struct CompactParams {
  CacheRows cache;
  const int32_t* qo_indptr;     // [num_seqs + 1]
  const int32_t* accepted;      // [num_seqs, max_accept]
  const int32_t* block_tables;  // [num_seqs, maxb]
  const int32_t* seq_lens;      // [num_seqs]
  int32_t* seq_lens_out;        // [num_seqs], not seq_lens
  int num_seqs, max_accept, maxb;
  int32_t* status;
};

struct ForkParams {
  CacheRows cache;
  int32_t* block_tables;        // [num_rows, maxb]
  int32_t* seq_lens;            // [num_rows]
  const int32_t* parents;       // [num_forks]
  const int32_t* children;      // [num_forks]
  int32_t* block_refs;          // [num_blocks] holders of a block past the first
  const int32_t* free_blocks;   // [free_capacity]
  const int32_t* free_count;    // [1]
  int32_t* free_count_out;      // [1] (may be free_count)
  int32_t* refused;             // [1] or null
  int num_forks, num_rows, maxb, free_capacity;
  int32_t* status;
#ifdef PAGED_ATTN_WAIT_TEST
  // Test build only: the copy of the K or V rows to this KV head page (block * H_kv + head) is
  // waited for and never issued.  -1: off.
  long long test_skip_page;
#endif
};

struct ReleaseParams {
  const int32_t* block_tables;  // [num_seqs, maxb]
  const int32_t* seq_lens;      // [num_seqs]
  const int32_t* keep_lens;     // [num_seqs]
  int32_t* block_refs;          // [num_blocks] or null
  int32_t* free_blocks;         // [free_capacity]
  const int32_t* free_count;    // [1]
  int32_t* seq_lens_out;        // [num_seqs] (may be seq_lens or keep_lens)
  int32_t* free_count_out;      // [1] (may be free_count)
  int num_seqs, maxb, BS, free_capacity;
  long long num_blocks;         // with block_refs
  int32_t* status;
};

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);
cudaError_t launch_fork(const ForkParams& p, int sms, cudaStream_t stream);
cudaError_t launch_release(const ReleaseParams& p, cudaStream_t stream);

}  // namespace pagedattn
