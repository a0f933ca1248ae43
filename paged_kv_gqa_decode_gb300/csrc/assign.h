// Block assignment from request lengths (see assign.cu).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace pagedattn {

struct AssignParams {
  const int32_t* seq_lens;     // [num_seqs] tokens held
  const int32_t* new_lens;     // [num_seqs] tokens arriving
  int32_t* block_tables;       // [num_seqs, maxb]: entries of fresh pages are written
  const int32_t* free_blocks;  // [free_capacity] a stack of block ids, its top at free_count - 1
  const int32_t* free_count;   // [1]
  int32_t* seq_lens_out;       // [num_seqs] (may be seq_lens)
  int32_t* qo_indptr;          // [num_seqs + 1]
  int64_t* slot_map;           // [max_new]
  int32_t* free_count_out;     // [1] (may be free_count)
  int32_t* refused;            // [1] or null
  int num_seqs, maxb, BS, free_capacity, max_new;
  long long num_blocks;        // > 0: ids outside the pool are reported
  int32_t* status;             // with num_blocks > 0
};

cudaError_t launch_assign(const AssignParams& a, cudaStream_t stream);

}  // namespace pagedattn
