// Row-tile attention over the paged cache (tile_kernel.cuh) and the merge of its
// partial states: the interface between the C-ABI layer and the kernels.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace pagedattn {

// Softmax teams of a CTA, each with a tile of 128 query rows.  Two for head_dim 64
// and 128, where a sequence has more than 128 rows for a KV head on average and the
// pieces of 256 rows fill the SMs (a K/V tile then serves both: four capped prompt
// chunks 476 us, 543 with one; plain 401 / 450; of head_dim 64 441 / 478 and 334 /
// 367); else one, in CTAs of which two run on an SM (64, 128), as their starts and ends
// then overlap (eight chunks of 40 to 64 tokens 41.9 us, 46.8 with two; verification of
// five tokens 50.3 / 56.6); one for 256, whose accumulators take half the tensor memory.
// (Just past the border two teams are not yet the better choice: twelve chunks of 40 to
// 64 tokens 64.1 us, 50.3 with one, eight of 200 to 400 tokens 95.0 / 88.5; at 500 tokens
// it is 194.8 / 206.)
constexpr int tile_teams(int D, long long total_rows, long long num_seqs, int H_kv, int sms) {
  return D < 256 && total_rows > 128 * num_seqs &&
                 (total_rows / 256 + num_seqs) * H_kv >= sms
             ? 2
             : 1;
}

struct TileParams {
  const __nv_bfloat16* q;       // [total_q, H_q, D]
  __nv_bfloat16* out;           // [total_q, H_q, D]
  const int32_t* block_tables;  // [num_seqs, maxb]
  const int32_t* seq_lens;      // [num_seqs] cached tokens
  const int32_t* qo_indptr;     // [num_seqs + 1] rows of q
  int num_seqs, total_q, H_q, H_kv, G, maxb, BS, causal;
  float scale_log2;             // scale * log2(e)
  float cap_log2, cap_in;       // softcap * log2(e) (0: off), scale / softcap
  const float* slopes;          // [H_q] or null
  int window;
  const int32_t* prefix_lens;   // [num_seqs] or null
  const int32_t* doc_starts;    // [total_q] or null
  // Shared prefix: query row t stands tail_lens[t] tokens past the sequence's
  // (the prefix's) last one (null: the rows are the sequence's last tokens).
  const int32_t* tail_lens;     // [total_q] or null
  int tail_cap;                 // largest value tail_lens is clamped to
  int teams;                    // tile_teams: picks the kernel
  int splits;                   // parts of each piece's token range
  int single;                   // 1: splits is 1 and the kernel writes the output itself
  float* part_o;                // [splits][total_q * H_q][D]
  float2* part_ml;              // [splits][total_q * H_q] (running max, log2 domain; sum)
  int32_t* status;
  long long num_blocks;         // > 0: block ids are checked against it
};

struct MergeParams {
  const float* part_o;
  const float2* part_ml;
  int splits;
  const int32_t* qo_indptr;  // rows [qo_indptr[0], qo_indptr[num_seqs]) have parts
  int num_seqs, total_q, H_q, D;
  const float* state;        // [total_q * H_q][D + 4] one more state of every row, or null
  __nv_bfloat16* out;
};

cudaError_t launch_tile_d64(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                            cudaStream_t stream);
cudaError_t launch_tile_d128(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                             cudaStream_t stream);
cudaError_t launch_tile_d256(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                             cudaStream_t stream);
cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream);

}  // namespace pagedattn
