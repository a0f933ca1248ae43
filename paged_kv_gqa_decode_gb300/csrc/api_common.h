// What the C-ABI layer's translation units share (defined in paged_attn_api.cu).
#pragma once

#include <cstdint>

namespace pagedattn {

// The size rules of every entry point: PAGED_ATTN_OK or an error code.
int api_validate_sizes(int num_seqs, int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
                       int block_size);
// Keeps a CUDA error for paged_attn_last_cuda_error and returns PAGED_ATTN_ERR_CUDA.
int api_cuda_fail(int err);
// SMs of the current device.
int api_sms(int* sms);
// The calling thread's status word (paged_attn_set_checks), null with checks off.
int32_t* api_check_status();

}  // namespace pagedattn
