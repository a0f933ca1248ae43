// Norms and rotation of query and key heads, and the append of K and V by slot (see rope.cu).
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace pagedattn {

struct RopeParams {
  const __nv_bfloat16* q;      // row r at r * q_stride: [H_q, D]
  const __nv_bfloat16* k;      // row r at r * k_stride: [H_kv, D]
  const __nv_bfloat16* v;
  long long q_stride, k_stride, v_stride;  // elements between rows (multiples of 8)
  __nv_bfloat16* q_out;        // [rows, H_q, D]
  void* k_cache;               // [num_blocks, H_kv, BS, D]: bf16, or e4m3 bytes
  void* v_cache;
  float* k_scale;              // [num_blocks, H_kv, BS] dequant floats, or null (bf16 caches)
  float* v_scale;
  const int64_t* slot_map;     // [rows]; outside [0, num_blocks * BS): K and V are not written
  const int32_t* positions;    // [axes, rows]
  const int32_t* freq_axis;    // [R / 2] axis of each pair, or null (axis 0)
  const float* cos_sin;        // [max_positions, R]: R / 2 cosines, then R / 2 sines
  const float* q_norm;         // [D] or null
  const float* k_norm;         // [D] or null
  float eps;
  int rows, axes, max_positions, R, interleaved, H_q, H_kv, D, BS;
  long long num_blocks;
  int32_t* status;             // null, or: bit 0 a slot past the pool, bit 1 a position outside,
                               // bit 2 a copy that did not come
#ifdef PAGED_ATTN_WAIT_TEST
  // Test build only: the copies of this row's queries are waited for and never issued.  -1: off.
  long long test_skip_row;
#endif
};

cudaError_t launch_rope_append(const RopeParams& p, int sms, cudaStream_t stream);

}  // namespace pagedattn
