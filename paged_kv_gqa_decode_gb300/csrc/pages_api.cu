// C ABI of the operators on rows and pages of a cache (include/paged_attn.h):
// paged_kv_rope_append_slots, paged_kv_compact, paged_kv_fork, paged_kv_release.
// Argument validation and the kernels' parameters.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "api_common.h"
#include "pages.h"
#include "paged_attn.h"
#include "rope.h"

namespace pagedattn {
namespace {

bool aligned(const void* p, uintptr_t n) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}
bool aligned16(const void* p) { return aligned(p, 16); }
bool aligned4(const void* p) { return aligned(p, 4); }

int done(cudaError_t e) { return e == cudaSuccess ? PAGED_ATTN_OK : api_cuda_fail(e); }

// Sizes and pointers of a pair of caches: bf16, or e4m3 with both scales.
int cache_sizes(const float* k_scale, const float* v_scale, int H_kv, int head_dim,
                int max_blocks_per_seq, int block_size, long long num_blocks) {
  int rc = api_validate_sizes(0, H_kv, H_kv, head_dim, max_blocks_per_seq, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  if ((k_scale != nullptr || v_scale != nullptr) && head_dim == 64) return PAGED_ATTN_ERR_HEAD_DIM;
  if (num_blocks < 1 || num_blocks > 0x7fffffffLL ||
      2LL * H_kv * block_size * head_dim > 0x7fffffffLL)
    return PAGED_ATTN_ERR_SIZES;
  return PAGED_ATTN_OK;
}

bool cache_pointers(const void* k_cache, const void* v_cache, const float* k_scale,
                    const float* v_scale) {
  if (!aligned16(k_cache) || !aligned16(v_cache)) return false;
  if (k_scale == nullptr && v_scale == nullptr) return true;
  return aligned16(k_scale) && aligned16(v_scale);
}

// Whether bytes [out, out + size) meet one of the rows of `row` bytes, `stride` apart.
bool meets_rows(const void* out, long long size, const void* src, long long row, long long stride,
                int rows) {
  const long long from = (long long)(reinterpret_cast<uintptr_t>(out) -
                                     reinterpret_cast<uintptr_t>(src));  // out's place behind src
  // the first row that ends past `from`
  const long long r = from < row ? 0 : (from - row) / stride + 1;
  return r < rows && r * stride < from + size;
}

CacheRows cache_rows(void* k_cache, void* v_cache, float* k_scale, float* v_scale, int H_kv,
                     int head_dim, int block_size, long long num_blocks) {
  CacheRows c;
  c.k = static_cast<uint8_t*>(k_cache);
  c.v = static_cast<uint8_t*>(v_cache);
  c.k_scale = k_scale;
  c.v_scale = v_scale;
  c.H_kv = H_kv;
  c.BS = block_size;
  c.row_bytes = k_scale != nullptr ? head_dim : 2 * head_dim;
  c.num_blocks = num_blocks;
  return c;
}

#ifdef PAGED_ATTN_WAIT_TEST
thread_local long long g_test_skip_page = -1, g_test_skip_row = -1;
#endif

}  // namespace
}  // namespace pagedattn

using namespace pagedattn;

#ifdef PAGED_ATTN_WAIT_TEST
// Test build only (not in include/paged_attn.h): the next forks of this thread wait for copies to KV
// head page `page` that they do not issue (-1: off).
extern "C" PAGED_ATTN_API int paged_attn_test_set_fork_fault(long long page) {
  g_test_skip_page = page;
  return PAGED_ATTN_OK;
}
// The same for the copies of the queries of row `row` that the rotation streams.
extern "C" PAGED_ATTN_API int paged_attn_test_set_rope_fault(long long row) {
  g_test_skip_row = row;
  return PAGED_ATTN_OK;
}
#endif

int paged_kv_rope_append_slots(const void* q, const void* k_new, const void* v_new,
                               long long q_stride, long long k_stride, long long v_stride,
                               void* q_out, void* k_cache, void* v_cache, float* k_scale,
                               float* v_scale, const int64_t* slot_map, const int32_t* positions,
                               int num_axes, const int32_t* freq_axis, const float* cos_sin,
                               int max_positions, int rotary_dim, int interleaved,
                               const float* q_norm, const float* k_norm, float eps, int rows,
                               int H_q, int H_kv, int head_dim, int block_size,
                               long long num_blocks, void* stream) {
  int rc = api_validate_sizes(0, H_q, H_kv, head_dim, 1, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  rc = cache_sizes(k_scale, v_scale, H_kv, head_dim, 1, block_size, num_blocks);
  if (rc != PAGED_ATTN_OK) return rc;
  const long long q_row = (long long)H_q * head_dim, kv_row = (long long)H_kv * head_dim;
  if (rows < 0 || q_stride < q_row || k_stride < kv_row || v_stride < kv_row ||
      q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0)
    return PAGED_ATTN_ERR_SIZES;
  if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16 != 0 || !(eps >= 0.f) ||
      std::isinf(eps) || (rotary_dim > 0 && (num_axes < 1 || max_positions < 1)))
    return PAGED_ATTN_ERR_ROPE;
  if (rows == 0) return PAGED_ATTN_OK;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q_out) ||
      !cache_pointers(k_cache, v_cache, k_scale, v_scale) || !aligned16(slot_map) ||
      (q_norm != nullptr && !aligned16(q_norm)) || (k_norm != nullptr && !aligned16(k_norm)))
    return PAGED_ATTN_ERR_POINTER;
  if (rotary_dim > 0 && (!aligned4(positions) || !aligned16(cos_sin) ||
                         (freq_axis != nullptr && !aligned16(freq_axis))))
    return PAGED_ATTN_ERR_POINTER;
  // q_out is q, row by row, or apart from what is read: a row written over another one is
  // written before or after that one is read
  const long long out_bytes = 2 * q_row * rows;
  if ((q_out != q || q_stride != q_row) &&
      meets_rows(q_out, out_bytes, q, 2 * q_row, 2 * q_stride, rows))
    return PAGED_ATTN_ERR_POINTER;
  if (meets_rows(q_out, out_bytes, k_new, 2 * kv_row, 2 * k_stride, rows) ||
      meets_rows(q_out, out_bytes, v_new, 2 * kv_row, 2 * v_stride, rows))
    return PAGED_ATTN_ERR_POINTER;
  int sms = 0;
  if ((rc = api_sms(&sms)) != PAGED_ATTN_OK) return rc;
  RopeParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k_new);
  p.v = static_cast<const __nv_bfloat16*>(v_new);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.slot_map = slot_map;
  p.positions = positions;
  p.freq_axis = freq_axis;
  p.cos_sin = cos_sin;
  p.q_norm = q_norm;
  p.k_norm = k_norm;
  p.eps = eps;
  p.rows = rows;
  p.axes = num_axes;
  p.max_positions = max_positions;
  p.R = rotary_dim;
  p.interleaved = interleaved != 0;
  p.H_q = H_q;
  p.H_kv = H_kv;
  p.D = head_dim;
  p.BS = block_size;
  p.num_blocks = num_blocks;
  p.status = api_check_status();
#ifdef PAGED_ATTN_WAIT_TEST
  p.test_skip_row = g_test_skip_row;
#endif
  return done(launch_rope_append(p, sms, static_cast<cudaStream_t>(stream)));
}

int paged_kv_compact(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                     const int32_t* qo_indptr, const int32_t* accepted,
                     const int32_t* block_tables, const int32_t* seq_lens, int32_t* seq_lens_out,
                     int num_seqs, int max_accept, int H_kv, int head_dim,
                     int max_blocks_per_seq, int block_size, long long num_blocks, void* stream) {
  int rc = cache_sizes(k_scale, v_scale, H_kv, head_dim, max_blocks_per_seq, block_size,
                       num_blocks);
  if (rc != PAGED_ATTN_OK) return rc;
  if (num_seqs < 0 || max_accept < 0 || max_accept > (1 << 30) ||
      (long long)num_seqs * H_kv > 0x7fffffffLL)
    return PAGED_ATTN_ERR_SIZES;
  if (num_seqs == 0) return PAGED_ATTN_OK;
  if (!cache_pointers(k_cache, v_cache, k_scale, v_scale) || !aligned16(qo_indptr) ||
      (max_accept > 0 && !aligned16(accepted)) || !aligned16(block_tables) ||
      !aligned16(seq_lens) || !aligned16(seq_lens_out) || seq_lens_out == seq_lens)
    return PAGED_ATTN_ERR_POINTER;
  CompactParams p;
  p.cache = cache_rows(k_cache, v_cache, k_scale, v_scale, H_kv, head_dim, block_size, num_blocks);
  p.qo_indptr = qo_indptr;
  p.accepted = accepted;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.seq_lens_out = seq_lens_out;
  p.num_seqs = num_seqs;
  p.max_accept = max_accept;
  p.maxb = max_blocks_per_seq;
  p.status = api_check_status();
  return done(launch_compact(p, static_cast<cudaStream_t>(stream)));
}

int paged_kv_fork(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                  int32_t* block_tables, int32_t* seq_lens, const int32_t* parents,
                  const int32_t* children, int32_t* block_refs, const int32_t* free_blocks,
                  const int32_t* free_count, int32_t* free_count_out, int32_t* refused,
                  int num_forks, int num_rows, int H_kv, int head_dim, int max_blocks_per_seq,
                  int block_size, int free_capacity, long long num_blocks, void* stream) {
  int rc = cache_sizes(k_scale, v_scale, H_kv, head_dim, max_blocks_per_seq, block_size,
                       num_blocks);
  if (rc != PAGED_ATTN_OK) return rc;
  if (num_forks < 0 || num_rows < 0 || free_capacity < 0 ||
      2LL * num_forks * H_kv > 0x3fffffffLL)
    return PAGED_ATTN_ERR_SIZES;
  if (!aligned4(free_count) || !aligned4(free_count_out) ||
      (refused != nullptr && !aligned4(refused)))
    return PAGED_ATTN_ERR_POINTER;
  if (num_forks > 0 &&
      (!cache_pointers(k_cache, v_cache, k_scale, v_scale) || !aligned16(block_tables) ||
       !aligned16(seq_lens) || !aligned16(parents) || !aligned16(children) ||
       !aligned16(block_refs) || (free_capacity > 0 && !aligned16(free_blocks))))
    return PAGED_ATTN_ERR_POINTER;
  int sms = 0;
  if ((rc = api_sms(&sms)) != PAGED_ATTN_OK) return rc;
  ForkParams p;
  p.cache = cache_rows(k_cache, v_cache, k_scale, v_scale, H_kv, head_dim, block_size, num_blocks);
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.parents = parents;
  p.children = children;
  p.block_refs = block_refs;
  p.free_blocks = free_blocks;
  p.free_count = free_count;
  p.free_count_out = free_count_out;
  p.refused = refused;
  p.num_forks = num_forks;
  p.num_rows = num_rows;
  p.maxb = max_blocks_per_seq;
  p.free_capacity = free_capacity;
  p.status = api_check_status();
#ifdef PAGED_ATTN_WAIT_TEST
  p.test_skip_page = g_test_skip_page;
#endif
  return done(launch_fork(p, sms, static_cast<cudaStream_t>(stream)));
}

int paged_kv_release(const int32_t* block_tables, const int32_t* seq_lens,
                     const int32_t* keep_lens, int32_t* block_refs, long long num_blocks,
                     int32_t* free_blocks, const int32_t* free_count, int32_t* seq_lens_out,
                     int32_t* free_count_out, int num_seqs, int max_blocks_per_seq,
                     int block_size, int free_capacity, void* stream) {
  int rc = api_validate_sizes(num_seqs, 1, 1, 64, max_blocks_per_seq, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  // (an entry's place in the table is its key, which has to fit an int)
  if (free_capacity < 0 || (long long)num_seqs * max_blocks_per_seq > 0x7fffffffLL ||
      (block_refs != nullptr && (num_blocks < 1 || num_blocks > 0x7fffffffLL)))
    return PAGED_ATTN_ERR_SIZES;
  if (!aligned4(free_count) || !aligned4(free_count_out) ||
      (block_refs != nullptr && !aligned16(block_refs)) ||
      (free_capacity > 0 && !aligned16(free_blocks)))
    return PAGED_ATTN_ERR_POINTER;
  if (num_seqs > 0 && (!aligned16(block_tables) || !aligned16(seq_lens) || !aligned16(keep_lens) ||
                       !aligned16(seq_lens_out)))
    return PAGED_ATTN_ERR_POINTER;
  ReleaseParams p;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.keep_lens = keep_lens;
  p.block_refs = block_refs;
  p.free_blocks = free_blocks;
  p.free_count = free_count;
  p.seq_lens_out = seq_lens_out;
  p.free_count_out = free_count_out;
  p.num_seqs = num_seqs;
  p.maxb = max_blocks_per_seq;
  p.BS = block_size;
  p.free_capacity = free_capacity;
  p.num_blocks = num_blocks;
  p.status = api_check_status();
  return done(launch_release(p, static_cast<cudaStream_t>(stream)));
}
