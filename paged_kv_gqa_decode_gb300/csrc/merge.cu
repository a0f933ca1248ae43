// The merge of the partial softmax states of query rows (tile_kernel.cuh's parts
// of a token range, and a decode's state over other tokens):
//
//     M = max_j m_j,   out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j
//
// in a fixed order, rounded once to bf16.  One warp per row: lane j holds the
// weight of part j, then every lane adds its columns of the parts.  It reads
// each state once, mostly from L2, right after the kernels that wrote them.
#include "ptx.cuh"
#include "tile.h"

namespace pagedattn {
namespace {

constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(const MergeParams p) {
  constexpr int E = D / 32;  // columns of a lane
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)p.total_q * p.H_q;
  const long long row = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int t = (int)(row / p.H_q);
  const bool parts = t >= __ldg(p.qo_indptr) && t < __ldg(p.qo_indptr + p.num_seqs);
  if (!parts && p.state == nullptr) return;  // a row no sequence owns
  const float2 ml = parts && lane < p.splits ? p.part_ml[lane * rows + row]
                                             : make_float2(-INFINITY, 0.f);
  const float* st = p.state != nullptr ? p.state + row * (D + 4) : nullptr;
  const float2 own = st != nullptr ? *reinterpret_cast<const float2*>(st)
                                   : make_float2(-INFINITY, 0.f);
  float M = fmaxf(ml.x, own.x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  // (empty states, m = -inf, weigh nothing; what they hold is not read.  States that hold a
  // NaN have m = NaN.)
  const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
  const float w_own = own.x == -INFINITY ? 0.f : fast_exp2(own.x - M);
  float l = ml.x == -INFINITY ? 0.f : ml.y * w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (own.x != -INFINITY) l += own.y * w_own;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  auto add = [&](const float* src, float wt) {
    float v[E];
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<float2*>(v + e) = *reinterpret_cast<const float2*>(src + lane * E + e);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, v[e], acc[e]);
  };
#pragma unroll 4
  for (int j = 0; j < p.splits; ++j) {
    const float wj = __shfl_sync(0xffffffffu, w, j);
    const float mj = __shfl_sync(0xffffffffu, ml.x, j);
    if (mj != -INFINITY) add(p.part_o + (j * rows + row) * D, wj);
  }
  if (own.x != -INFINITY) add(st + 4, w_own);
  const float inv = l > 0.f ? 1.f / l : 0.f;  // a row that saw no token: 0
  __nv_bfloat16* out = p.out + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
}

}  // namespace

cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.total_q * p.H_q;
  if (rows == 0) return cudaSuccess;
  const long long grid = (rows + kMergeWarps - 1) / kMergeWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.D == 64) return cudaLaunchKernelEx(&cfg, paged_merge_kernel<64>, p);
  if (p.D == 128) return cudaLaunchKernelEx(&cfg, paged_merge_kernel<128>, p);
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<256>, p);
}

}  // namespace pagedattn
