// Block tables, query offsets and the slot map of a serving step, from request
// lengths (include/paged_attn.h, paged_kv_assign).
//
// With L_s tokens held and n_s arriving, sequence s needs
//
//     need_s = ceil((L_s + n_s) / BS) - ceil(L_s / BS)
//
// fresh blocks; E_s is the running sum of need up to and including s.  It is
// served when E_s does not pass the free count (a sequence that needs none is
// always served), and takes the stack entries free_count - 1 - k for k in
// [E_s - need_s, E_s).  Row qo_indptr[s] + i is token t = L_s + i, at slot
// block * BS + t % BS.
//
// What bounds it: eight bytes written per token and the latency of one scan.
// Every CTA scans all the lengths into per-thread sums in shared memory and fills
// its part of the slot map from them.  When the new lengths or the free count go
// over the old ones, all those reads have to come before the writes: the grid is
// then one thread-block cluster (of one, two, four or eight CTAs by the rows there may
// be, one up to 4096), whose barrier separates them without a workspace; else it is as
// large as the rows ask for, up to 128 CTAs.
#include "assign.h"

namespace pagedattn {
namespace {

constexpr int kAssignThreads = 1024;
constexpr int kClusterCtas = 8;          // a portable cluster
constexpr int kMaxCtas = 128;
constexpr int kRowsPerCta = 4096;        // rows from which a further CTA joins
// Consecutive rows that a thread fills after one search: few while a CTA has
// threads for all rows (the rows of a thread are filled one after the other), else
// 64 bytes of slots.
constexpr int kFewRows = 2, kManyRows = 8;
constexpr int kStatusBadBlockId = 1, kStatusBadLengthGiven = 2;

// One sequence as the scan sees it.
struct Seq {
  int old_len, new_len;  // new_len: rows it owns (0 for a negative count)
  int old_pages, need;   // need: 0 when it cannot be served whatever is free
  bool fits;             // lengths valid and inside the table row
};

__device__ __forceinline__ Seq load_seq(const AssignParams& a, int s) {
  Seq x;
  const int L = a.seq_lens[s], n = a.new_lens[s];
  const long long cap = (long long)a.maxb * a.BS;
  x.old_len = L;
  x.new_len = max(n, 0);
  x.fits = L >= 0 && n >= 0 && (long long)L + n <= cap;
  x.old_pages = x.fits ? (L + a.BS - 1) / a.BS : 0;
  x.need = x.fits ? (int)(((long long)L + n + a.BS - 1) / a.BS) - x.old_pages : 0;
  return x;
}

// `tokens`, `blocks`: rows and fresh blocks of the sequences before this one.
__device__ __forceinline__ bool served(const AssignParams& a, const Seq& x, long long tokens,
                                       long long blocks, int free_count) {
  return x.fits && (x.need == 0 || blocks + x.need <= free_count) &&
         tokens + x.new_len <= a.max_new;
}

template <int kRowsPerThread, bool CLUSTER>
__global__ void __launch_bounds__(kAssignThreads) paged_kv_assign_kernel(const AssignParams a) {
  __shared__ long long tok[kAssignThreads + 1], blk[kAssignThreads + 1];
  __shared__ long long warp_tok[32], warp_blk[32];
  __shared__ int sm_refused;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int N = a.num_seqs;
  const int per = (N + kAssignThreads - 1) / kAssignThreads;  // sequences a thread sums
  const int free_count = min(max(*a.free_count, 0), a.free_capacity);

  // ---- 1. rows and fresh blocks ahead of each thread's sequences
  const int s0 = min(N, tid * per), s1 = min(N, s0 + per);
  long long t_sum = 0, b_sum = 0;
  for (int s = s0; s < s1; ++s) {
    const Seq x = load_seq(a, s);
    t_sum += x.new_len;
    b_sum += x.need;
  }
  long long t_inc = t_sum, b_inc = b_sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long tv = __shfl_up_sync(0xffffffffu, t_inc, o);
    const long long bv = __shfl_up_sync(0xffffffffu, b_inc, o);
    if (lane >= o) {
      t_inc += tv;
      b_inc += bv;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = t_inc;
    warp_blk[warp] = b_inc;
  }
  if (tid == 0) sm_refused = 0;
  __syncthreads();
  if (warp == 0) {
    long long tv = warp_tok[lane], bv = warp_blk[lane];
    const long long t_own = tv, b_own = bv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long tu = __shfl_up_sync(0xffffffffu, tv, o);
      const long long bu = __shfl_up_sync(0xffffffffu, bv, o);
      if (lane >= o) {
        tv += tu;
        bv += bu;
      }
    }
    warp_tok[lane] = tv - t_own;
    warp_blk[lane] = bv - b_own;
  }
  __syncthreads();
  tok[tid] = warp_tok[warp] + t_inc - t_sum;
  blk[tid] = warp_blk[warp] + b_inc - b_sum;
  if (tid == kAssignThreads - 1) {
    tok[kAssignThreads] = warp_tok[warp] + t_inc;
    blk[kAssignThreads] = warp_blk[warp] + b_inc;
  }
  __syncthreads();
  const long long total = tok[kAssignThreads];

  // ---- 2. slots, and the table entries of fresh pages (the row of a page's
  // first token writes its entry)
  const int shift = a.BS == 32 ? 5 : 4;
  const int step = (int)gridDim.x * kAssignThreads * kRowsPerThread;
  for (long long r0 = ((long long)blockIdx.x * kAssignThreads + tid) * kRowsPerThread;
       r0 < a.max_new; r0 += step) {
    int64_t out[kRowsPerThread];
#pragma unroll
    for (int j = 0; j < kRowsPerThread; ++j) out[j] = -1;
    if (r0 < total) {
      int lo = 0, hi = kAssignThreads - 1;  // largest group of sequences starting at or before r0
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tok[mid] <= r0)
          lo = mid;
        else
          hi = mid - 1;
      }
      int s = min(N - 1, lo * per);
      long long first = tok[lo], blocks = blk[lo];
      Seq x = load_seq(a, s);
      bool ok = served(a, x, first, blocks, free_count);
      int page = -1;   // the page `block` belongs to
      int block = 0;
#pragma unroll
      for (int j = 0; j < kRowsPerThread; ++j) {
        const long long r = r0 + j;
        if (r < total) {
          while (r >= first + x.new_len && s + 1 < N) {
            first += x.new_len;
            blocks += x.need;
            x = load_seq(a, ++s);
            ok = served(a, x, first, blocks, free_count);
            page = -1;
          }
          if (ok) {
            const int t = x.old_len + (int)(r - first);
            const int p = t >> shift;
            int32_t* entry = a.block_tables + (size_t)s * a.maxb + p;
            if (p != page) {
              page = p;
              block = p < x.old_pages
                          ? *entry
                          : a.free_blocks[free_count - 1 - (blocks + p - x.old_pages)];
              if (a.num_blocks > 0 && a.status != nullptr &&
                  (block < 0 || (long long)block >= a.num_blocks))
                atomicOr(a.status, kStatusBadBlockId);
            }
            if (p >= x.old_pages && t == p * a.BS) *entry = block;
            out[j] = (int64_t)block * a.BS + (t - p * a.BS);
          }
        }
      }
    }
    if (r0 + kRowsPerThread <= a.max_new) {
      longlong2* dst = reinterpret_cast<longlong2*>(a.slot_map + r0);
#pragma unroll
      for (int j = 0; j < kRowsPerThread / 2; ++j)
        dst[j] = make_longlong2(out[2 * j], out[2 * j + 1]);
    } else {
#pragma unroll
      for (int j = 0; j < kRowsPerThread; ++j)
        if (r0 + j < a.max_new) a.slot_map[r0 + j] = out[j];
    }
  }

  // ---- 3. every CTA has read the lengths and the free count: they may be overwritten
  if constexpr (CLUSTER) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
  } else {
    __syncthreads();
  }
  if (blockIdx.x != 0) return;
  long long first = tok[tid], blocks = blk[tid], used = 0;
  int refused = 0;
  for (int s = s0; s < s1; ++s) {
    const Seq x = load_seq(a, s);
    const bool ok = served(a, x, first, blocks, free_count);
    if (!ok) ++refused;
    if (!x.fits && a.num_blocks > 0 && a.status != nullptr)
      atomicOr(a.status, kStatusBadLengthGiven);
    a.qo_indptr[s] = (int)min(first, 0x7fffffffLL);
    a.seq_lens_out[s] = x.old_len + (ok ? x.new_len : 0);
    first += x.new_len;
    blocks += x.need;
    if (ok) used += x.need;
  }
  // the blocks taken: those of the served sequences (integer sums: any order)
  __syncthreads();  // warp_tok is reused
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) used += __shfl_xor_sync(0xffffffffu, used, o);
  if (lane == 0) warp_blk[warp] = used;
  if (refused) atomicAdd(&sm_refused, refused);
  __syncthreads();
  if (tid == 0) {
    long long all = 0;
    for (int w = 0; w < kAssignThreads / 32; ++w) all += warp_blk[w];
    *a.free_count_out = free_count - (int)all;
    a.qo_indptr[N] = (int)min(total, 0x7fffffffLL);
    if (a.refused != nullptr) *a.refused = sm_refused;
  }
}

}  // namespace

cudaError_t launch_assign(const AssignParams& a, cudaStream_t stream) {
  const bool in_place = a.seq_lens_out == a.seq_lens || a.free_count_out == a.free_count;
  const int most = in_place ? kClusterCtas : kMaxCtas;
  int ctas = 1;  // a power of two, by the rows there may be
  while (ctas < most && (long long)ctas * kRowsPerCta < a.max_new) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kAssignThreads);
  cfg.stream = stream;
  if (!in_place || ctas == 1)
    return ctas == 1 ? cudaLaunchKernelEx(&cfg, paged_kv_assign_kernel<kFewRows, false>, a)
                     : cudaLaunchKernelEx(&cfg, paged_kv_assign_kernel<kManyRows, false>, a);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_kv_assign_kernel<kManyRows, true>, a);
}

}  // namespace pagedattn
