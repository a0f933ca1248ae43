// Compaction, forks and release of the pages of a cache (include/paged_attn.h:
// paged_kv_compact, paged_kv_fork, paged_kv_release).
//
// All three move little: rows of a few accepted tokens, the last pages of forked
// sequences, four bytes a page.  What bounds them is latency, of dependent reads (a length,
// then a table entry, then rows) and of the steps that have to follow one another, so
// each is one launch that keeps several reads of a thread in flight.
#include <atomic>
#include <climits>
#include <cstdint>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "pages.h"
#include "ptx.cuh"

namespace pagedattn {
namespace {

namespace cg = cooperative_groups;

constexpr int kBadBlock = 1, kBadLength = 2, kTimeout = 4;

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (status != nullptr) atomicOr(status, bits);
}

__device__ __forceinline__ int clamped_length(int L, int maxb, int BS, int32_t* status) {
  const long long cap = (long long)maxb * BS;
  if (L < 0 || L > cap) report(status, kBadLength);
  return (int)min(max((long long)L, 0LL), cap);
}

// The two halves of the cluster's barrier.  (Not the aligned forms: the loops ahead of them end
// earlier for some threads of a warp than for others, and nothing says that the warp is
// together again.)
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Exclusive sum over the block's threads; the block's total in every thread.  `warp_sums`
// is of 32 ints and is free again after the call.
template <int THREADS>
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int w = lane < THREADS / 32 ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, THREADS / 32 - 1);
  const int before = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
  __syncthreads();
  return before + inc - v;
}

// ------------------------------------------------------------------ compaction
//
// Entry i of the list of sequence s moves the row of token ctx + accepted[i] to token ctx
// + i, ctx = L - q_len.  The list rises, so a row moves towards the front or stays, and
// accepted[j] >= j: rows written by one pass of a warp lie before every row that a later
// pass reads, and within a pass all reads come before the writes.  A warp has K or V of one KV
// head of a sequence; its CTA looks the rows' places up once for eight of them.
constexpr int kCompactThreads = 256, kCompactWarps = kCompactThreads / 32;
constexpr int kCompactUnroll = 4;

__global__ void __launch_bounds__(kCompactThreads) paged_kv_compact_kernel(const CompactParams p,
                                                                           int ctas_per_seq) {
  __shared__ int sm_n;
  __shared__ longlong2 sm_move[kCompactThreads];  // (from, to): cache rows of KV head 0
  griddep_wait();
  griddep_launch_dependents();  // (after the wait: what is ahead of this launch is complete)
  const int s = blockIdx.x / ctas_per_seq, part = blockIdx.x - s * ctas_per_seq;
  const int tid = threadIdx.x, BS = p.cache.BS, H = p.cache.H_kv;
  const int a = p.qo_indptr[s], b = p.qo_indptr[s + 1];
  const int q_len = (int)min(max((long long)b - a, 0LL), 0x7fffffffLL);
  const int len =
      clamped_length(p.seq_lens[s], p.maxb, BS, tid == 0 && part == 0 ? p.status : nullptr);
  const int ctx = len - q_len;
  const int32_t* list = p.accepted + (size_t)s * p.max_accept;
  const int32_t* table = p.block_tables + (size_t)s * p.maxb;
  // the cache row of a token and KV head 0, -1: there is none
  auto row_of = [&](int t) -> long long {
    if (t < 0) return -1;
    const int block = table[t / BS];
    if (block < 0 || block >= p.cache.num_blocks) {
      report(p.status, kBadBlock);
      return -1;
    }
    return (long long)block * H * BS + t % BS;
  };
  if (tid == 0) sm_n = p.max_accept;
  __syncthreads();
  // the list ends at its first entry that is not past the one before or not in the tree
  for (int i = tid; i < p.max_accept; i += kCompactThreads) {
    const int x = list[i], before = i > 0 ? list[i - 1] : -1;
    if (x <= before || x >= q_len) {
      atomicMin(&sm_n, i);
      break;
    }
  }
  __syncthreads();
  const int n = sm_n;
  if (part == 0 && tid == 0) p.seq_lens_out[s] = max(ctx + n, 0);
  const int pair = part * kCompactWarps + (tid >> 5);  // K of each KV head, then V
  const int g = pair < H ? pair : pair - H;
  uint8_t* cache = pair < H ? p.cache.k : p.cache.v;
  float* floats = pair < H ? p.cache.k_scale : p.cache.v_scale;
  const int chunks = p.cache.row_bytes / 16;  // 8 .. 32, a power of two
  const int rows = 32 / chunks, lane = tid & 31, c = lane % chunks, r = lane / chunks;
  for (int base = 0; base < n; base += kCompactThreads) {
    const int m = min(kCompactThreads, n - base);
    if (base > 0) __syncthreads();  // (every warp is done with the places before)
    if (tid < m) {
      const int i = base + tid, from = list[i];
      longlong2 mv = make_longlong2(-1, -1);
      if (from != i) {  // (else it is in its place)
        mv.x = row_of(ctx + from);
        mv.y = row_of(ctx + i);
      }
      sm_move[tid] = mv;
    }
    __syncthreads();
    if (pair >= 2 * H) continue;
    for (int i0 = 0; i0 < m; i0 += rows * kCompactUnroll) {
      uint4 x[kCompactUnroll];
      float f[kCompactUnroll];
      long long to[kCompactUnroll];
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int i = i0 + u * rows + r;
        to[u] = -1;
        f[u] = 0.f;
        if (i >= m) continue;
        const longlong2 mv = sm_move[i];
        if (mv.x < 0 || mv.y < 0) continue;
        const long long src = mv.x + (long long)g * BS;
        to[u] = mv.y + (long long)g * BS;
        x[u] = *(reinterpret_cast<const uint4*>(cache + src * p.cache.row_bytes) + c);
        if (floats != nullptr && c == 0) f[u] = floats[src];
      }
      __syncwarp();  // every row of this pass is read
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        if (to[u] < 0) continue;
        *(reinterpret_cast<uint4*>(cache + to[u] * p.cache.row_bytes) + c) = x[u];
        if (floats != nullptr && c == 0) floats[to[u]] = f[u];
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ forks
//
// Fork i needs a fresh block when its parent's last page is not full; R_i of the forks
// before it do, and it takes the stack entry free_count - 1 - R_i.  The runs to copy, one for
// each fork, tensor and KV head, are dealt to one CTA an SM in equal consecutive shares.  A
// CTA scans the parents' lengths once and looks all its forks up at once, a thread each; then each
// warp moves pieces of 4 KB by bulk copies into its place in shared memory and out of it,
// with no dependent read in between (512 forks of 64 prompts, 33 MB written: copied
// through registers, eight 16-byte chunks a thread in flight, 17 us).  The CTA with a fork's
// first run does its table row and the counts of its blocks.
constexpr int kForkThreads = 512, kForkWarps = kForkThreads / 32;
constexpr int kForkPiece = 4096;
// Calls of up to so many forks are looked through for children that are parents or children of
// other forks (with checks on): all pairs, 65536 forks 0.15 -> 6.1 ms.
constexpr int kForkChecked = 65536;
constexpr size_t kForkSmem = (size_t)kForkWarps * (kForkPiece + 8);

struct Fork {
  int parent, child, len, need;
  bool valid;
};

__device__ __forceinline__ Fork load_fork(const ForkParams& p, int i) {
  Fork f;
  f.parent = p.parents[i];
  f.child = p.children[i];
  f.valid = f.parent >= 0 && f.parent < p.num_rows && f.child >= 0 && f.child < p.num_rows &&
            f.parent != f.child;
  f.len = f.valid ? clamped_length(p.seq_lens[f.parent], p.maxb, p.cache.BS, nullptr) : 0;
  f.need = f.len % p.cache.BS != 0;
  return f;
}

__global__ void __launch_bounds__(kForkThreads, 1)
    paged_kv_fork_kernel(const ForkParams p, int share, int count_apart) {
  extern __shared__ __align__(128) uint8_t fork_smem[];
  __shared__ int before[kForkThreads];
  __shared__ int warp_sums[32];
  // forks of a batch: blocks copied from and to (-1: no copy) and the tokens of the last page
  __shared__ int sm_from[kForkThreads], sm_to[kForkThreads], sm_tail[kForkThreads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* place = fork_smem + warp * kForkPiece;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(fork_smem + kForkWarps * kForkPiece) + warp;
  if (lane == 0) {
    mbar_init(full_bar, 1);
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();  // (after the wait: what is ahead of this launch is complete)
  const int n = p.num_forks, BS = p.cache.BS;
  const int free_count = min(max(*p.free_count, 0), p.free_capacity);
  const int per = (n + kForkThreads - 1) / kForkThreads;  // forks that a thread sums
  const int i0 = (int)min((long long)n, (long long)tid * per);
  const int i1 = (int)min((long long)n, (long long)i0 + per);
  int needs = 0, invalid = 0;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    const Fork f = load_fork(p, i);
    needs += f.need;
    invalid += !f.valid;
  }
  int total, bad = 0;
  before[tid] = block_exclusive<kForkThreads>(needs, warp_sums, &total);
  if (blockIdx.x == 0) {
    block_exclusive<kForkThreads>(invalid, warp_sums, &bad);
    if (tid == 0) {
      if (!count_apart) *p.free_count_out = free_count - min(total, free_count);
      if (p.refused != nullptr) *p.refused = bad + max(total - free_count, 0);
    }
  }
  // ---- this CTA's runs: run r is fork r / pairs, tensor and KV head r % pairs
  const int H = p.cache.H_kv, pairs = 2 * H;
  const int runs = n * pairs;  // (the host has seen to it that it fits)
  const int first = (int)min((long long)runs, (long long)blockIdx.x * share);
  const int last = (int)min((long long)runs, (long long)first + share);
  const long long page = (long long)BS * p.cache.row_bytes;
  const int pieces = max(1, (int)page / kForkPiece);  // of a run at most: 1, 2 or 4
  const int shift = pieces == 4 ? 2 : pieces - 1;
  uint32_t phase = 0;
  bool lost = false;  // a copy did not come (never expected): this warp's barrier is not used again
  for (int f0 = first / pairs; (long long)f0 * pairs < last; f0 += kForkThreads) {
    const int r0 = max(first, f0 * pairs);  // this batch's runs
    const int r1 = (int)min((long long)last, ((long long)f0 + kForkThreads) * pairs);
    __syncthreads();  // (`before` is written; the batch before is done with)
    if (((long long)f0 + tid) * pairs < last) {
      const int i = f0 + tid;
      const Fork f = load_fork(p, i);
      int rank = before[i / per];
      for (int j = i / per * per; j < i; ++j) rank += load_fork(p, j).need;
      const bool given = f.valid && (!f.need || rank < free_count);
      const int full = f.len / BS;
      int from = -1, to = -1;
      if (given && f.need) {
        from = p.block_tables[(size_t)f.parent * p.maxb + full];
        to = p.free_blocks[free_count - 1 - rank];
      }
      if (i * pairs >= first) {  // the fork's first run is this CTA's
        if (given) {
          if (f.need) p.block_tables[(size_t)f.child * p.maxb + full] = to;
          if (p.seq_lens[f.parent] != f.len) report(p.status, kBadLength);
        } else if (!f.valid) {
          report(p.status, kBadLength);
        }
        if (f.child >= 0 && f.child < p.num_rows && f.child != f.parent)
          p.seq_lens[f.child] = given ? f.len : 0;
        if (p.status != nullptr && n <= kForkChecked && f.valid) {
          bool other = false;
          for (int j = 0; j < n; ++j)
            other |= p.parents[j] == f.child || (j != i && p.children[j] == f.child);
          if (other) report(p.status, kBadLength);
        }
      }
      if (given && f.need &&
          (from < 0 || from >= p.cache.num_blocks || to < 0 || to >= p.cache.num_blocks)) {
        report(p.status, kBadBlock);
        from = -1;
      }
      sm_from[tid] = from;
      sm_to[tid] = to;
      sm_tail[tid] = given ? f.len - full * BS : -1;  // (-1: no table row either)
    }
    __syncthreads();
    // ---- the rows of the last pages: a warp's first piece is under way while it works on
    // the table rows
    struct Piece {
      long long from, to;  // KV head pages
      uint8_t* cache;
      float* floats;
      int at, bytes, tail;
    };
    const long long most = (long long)(r1 - r0) * pieces;
    auto find = [&](long long& q, Piece& x) -> bool {  // this warp's next one from place q on
      for (; !lost && q < most; q += kForkWarps) {
        // (pieces is a power of two, at most four)
        const int r = r0 + (int)(q >> shift), piece = (int)q & (pieces - 1);
        const int k = (int)((uint32_t)r / (uint32_t)pairs) - f0, pair = r - (k + f0) * pairs;
        x.tail = sm_tail[k];
        x.at = piece * kForkPiece;
        x.bytes = min(kForkPiece, x.tail * p.cache.row_bytes - x.at);
        if (sm_from[k] < 0 || x.bytes <= 0) continue;
        const int h = pair < H ? pair : pair - H;
        x.cache = pair < H ? p.cache.k : p.cache.v;
        x.floats = pair < H ? p.cache.k_scale : p.cache.v_scale;
        x.from = (long long)sm_from[k] * H + h;
        x.to = (long long)sm_to[k] * H + h;
        return true;
      }
      return false;
    };
    auto load = [&](const Piece& x) {
      if (lane == 0) {
        mbar_arrive_expect_tx(full_bar, (uint32_t)x.bytes);
#ifdef PAGED_ATTN_WAIT_TEST
        if (x.at == 0 && x.to == p.test_skip_page) return;  // (armed and never filled)
#endif
        bulk_load(place, x.cache + x.from * page + x.at, (uint32_t)x.bytes, full_bar);
      }
      if (x.floats != nullptr && x.at == 0 && lane < x.tail)
        x.floats[x.to * BS + lane] = x.floats[x.from * BS + lane];
    };
    long long q = warp;
    Piece x;
    bool some = find(q, x);
    if (some) load(x);
    // ---- the table rows and the counts of the blocks in them: the warps shared out among the
    // forks whose first run is this CTA's
    const int own = max(f0, first / pairs + (first % pairs != 0));
    const int end = min(last / pairs + (last % pairs != 0), f0 + kForkThreads);
    const int forks = max(0, end - own);
    const int each = max(1, kForkWarps / max(forks, 1));  // warps of a fork
    for (int k = warp / each; k < forks; k += kForkWarps / each) {
      if (sm_tail[own - f0 + k] < 0) continue;
      const Fork f = load_fork(p, own + k);
      const int32_t* from = p.block_tables + (size_t)f.parent * p.maxb;
      int32_t* to = p.block_tables + (size_t)f.child * p.maxb;
#pragma unroll 4
      for (int j = warp % each * 32 + lane; j < f.len / BS; j += each * 32) {
        const int block = from[j];
        to[j] = block;
        if (block >= 0 && block < p.cache.num_blocks)
          atomicAdd(p.block_refs + block, 1);
        else
          report(p.status, kBadBlock);
      }
    }
    while (some) {
      bool landed = true;
      if (lane == 0) {
        landed = mbar_wait(full_bar, phase);
        if (landed) {
          bulk_store(x.cache + x.to * page + x.at, place, (uint32_t)x.bytes);
        } else {
          report(p.status, kTimeout);
          mbar_wait(full_bar, phase);  // (no copy may be in flight when the CTA exits)
        }
        bulk_store_read();  // the place is free again
      }
      lost = !__shfl_sync(0xffffffffu, landed, 0);
      phase ^= 1u;
      __syncwarp();
      q += kForkWarps;
      some = find(q, x);
      if (some) load(x);
    }
  }
  if (lane == 0) bulk_store_done();
}

// The free count where it is updated in place: the kernel above, whose CTAs all read the
// old one, has completed.
__global__ void __launch_bounds__(kForkThreads, 1) paged_kv_fork_count_kernel(const ForkParams p) {
  __shared__ int warp_sums[32];
  griddep_wait();
  griddep_launch_dependents();
  int needs = 0, total;
  for (int i = threadIdx.x; i < p.num_forks; i += kForkThreads) needs += load_fork(p, i).need;
  block_exclusive<kForkThreads>(needs, warp_sums, &total);
  if (threadIdx.x == 0) {
    const int free_count = min(max(*p.free_count, 0), p.free_capacity);
    *p.free_count_out = free_count - min(total, free_count);
  }
}

// ------------------------------------------------------------------ release
//
// Entry (s, p) of the table is released when it lies past the page of the last kept token
// and in the sequence; its key is e = s * maxb + p.  block_refs holds a block's holders past
// the first, so with m of the released entries its count falls by m, and it is free when
// the count is then below zero.  Which of its entries places it on the stack must not
// hang on the order of atomics: it is the one of lowest key.  Steps, each one after all of
// the one before:
//
//   1. refs[b] -= 1 for each entry
//   2. where refs[b] < 0: refs[b] = min(refs[b], INT_MIN + e), so the lowest key remains
//   3. entries with refs[b] == INT_MIN + e are counted, the counts summed
//   4. those write their block to the stack at their rank and refs[b] = 0
//
// When every entry finds a count of zero in step 1 (nothing released is shared: all blocks are
// distinct), each one places its block, its rank is its place among the entries, and steps 2
// and 3 fall away.
//
// The grid is one thread-block cluster, whose barrier separates the steps (and all reads
// of lengths and the free count from their writes in place).  A thread has a run of
// consecutive entries, so ranks need one scan.
constexpr int kReleaseThreads = 1024;
constexpr int kReleaseCtas = 16, kPortableCtas = 8;  // the largest cluster, where the device has room
constexpr int kReleaseBatch = 8;  // entries of a thread in flight

__global__ void __launch_bounds__(kReleaseThreads) paged_kv_release_kernel(const ReleaseParams p) {
  __shared__ int before[kReleaseThreads];  // entries ahead of each thread's sequences
  __shared__ int warp_sums[32];
  __shared__ int sm_count, sm_plain;
  griddep_wait();
  griddep_launch_dependents();  // (after the wait: what is ahead of this launch is complete)
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, N = p.num_seqs;
  const int ctas = (int)gridDim.x, cta = (int)blockIdx.x;
  const int free_count = min(max(*p.free_count, 0), p.free_capacity);
  const int per = (N + kReleaseThreads - 1) / kReleaseThreads;
  const int s0 = (int)min((long long)N, (long long)tid * per);
  const int s1 = (int)min((long long)N, (long long)s0 + per);
  // first released page and the number of them
  auto span = [&](int s, int& first) -> int {
    const int len = clamped_length(p.seq_lens[s], p.maxb, p.BS, nullptr);
    const int keep = min(max(p.keep_lens[s], 0), len);
    first = (keep + p.BS - 1) / p.BS;
    return (len + p.BS - 1) / p.BS - first;
  };
  int own = 0, all;
  for (int s = s0; s < s1; ++s) {
    int first;
    own += span(s, first);
    if (cta == 0) clamped_length(p.seq_lens[s], p.maxb, p.BS, p.status);
  }
  before[tid] = block_exclusive<kReleaseThreads>(own, warp_sums, &all);
  __syncthreads();
  // ---- this thread's run of entries [e0, e1) of all the released ones
  const int run = (int)(((long long)all + ctas * kReleaseThreads - 1) / (ctas * kReleaseThreads));
  const long long at = ((long long)cta * kReleaseThreads + tid) * run;
  // (unsigned, as a batch behind the last one may begin past an int)
  const uint32_t e0 = (uint32_t)min((long long)all, at), e1 = (uint32_t)min((long long)all, at + run);
  int start_s = 0, start_p = 0, start_left = 0;  // sequence, page and pages left at e0
  if (e0 < e1) {
    int lo = 0, hi = kReleaseThreads - 1;  // the last group of sequences starting at or before e0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= (int)e0)
        lo = mid;
      else
        hi = mid - 1;
    }
    int ahead = before[lo];
    start_s = lo * per;
    for (;;) {
      int first;
      const int n = span(start_s, first);
      if ((int)e0 < ahead + n || start_s + 1 >= N) {
        start_p = first + ((int)e0 - ahead);
        start_left = ahead + n - (int)e0;
        break;
      }
      ahead += n;
      ++start_s;
    }
  }
  // The entries of a batch: keys (-1: none) and blocks.  A run of one batch, the usual one, is
  // looked up once; a longer one in every step.
  int key[kReleaseBatch], block[kReleaseBatch];
  int s = start_s, page = start_p, left = start_left;
  uint32_t e_at = 0;  // first of the batch
  auto look_up = [&](uint32_t e) {
#pragma unroll
    for (int u = 0; u < kReleaseBatch; ++u) {
      key[u] = -1;
      if (e + u >= e1) continue;
      while (left <= 0 && s + 1 < N) left = span(++s, page);
      key[u] = s * p.maxb + page;
      ++page;
      --left;
    }
#pragma unroll
    for (int u = 0; u < kReleaseBatch; ++u) block[u] = key[u] >= 0 ? p.block_tables[key[u]] : -1;
#pragma unroll
    for (int u = 0; u < kReleaseBatch; ++u) {
      // (a block that is none has no count and is not freed)
      if (key[u] < 0) continue;
      if (block[u] < 0 || (p.block_refs != nullptr && block[u] >= p.num_blocks)) {
        report(p.status, kBadBlock);
        key[u] = -1;
      }
    }
  };
  const bool once = run <= kReleaseBatch;
  if (once) look_up(e0);
  auto each_batch = [&](auto&& f) {
    s = start_s;
    page = start_p;
    left = start_left;
    for (e_at = e0; e_at < e1; e_at += kReleaseBatch) {
      if (!once) look_up(e_at);
      f();
    }
  };
  int refs[kReleaseBatch];
  auto counts = [&] {  // (written by other SMs: not from the L1)
#pragma unroll
    for (int u = 0; u < kReleaseBatch; ++u)
      refs[u] = key[u] >= 0 && p.block_refs != nullptr ? __ldcg(p.block_refs + block[u]) : 0;
  };
  auto places = [&](int u) -> bool {
    return key[u] >= 0 && (p.block_refs == nullptr || refs[u] == INT_MIN + key[u]);
  };
  // A value of each CTA's shared memory: lane c of a warp gets CTA c's.
  auto of_cta = [&](int* x, int none) -> int {
    return lane < ctas ? *cluster.map_shared_rank(x, lane) : none;
  };
  // ---- 1.
  int old[kReleaseBatch];  // counts before, of a run of one batch
  bool plain = true;
  each_batch([&] {
    int was[kReleaseBatch];
#pragma unroll
    for (int u = 0; u < kReleaseBatch; ++u)
      was[u] = key[u] >= 0 && p.block_refs != nullptr ? atomicSub(p.block_refs + block[u], 1) : 0;
#pragma unroll
    for (int u = 0; u < kReleaseBatch; ++u) {
      old[u] = was[u];
      // (an entry that is none would leave a gap in the ranks)
      if (was[u] != 0 || (key[u] < 0 && e_at + u < e1)) plain = false;
    }
  });
  plain = __syncthreads_and(plain) != 0;
  if (tid == 0) sm_plain = plain;
  cluster.sync();
  // (the same in all CTAs, whatever the caller does to the lengths meanwhile: they all read
  // the same words)
  plain = __all_sync(0xffffffffu, of_cta(&sm_plain, 1) != 0) != 0;
  // What all paths end with: every CTA has read the lengths and the free count by now, except
  // those of a long run, which reads the lengths once more.
  auto write_lengths = [&](int total) {
    for (uint32_t i = cta * kReleaseThreads + tid; i < (uint32_t)N; i += ctas * kReleaseThreads) {
      const int len = clamped_length(p.seq_lens[i], p.maxb, p.BS, nullptr);
      p.seq_lens_out[i] = min(max(p.keep_lens[i], 0), len);
    }
    if (cta == 0 && tid == 0)
      *p.free_count_out = (int)min((long long)free_count + total, (long long)p.free_capacity);
  };
  auto place = [&](int u, int rank) {
    const long long to = (long long)free_count + rank;
    if (to < p.free_capacity)
      p.free_blocks[to] = block[u];
    else
      report(p.status, kBadLength);
    if (p.block_refs != nullptr) p.block_refs[block[u]] = 0;
  };
  if (plain) {
    if (once) {
      cluster_arrive();
      write_lengths(all);
    }
    each_batch([&] {
#pragma unroll
      for (int u = 0; u < kReleaseBatch; ++u)
        if (key[u] >= 0) place(u, (int)(e_at + u));
    });
    if (!once) cluster_arrive();
    cluster_wait();  // (no CTA exits before its word is read)
    if (!once) write_lengths(all);
    return;
  }
  // ---- 2.
  if (p.block_refs != nullptr) {
    each_batch([&] {
      // (a count that was zero or less before is below zero now)
#pragma unroll
      for (int u = 0; u < kReleaseBatch; ++u)
        refs[u] = key[u] < 0 ? 0 : once && old[u] <= 0 ? -1 : __ldcg(p.block_refs + block[u]);
#pragma unroll
      for (int u = 0; u < kReleaseBatch; ++u)
        if (refs[u] < 0) atomicMin(p.block_refs + block[u], INT_MIN + key[u]);
    });
    cluster.sync();
  }
  // ---- 3.
  int freed = 0, in_cta;
  each_batch([&] {
    counts();
#pragma unroll
    for (int u = 0; u < kReleaseBatch; ++u) freed += places(u);
  });
  int rank = block_exclusive<kReleaseThreads>(freed, warp_sums, &in_cta);
  if (tid == 0) sm_count = in_cta;
  cluster.sync();
  const int in_it = of_cta(&sm_count, 0);
  const int total = __reduce_add_sync(0xffffffffu, in_it);
  rank += __reduce_add_sync(0xffffffffu, lane < cta ? in_it : 0);
  if (once) {
    cluster_arrive();
    write_lengths(total);
  }
  // ---- 4.
  each_batch([&] {
    // (looked up again, a block's other entries see the winner's key or the zero written over
    // it: not theirs)
    if (!once) counts();
#pragma unroll
    for (int u = 0; u < kReleaseBatch; ++u) {
      if (places(u)) place(u, rank++);
    }
  });
  if (!once) cluster_arrive();
  cluster_wait();
  if (!once) write_lengths(total);
}

cudaLaunchAttribute dependent_launch() {  // may be scheduled while the kernel before it ends
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

}  // namespace

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  const int per_seq = (2 * p.cache.H_kv + kCompactWarps - 1) / kCompactWarps;
  const long long ctas = (long long)p.num_seqs * per_seq;
  if (ctas == 0) return cudaSuccess;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kCompactThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {dependent_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_kv_compact_kernel, p, per_seq);
}

cudaError_t launch_fork(const ForkParams& p, int sms, cudaStream_t stream) {
  static std::atomic<bool> limit_raised[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !limit_raised[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(paged_kv_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kForkSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) limit_raised[dev].store(true, std::memory_order_release);
  }
  const int runs = 2 * p.num_forks * p.cache.H_kv, share = runs < sms ? 1 : (runs + sms - 1) / sms;
  const int apart = p.free_count_out == p.free_count;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(runs < 1 ? 1 : (runs + share - 1) / share));
  cfg.blockDim = dim3(kForkThreads);
  cfg.dynamicSmemBytes = kForkSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {dependent_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_kv_fork_kernel, p, share, apart);
  if (e != cudaSuccess || !apart) return e;
  cfg.gridDim = dim3(1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_kv_fork_count_kernel, p);
}

cudaError_t launch_release(const ReleaseParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kReleaseThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {{}, dependent_launch()};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  auto set_ctas = [&](int n) {
    cfg.gridDim = dim3((unsigned)n);
    attr[0].val.clusterDim.x = (unsigned)n;
  };
  static std::atomic<int> most[64];  // CTAs of a cluster that this device takes
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int limit = dev >= 0 && dev < 64 ? most[dev].load(std::memory_order_acquire) : 0;
  if (limit == 0) {
    e = cudaFuncSetAttribute(paged_kv_release_kernel,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    int clusters = 0;
    set_ctas(kReleaseCtas);
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters, paged_kv_release_kernel, &cfg);
    if (e != cudaSuccess) return e;
    limit = clusters > 0 ? kReleaseCtas : kPortableCtas;
    if (dev >= 0 && dev < 64) most[dev].store(limit, std::memory_order_release);
  }
  const long long entries = (long long)p.num_seqs * p.maxb;
  int ctas = 1;  // by the entries there may be
  while (ctas < limit && (long long)ctas * 4 * kReleaseThreads < entries) ctas *= 2;
  set_ctas(ctas);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, paged_kv_release_kernel, p);
}

}  // namespace pagedattn
