// Attention of many query rows over the paged KV cache on the 5th-generation
// tensor cores: chunks of a prompt, drafted tokens, and the members of a group
// that share a prefix (include/paged_attn.h).
//
// One piece of work is (sequence, KV head, tile of query rows, part of the
// token range).  The q_len * G rows of a KV head are token-major (row r is query
// r / G, head r % G), so a K/V tile read once serves the whole group and up to
// 256 rows.  Per 128 x 128 tile of scores and D = 128:
//
//   S = Q K^T   tcgen05.mma, Q and K in shared memory, S (fp32) in tensor memory
//   P = 2^(x - m), x the scaled, capped, biased, masked score in the log2 domain
//   O = O + P V tcgen05.mma, P (bf16) in tensor memory, V in shared memory
//
// Roles: one warp copies pages (TMA, one box per page and 128-byte column half,
// K and V tiles through one ring), one thread issues the products, and each warpgroup
// of 128 threads owns the 128 rows of a score tile, a thread per row, so the
// running maximum and sum never leave a thread.  Two warpgroups (head_dim 64 and
// 128) work on different score tiles while the products of the other run: on the
// two row tiles of a full piece, or, when a piece has at most 128 rows, on
// alternate token tiles of the same rows, merged at the end.  head_dim 256 has
// one warpgroup with two score buffers (its accumulators take half the tensor
// memory).
//
// A score tile is read from tensor memory twice, in chunks of 64 columns: for its
// maximum, then for its weights.  (Holding all 128 scores of a row in registers
// between the two spills at the 168 registers that ten warps leave a thread.)
//
// The running maximum is raised only when a tile passes it by 2^8, so most tiles
// do not rescale O in tensor memory; the weights (at most 2^8) are rounded to bf16
// for the product, as relative accuracy is what counts there, and summed in fp32.
//
// Masks: a query at position pos sees [lo, hi] and the prefix [0, pre).  Token
// tiles that no row of the piece sees are not walked, their pages not read; in
// the few tiles where an interval ends the scores are selected, and V rows that no
// row of the piece sees, which may hold anything, are zeroed in shared memory
// before the product.
#pragma once

#include <atomic>

#include "tcgen05.cuh"
#include "tile.h"

namespace pagedattn {

constexpr int kTileStatusBadBlock = 1, kTileStatusBadLength = 2, kTileStatusTimeout = 4;
constexpr float kTileLazyMax = 8.f;
constexpr int kTileTmemColumns = 512;

template <int D>
struct TileShape {
  static constexpr int kGroups = D == 256 ? 1 : 2;        // softmax warpgroups
  static constexpr int kRows = tile_rows(D);
  static constexpr int BN = tile_tokens(D);
  static constexpr int kHalves = D / 64;                  // 128-byte column halves of a row
  static constexpr int kQTileBytes = 128 * D * 2;         // one 128-row query tile
  static constexpr int kSlotBytes = BN * D * 2;           // one K or V tile
  static constexpr int kSlots = D == 64 ? 8 : 5;
  // softmax warpgroups, then a producer and a product warp
  static constexpr int kThreads = kGroups * 128 + 64;
  static constexpr int kOCol = 256;                       // first accumulator column
  static constexpr int kBarOff = kGroups * kQTileBytes + kSlots * kSlotBytes;
  static constexpr int kSmem = kBarOff + 1024 + 1024;     // + barriers and scalars, + alignment
};

template <int D>
__global__ void __launch_bounds__(TileShape<D>::kThreads, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const TileParams p) {
  using T = TileShape<D>;
  constexpr int kGroups = T::kGroups, kRows = T::kRows, BN = T::BN, kHalves = T::kHalves;
  constexpr int kSlots = T::kSlots, kThreads = T::kThreads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sm_q = smem;
  uint8_t* sm_kv = smem + kGroups * T::kQTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::kBarOff);
  uint64_t* full = bars;                  // [kSlots] a tile has landed
  uint64_t* empty = bars + kSlots;        // [kSlots] its products are done
  uint64_t* s_full = bars + 2 * kSlots;   // [2] scores ready
  uint64_t* p_full = s_full + 2;          // [2] weights stored, O rescaled
  uint64_t* o_done = p_full + 2;          // [2] product with V done
  uint64_t* q_full = o_done + 2;
  uint64_t* drain = q_full + 1;
  int* sm_i = reinterpret_cast<int*>(smem + T::kBarOff + 512);
  // sm_i: [0] TMEM address, [1] sequence, [2] row tile, [3] min lo, [4] max hi,
  // [8..24) warp sums of the tile search
  uint32_t* sm_tmem = reinterpret_cast<uint32_t*>(sm_i);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int N = p.num_seqs, G = p.G;
  auto report = [&](int bits) { atomicOr(p.status, bits); };

  griddep_launch_dependents();
  if (tid == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  griddep_wait();

  // ---- which piece: tiles are numbered through the sequences, the last first (a
  // causal batch's longest pieces start first)
  const int split = (int)(blockIdx.x % p.splits);
  const int g = (int)(blockIdx.x / p.splits % p.H_kv);
  const int tiles_bound = (int)(gridDim.x / ((unsigned)p.splits * p.H_kv));
  const int want = tiles_bound - 1 - (int)(blockIdx.x / ((unsigned)p.splits * p.H_kv));
  // rows of sequence s, and the first of them (clamped into [0, total_q])
  auto rows_at = [&](int s, int& first) -> int {
    first = min(max(__ldg(p.qo_indptr + s), 0), p.total_q);
    return max(min(__ldg(p.qo_indptr + s + 1), p.total_q) - first, 0);
  };
  auto tiles_of = [&](int s) -> int {
    int first;
    return (int)(((long long)rows_at(s, first) * G + kRows - 1) / kRows);
  };
  {
    const int per = (N + kThreads - 1) / kThreads;
    const int s0 = min(N, tid * per), s1 = min(N, s0 + per);
    int local = 0;
    for (int s = s0; s < s1; ++s) local += tiles_of(s);
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sm_i[8 + warp] = incl;
    if (tid == 0) {
      sm_i[1] = -1;
      sm_i[3] = 0x7fffffff;
      sm_i[4] = -1;
      for (int i = 0; i < kSlots; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], 128);
        mbar_init(&o_done[i], 1);
      }
      mbar_init(q_full, kGroups * 128);
      mbar_init(drain, 1);
      fence_barrier_init();
    }
    __syncthreads();
    int before = incl - local;
    for (int w = 0; w < warp; ++w) before += sm_i[8 + w];
    if (want >= before && want < before + local) {
      int s = s0;
      for (;;) {
        const int n = tiles_of(s);
        if (want < before + n) break;
        before += n;
        ++s;
      }
      sm_i[1] = s;
      sm_i[2] = want - before;
    }
    __syncthreads();
  }
  const int s = sm_i[1];
  if (s < 0) return;  // the bound on tiles is not reached
  const int row0 = sm_i[2] * kRows;  // first row of the tile among the q_len * G of the KV head
  int qo;
  const int q_len = rows_at(s, qo);
  int len = __ldg(p.seq_lens + s);
  {
    const long long cap = (long long)p.maxb * p.BS;
    if (len < 0 || (long long)len > cap) {
      if (p.num_blocks > 0 && tid == 0) report(kTileStatusBadLength);
      len = (int)min(max((long long)len, 0LL), cap);
    }
  }
  const int pre = p.prefix_lens != nullptr ? min(max(__ldg(p.prefix_lens + s), 0), len) : 0;
  const int n_rows = (int)min((long long)kRows, (long long)q_len * G - row0);
  const bool both = kGroups == 2 && n_rows > 128;  // a row tile per warpgroup

  // ---- this thread's row (softmax threads) and the tokens it sees
  const int wg = warp >> 2;                // softmax warpgroup (kGroups and up: other roles)
  const int r128 = tid & 127;
  const int rr = row0 + (both ? wg * 128 : 0) + r128;
  const bool softmax_thread = wg < kGroups;
  const int qi = rr / G;
  const bool valid = softmax_thread && (long long)rr < (long long)q_len * G && rr < row0 + kRows;
  long long q_row = -1;                    // row of q / out viewed as rows of D
  int lo = 0, hi = 0x7fffffff, pos = 0, head = 0;
  if (valid) {
    head = g * G + (rr - qi * G);
    q_row = (long long)(qo + qi) * p.H_q + head;
    if (p.tail_lens != nullptr) {
      const int tail = min(max(__ldg(p.tail_lens + qo + qi), 0), p.tail_cap);
      pos = (int)min((long long)len - 1 + tail, 0x7fffffffLL);
      hi = len - 1;
    } else {
      pos = len - q_len + qi;
      hi = p.causal ? pos : len - 1;
    }
    if (p.window > 0) lo = (int)max(0LL, (long long)pos - p.window + 1);
    if (p.doc_starts != nullptr) lo = max(lo, min(__ldg(p.doc_starts + qo + qi), len));
    if (lo <= hi) {
      atomicMin(&sm_i[3], lo);
      atomicMax(&sm_i[4], hi);
    }
  }
  // ---- the query rows, swizzled for the products (128-byte rows, 16-byte chunk c
  // of row r at c ^ (r % 8)); with one row tile the two warpgroups share the work
  if (softmax_thread) {
    const int chunks = D / 8;
    const int c0 = both || kGroups == 1 ? 0 : wg * (chunks / 2);
    const int c1 = both || kGroups == 1 ? chunks : c0 + chunks / 2;
    uint8_t* tile = sm_q + (both ? wg * T::kQTileBytes : 0);
    for (int c = c0; c < c1; ++c) {
      const uint4 v = valid ? __ldg(reinterpret_cast<const uint4*>(p.q + q_row * D) + c)
                            : make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(tile + (c >> 3) * (128 * 128) + r128 * 128 +
                                (((c & 7) ^ (r128 & 7)) << 4)) = v;
    }
    fence_proxy_async_shared();
    mbar_arrive(q_full);
  }
  __syncthreads();
  const int min_lo = sm_i[3], max_hi = sm_i[4];

  // ---- the walk over token tiles: those of the prefix, then those from the first
  // to the last one an interval touches
  const int head_tiles = (pre + BN - 1) / BN;
  int skip = 0, n_all = head_tiles;
  if (min_lo <= max_hi) {
    skip = max(0, min_lo / BN - head_tiles);
    n_all = max(head_tiles, max_hi / BN + 1 - skip);
  }
  // the parts: at least two tiles each, so that short ranges are not split
  const int parts = max(1, min(p.splits, n_all / 2));
  const int k0 = split < parts ? (int)((long long)split * n_all / parts) : 0;
  const int k1 = split < parts ? (int)((long long)(split + 1) * n_all / parts) : 0;
  const int n = k1 - k0;
  auto token_of = [&](int j) -> int {  // first token of this part's tile j
    const int k = k0 + j;
    return (k < head_tiles ? k : k + skip) * BN;
  };
  const long long part_rows = (long long)p.total_q * p.H_q;
  if (n <= 0) {  // nothing to see here: a zero row, or an empty state
    if (valid && (both || wg == 0)) {
      if (p.single) {
        uint4* o = reinterpret_cast<uint4*>(p.out + q_row * D);
        for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
      } else {
        p.part_ml[split * part_rows + q_row] = make_float2(-INFINITY, 0.f);
      }
    }
    return;
  }

  constexpr int kProducerWarp = kGroups * 4, kMmaWarp = kGroups * 4 + 1;
  if (warp == kMmaWarp) tmem_alloc(sm_tmem, kTileTmemColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sm_tmem;

  // Items of the ring, in the order the products first use them: K_0, then K_j+1
  // and V_j for every j, then the last V.
  auto item_k = [&](int j) { return j == 0 ? 0 : 2 * j - 1; };
  auto item_v = [&](int j) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; };
  // Steps: one score tile each, alternating between the two score buffers.
  const int steps = both ? 2 * n : n;
  auto tile_of_step = [&](int k) { return both ? k >> 1 : k; };

  if (warp == kProducerWarp) {
    // =================================================================== producer
    const uint64_t policy = l2_evict_first_policy();
    const int pages = BN / p.BS, boxes = pages * kHalves;  // at most 16: one per lane
    const int page = lane % pages, half = lane / pages;
    auto block_of = [&](int j) -> int {  // this lane's page of tile j, -1: no row of it is seen
      if (j >= n || lane >= boxes) return -1;
      const int t0 = token_of(j) + page * p.BS;
      const bool seen = t0 < pre || (t0 <= max_hi && t0 + p.BS > min_lo);
      if (!seen) return -1;
      const int pb = __ldg(p.block_tables + (size_t)s * p.maxb + t0 / p.BS);
      if (p.num_blocks > 0 && (pb < 0 || (long long)pb >= p.num_blocks) && half == 0)
        report(kTileStatusBadBlock);  // the copy's bounds check reads it as zeros
      return pb;
    };
    int b_cur = block_of(0), b_next = block_of(1);  // blocks of tiles j and j + 1
    bool ok = true;
    int it = 0;
    auto copy = [&](const CUtensorMap* map, int pb) {
      const int slot = it % kSlots;
      ok = ok && mbar_wait(&empty[slot], (uint32_t)((it / kSlots) & 1) ^ 1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (lane == 0) mbar_arrive_expect_tx(&full[slot], T::kSlotBytes);
      __syncwarp();
      if (lane < boxes)  // a block id of -1 is out of the map's bounds: zeros
        tma_load_4d(sm_kv + slot * T::kSlotBytes + half * (BN * 128) + page * p.BS * 128, map,
                    &full[slot], 0, g * p.BS, half, pb < 0 ? -1 : pb, policy);
      ++it;
    };
    copy(&tm_k, b_cur);
    for (int j = 0; j < n; ++j) {
      const int b_after = block_of(j + 2);
      if (j + 1 < n) copy(&tm_k, b_next);
      copy(&tm_v, b_cur);
      b_cur = b_next;
      b_next = b_after;
    }
    if (!ok && lane == 0) report(kTileStatusTimeout);
    // no copy may be in flight when the CTA exits
    for (int i = max(0, it - kSlots); i < it; ++i)
      if (!mbar_wait(&full[i % kSlots], (uint32_t)((i / kSlots) & 1)) && lane == 0)
        report(kTileStatusTimeout);
  } else if (warp == kMmaWarp) {
    // ==================================================================== products
    if (lane == 0) {
      constexpr uint32_t kDescS = instr_desc(128, BN, false), kDescO = instr_desc(128, D, true);
      bool ok = mbar_wait(q_full, 0);
      tc_fence_after();
      const uint32_t q_addr = smem_addr(sm_q), kv_addr = smem_addr(sm_kv);
      auto wait_item = [&](int item) {
        ok = ok && mbar_wait(&full[item % kSlots], (uint32_t)((item / kSlots) & 1));
      };
      auto scores = [&](int k) {  // S[k & 1] = Q K^T
        const int j = tile_of_step(k), item = item_k(j);
        if (!both || !(k & 1)) wait_item(item);
        if (!ok) return;
        tc_fence_after();
        const uint32_t qa = q_addr + (both && (k & 1) ? T::kQTileBytes : 0);
        const uint32_t ka = kv_addr + (item % kSlots) * T::kSlotBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + (k & 1) * BN,
                 smem_desc(qa + (kk >> 2) * (128 * 128) + (kk & 3) * 32, 16, 1024),
                 smem_desc(ka + (kk >> 2) * (BN * 128) + (kk & 3) * 32, 16, 1024), kDescS, kk > 0);
        mma_commit(&s_full[k & 1]);
        if (!both || (k & 1)) mma_commit(&empty[item % kSlots]);
      };
      auto values = [&](int k) {  // O = O + P[k & 1] V
        const int j = tile_of_step(k), item = item_v(j);
        ok = ok && mbar_wait(&p_full[k & 1], (uint32_t)((k >> 1) & 1));
        if (!both || !(k & 1)) wait_item(item);
        if (!ok) return;
        tc_fence_after();
        const int o = kGroups == 2 ? (k & 1) : 0;
        const bool first = kGroups == 2 ? k < 2 : k == 0;
        const uint32_t va = kv_addr + (item % kSlots) * T::kSlotBytes;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          mma_ts(tmem + T::kOCol + o * D, tmem + (k & 1) * BN + kk * 8,
                 smem_desc(va + kk * 2048, BN * 128, 1024), kDescO, !first || kk > 0);
        mma_commit(&o_done[o]);
        if (!both || (k & 1)) mma_commit(&empty[item % kSlots]);
      };
      scores(0);
      if (steps > 1) scores(1);
      for (int k = 0; k < steps; ++k) {
        values(k);
        if (k + 2 < steps) scores(k + 2);
      }
      mma_commit(drain);
      if (!mbar_wait(drain, 0)) ok = false;
      if (!ok) report(kTileStatusTimeout);
    }
    __syncwarp();
  } else {
    // ===================================================================== softmax
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lane_base + T::kOCol + (kGroups == 2 ? wg * D : 0);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    int done = 0;  // products with V waited for
    const float slope = valid && p.slopes != nullptr
                            ? __ldg(p.slopes + head) * 1.4426950408889634f
                            : 0.f;
    const bool capped = p.cap_log2 > 0.f, biased = p.slopes != nullptr;
    // raw scores serve where the log2 score is a positive multiple of them
    const bool raw = !capped && !biased && p.scale_log2 > 0.f;
    const bool ordered = !biased && p.scale_log2 > 0.f;
    const float factor = raw ? p.scale_log2 : 1.f;
    const int last_seen = max(max_hi, pre - 1);
    constexpr int kStep = kGroups;  // this warpgroup's steps: wg, wg + kStep, ...
    for (int k = wg; k < steps; k += kStep) {
      const int buf = k & 1, j = tile_of_step(k), t0 = token_of(j);
      const uint32_t s_addr = tmem + lane_base + buf * BN;
      ok = ok && mbar_wait(&s_full[buf], (uint32_t)((k >> 1) & 1));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const bool whole = (t0 >= lo && t0 + BN - 1 <= hi) || t0 + BN <= pre;
      const bool masked = !__all_sync(0xffffffffu, whole);
      const int m_a = lo - t0, m_b = hi - t0, m_c = pre - t0;
      auto unseen = [&](int i) { return !((i >= m_a && i <= m_b) || i < m_c); };
      // 64 raw scores x (columns c..) -> the log2 domain, unless `raw`
      auto transform = [&](uint32_t* x, int c) {
        if (capped) {
          bool big = false;
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            const float y = __uint_as_float(x[i]) * p.cap_in;
            big |= !(fabsf(y) < kTanhSeries);
            x[i] = __float_as_uint(y);
          }
          // the series where every score of the warp is small next to the cap, which
          // is the ordinary case and costs no MUFU operation
          if (__any_sync(0xffffffffu, big)) {
#pragma unroll
            for (int i = 0; i < 64; ++i) {
              const float y = __uint_as_float(x[i]);
              const float a = tanh_series(y), b = tanh_exp(y);
              x[i] = __float_as_uint(p.cap_log2 * (fabsf(y) < kTanhSeries ? a : b));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              x[i] = __float_as_uint(p.cap_log2 * tanh_series(__uint_as_float(x[i])));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            x[i] = __float_as_uint(__uint_as_float(x[i]) * p.scale_log2);
        }
        if (biased) {
          const float d0 = (float)(pos - t0 - c);
#pragma unroll
          for (int i = 0; i < 64; ++i)
            x[i] = __float_as_uint(fmaf(-slope, fabsf(d0 - (float)i), __uint_as_float(x[i])));
        }
      };
      // ---- first pass: the tile's maximum.  Scaling by a positive factor and the cap
      // keep the order, so then only the maximum itself is transformed.
      float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
      for (int c = 0; c < BN; c += 64) {
        uint32_t x[64];
        tmem_ld64(s_addr + c, x);
        if (!ordered) transform(x, c);
        if (masked) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (unseen(c + i)) x[i] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          mx0 = fmaxf(mx0, __uint_as_float(x[i]));
          mx1 = fmaxf(mx1, __uint_as_float(x[i + 1]));
          mx2 = fmaxf(mx2, __uint_as_float(x[i + 2]));
          mx3 = fmaxf(mx3, __uint_as_float(x[i + 3]));
        }
      }
      float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
      if (ordered && mx != -INFINITY) {
        if (capped) {
          const float y = mx * p.cap_in;
          mx = p.cap_log2 * (fabsf(y) < kTanhSeries ? tanh_series(y) : tanh_exp(y));
        } else {
          mx *= p.scale_log2;
        }
      }
      float alpha = 1.f;
      if (mx > m + kTileLazyMax) {
        alpha = fast_exp2(m - mx);
        m = mx;
        l *= alpha;
      }
      const float sub = m == -INFINITY ? 0.f : m;  // a row that has seen nothing: weights 0
      // ---- second pass: the weights, over the scores they come from (columns c / 2 ..
      // of the packed weights cover scores already read)
      float l0 = 0.f, l1 = 0.f;
#pragma unroll
      for (int c = 0; c < BN; c += 64) {
        uint32_t x[64], w[32];
        tmem_ld64(s_addr + c, x);
        if (!raw) transform(x, c);
        if (masked) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (unseen(c + i)) x[i] = 0xff800000u;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float a = fast_exp2(fmaf(__uint_as_float(x[2 * i]), factor, -sub));
          const float b = fast_exp2(fmaf(__uint_as_float(x[2 * i + 1]), factor, -sub));
          l0 += a;
          l1 += b;
          w[i] = pack_bf16x2(a, b);
        }
        tmem_st32(s_addr + c / 2, w);
      }
      l += l0 + l1;
      tmem_st_wait();
      // ---- O of the step before, rescaled where the maximum rose
      if (k >= kStep) {
        ok = ok && mbar_wait(&o_done[kGroups == 2 ? wg : 0], (uint32_t)(done & 1));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++done;
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(o_addr + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(o_addr + c, o);
          }
          tmem_st_wait();
        }
      }
      // ---- V rows of this tile that no row of the piece sees (the first step on a
      // tile zeroes them; the product of the other row tile comes after its own)
      if ((!both || wg == 0) && (t0 + BN - 1 > last_seen || (t0 < min_lo && t0 + BN > pre))) {
        const int item = item_v(j);
        ok = ok && mbar_wait(&full[item % kSlots], (uint32_t)((item / kSlots) & 1));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* v = sm_kv + (item % kSlots) * T::kSlotBytes;
        for (int c = r128; c < BN * kHalves * 8; c += 128) {
          const int row = (c >> 3) % BN, t = t0 + row;
          if (t > last_seen || (t < min_lo && t >= pre))
            *reinterpret_cast<uint4*>(v + (c >> 3) / BN * (BN * 128) + row * 128 +
                                      (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_shared();
      }
      tc_fence_before();
      mbar_arrive(&p_full[buf]);
    }
    // ---- the last product of this warpgroup
    const bool worked = wg < steps;
    if (ok && worked) ok = mbar_wait(&o_done[kGroups == 2 ? wg : 0], (uint32_t)(done & 1));
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) report(kTileStatusTimeout);
    tc_fence_after();
    // ---- one row tile: the second warpgroup hands its state over through the ring
    // (idle once both have seen their last product), [D][128] floats, then (m, l)
    const bool merge = kGroups == 2 && !both && steps > 1;
    float* sm_o = reinterpret_cast<float*>(sm_kv);
    float2* sm_ml = reinterpret_cast<float2*>(sm_kv + D * 128 * 4);
    float f_own = 1.f, f_other = 0.f;
    if (merge) {
      named_barrier(1, kGroups * 128);
      if (wg == 1) {
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_addr + c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) sm_o[(c + i) * 128 + r128] = __uint_as_float(o[i]);
        }
        sm_ml[r128] = make_float2(m, l);
      }
      named_barrier(1, kGroups * 128);
      if (wg == 0) {
        const float2 x = sm_ml[r128];
        const float top = fmaxf(m, x.x);
        f_own = m == -INFINITY ? 0.f : fast_exp2(m - top);
        f_other = x.x == -INFINITY ? 0.f : fast_exp2(x.x - top);
        l = l * f_own + (f_other > 0.f ? x.y * f_other : 0.f);
        m = top;
      }
    }
    if (both || wg == 0) {
      const float inv = p.single ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(o_addr + c, o);
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          y[i] = __uint_as_float(o[i]);
          if (merge)
            y[i] = y[i] * f_own + (f_other > 0.f ? sm_o[(c + i) * 128 + r128] * f_other : 0.f);
          y[i] *= inv;
        }
        if (valid) {
          if (p.single) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + q_row * D + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]),
                                  pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                                  pack_bf16x2(y[8 * i + 4], y[8 * i + 5]),
                                  pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
          } else {
            float4* dst =
                reinterpret_cast<float4*>(p.part_o + (split * part_rows + q_row) * D + c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        }
      }
      if (valid && !p.single) p.part_ml[split * part_rows + q_row] = make_float2(m, l);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTileTmemColumns);
  }
}

template <int D>
cudaError_t launch_tile(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                        cudaStream_t stream) {
  using T = TileShape<D>;
  static std::atomic<bool> limit_raised[64];
  auto kernel = paged_tile_kernel<D>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !limit_raised[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) limit_raised[dev].store(true, std::memory_order_release);
  }
  const long long tiles = (long long)p.total_q * p.G / T::kRows + p.num_seqs;
  const long long grid = tiles * p.H_kv * p.splits;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(T::kThreads);
  cfg.dynamicSmemBytes = T::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, tk, tv, p);
}

}  // namespace pagedattn
