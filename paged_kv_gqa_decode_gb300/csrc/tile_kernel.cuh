// Attention of many query rows over the paged KV cache on the 5th-generation
// tensor cores: chunks of a prompt, drafted tokens, and the members of a group
// that share a prefix (include/paged_attn.h).
//
// One piece of work is (sequence, KV head, tile of query rows, part of the
// token range).  The q_len * G rows of a KV head are token-major (row r is query
// r / G, head r % G), so a K/V tile read once serves the whole group and up to
// 256 rows.  Per 128 x BN tile of scores:
//
//   S = Q K^T   tcgen05.mma, Q and K in shared memory, S (fp32) in tensor memory
//   P = 2^(x - m), x the scaled, capped, biased, masked score in the log2 domain
//   O = O + P V tcgen05.mma, P (bf16) in tensor memory, V in shared memory
//
// Roles: a few warps copy pages (TMA, one box per page and 128-byte column half,
// K and V tiles through one ring), one lane of another issues the products, and a
// team of 256 threads turns a score tile into weights: two threads per row, each
// with half of the columns in registers, exchanging only the row's maximum (one
// thread per row with all 128 columns left two warps per SM sub-partition, too few to
// hide their own latencies: four capped prompt chunks 702 us, 636 with two).  Two
// teams (head_dim 64 and 128, long query runs) work on different score tiles while
// the products of the other run: on the two row tiles of a full piece, or, when a
// piece has at most 128 rows, on alternate token tiles of the same rows, merged at
// the end.  One team has two score buffers; head_dim 64 and 128 then have two CTAs
// on an SM, while the accumulators of 256 take half the tensor memory.
//
// What bounds it.  On four prompt chunks (1500 to 2048 tokens each before up to 8192,
// window 4096, 32 query and 8 KV heads of 128, 472 GFLOP) it takes 476 us with capped
// scores and 401 without, 992 and 1177 TFLOP/s (0.51 and 0.61 of the measured peak):
// a team's weights and its products follow each other, since its one score buffer
// holds both, and the other team's products fill half of that.  Capped scores that come
// near the cap (deviation 4 and more under a cap of 50) take 870 to 900 us, the slow form
// of cap_score below.  For 64 tokens of
// head_dim 128 the two products take 620 cycles back to back; what keeps them apart is
// latency, of the tensor-memory loads, of the barrier operations behind the other
// warps' arithmetic, and of the 4 cycles a warp's 32 exponentials take.
//
// The running maximum is raised only when a tile passes it by 2^8, so most tiles
// do not rescale O in tensor memory; the weights (at most 2^8) are rounded to bf16
// for the product, as relative accuracy is what counts there, and summed in fp32.
//
// Masks: a query at position pos sees [lo, hi] and the prefix [0, pre).  Token
// tiles outside the prefix and the hull of the rows' intervals are not walked, pages
// outside them not read; in the few tiles where an interval ends the scores are selected, and V rows that no
// row of the piece sees, which may hold anything, are zeroed in shared memory
// before the product.  Those are the rows outside the hull of the rows' intervals and, where
// a row sees nothing, its own token if no later row sees it.
#pragma once

#include <atomic>
#include <type_traits>

#include "tcgen05.cuh"
#include "tile.h"

namespace pagedattn {

constexpr int kTileStatusBadBlock = 1, kTileStatusBadLength = 2, kTileStatusTimeout = 4,
              kTileStatusConfig = 8;
constexpr float kTileLazyMax = 8.f;
// Batches up to this many sequences start with the longest ones (a loop over all of
// them in every CTA): verification of five tokens, 32 sequences of 512 to 4096 tokens,
// 67.5 -> 50.5 us, two head_dim 256 chunks 185 -> 127.
constexpr int kRankedSeqs = 128;

template <int D, int TEAMS>
struct TileShape {
  static constexpr int kTeams = TEAMS;                    // softmax teams of 256 threads
  static constexpr int kRows = 128 * TEAMS;
  // Tokens of one K/V tile, and the score buffers of a team.  With two buffers the
  // scores of its next tile are there when it has finished one; but tensor memory
  // then leaves two teams only 64 columns a buffer, and the products' own warp,
  // which takes some hundred cycles of latency a step among busy ones, sets the pace
  // (four capped prompt chunks: 704 us, against 548 with one buffer of 128).
  static constexpr int BN = TEAMS == 2 ? 128 : 64;
  static constexpr int kBufs = TEAMS == 2 ? 1 : 2;
  static constexpr int kCtas = TEAMS == 1 && D < 256 ? 2 : 1;  // CTAs on an SM
  static constexpr int kCols = BN / 2;                    // score columns of a thread
  static constexpr int kHalves = D / 64;                  // 128-byte column halves of a row
  static constexpr int kQTileBytes = 128 * D * 2;         // one 128-row query tile
  static constexpr int kSlotBytes = BN * D * 2;           // one K or V tile
  static constexpr int kSlots = D == 256 ? 5 : D == 64 ? 8 : 4;
  // The teams' warps, then the producers and the product warp.  A warp's tensor
  // copies are issued one after the other, about 54 cycles each and 214 for a group,
  // whatever their size (measured on 2, 4 and 8 KB boxes), and warps side by side:
  // one producer brings 2 KB boxes at 18 to 30 bytes a cycle, two at 35, four at 70.
  // Slot s of the ring belongs to producer s % kProducers, which so waits for its
  // phases strictly in order (a parity wait cannot tell phase k from k - 2).
  static constexpr int kProducers = D == 256 ? 5 : 2;
  static_assert(kSlots % kProducers == 0, "a slot belongs to one producer");
  static constexpr int kThreads = kTeams * 256 + 32 + kProducers * 32;
  // tensor memory: the teams' score buffers, then the accumulators
  static constexpr int kOCol = kTeams * kBufs * BN;
  static constexpr int kTmemColumns = kCtas == 2 ? 256 : 512;
  static_assert(kOCol + kTeams * D <= kTmemColumns, "tensor memory");
  // shared memory: query tiles, the K/V ring, barriers (384 bytes) and scalars, the
  // row maxima the two threads of a row exchange, [team][kBufs][half][row]
  static constexpr int kRingOff = kTeams * kQTileBytes;
  static constexpr int kBarOff = kRingOff + kSlots * kSlotBytes;
  static constexpr int kMaxOff = kBarOff + 512;
  static constexpr int kSmem = kMaxOff + kTeams * kBufs * 2 * 128 * 4;
  static_assert((kSmem + 1024) * kCtas <= 228 * 1024 && (2 * kSlots + 14 + kProducers) * 8 <= 384,
                "shared memory");
};

// What the scores need, compiled apart so that each loop over a row holds only its
// own arithmetic (one kernel with all three spent a third of its issue slots
// waiting for instructions).  Plain and capped need scale > 0.
enum { kTilePlain = 0, kTileCapped = 1, kTileGeneral = 2 };

// Bits n .. 31 (all for n <= 0, none for n >= 32).
__device__ __forceinline__ uint32_t bits_from(long long n) {
  return n <= 0 ? 0xffffffffu : n >= 32 ? 0u : 0xffffffffu << (int)n;
}

// cap tanh(s c) - m for raw scores s, c = scale / cap, as the weights' exponent:
// where |s c| < kTanhSeries for every score of the warp (2048 of them, or 1024: under a
// cap of 50 nearly all tiles of scores of deviation 1 or 2, hardly one of deviation 4)
// from a polynomial with the powers of c and the cap folded into its
// coefficients, s (a0 + s^2 (a1 + s^2 a2)): four operations a score with the
// subtraction, and no MUFU operation.  tanh(y) / y = 1 - z / 3 + 2 z^2 / 15 -
// 17 z^3 / 315 + ..., z = y^2; on [0, h], h = kTanhSeries^2, z^3 differs by h^3 / 32 at
// most from 3 h z^2 / 2 - 9 h^2 z / 16 + h^3 / 32 (Chebyshev economisation), so the
// cubic term becomes a change of the others, and the error is below 17 / 315 h^3 / 32
// = 4.2e-7 plus the quartic term's 3.4e-7 of the score.
struct CapSeries {
  float a0, a1, a2;
  float reach;  // |s| below which it holds (0: a coefficient overflowed; never used then)
};
__device__ __forceinline__ CapSeries cap_series(float c, float cap_log2) {
  constexpr float h = kTanhSeries * kTanhSeries, t3 = -17.f / 315.f;
  CapSeries t;
  const float f = cap_log2 * c, z = c * c;
  t.a0 = f * (1.f + t3 * h * h * h / 32.f);
  t.a1 = f * z * (-1.f / 3.f - t3 * 9.f / 16.f * h * h);
  t.a2 = f * z * z * (2.f / 15.f + t3 * 1.5f * h);
  t.reach = isfinite(t.a2) ? kTanhSeries / c : 0.f;  // (c > 0)
  return t;
}
// Any score: both forms and a selection, three MUFU operations a score in place of one
// with the weight's.  Four capped prompt chunks of scores of deviation 1 / 2 / 4 / 10 / 50,
// cap 50: 476 / 482 / 879 / 896 / 870 us.
__device__ __forceinline__ float cap_score(float s, float c, float cap_log2) {
  const float y = s * c;
  return cap_log2 * (fabsf(y) < kTanhSeries ? tanh_series(y) : tanh_exp(y));
}

template <int D, int TEAMS, int MOD>
__global__ void __launch_bounds__(TileShape<D, TEAMS>::kThreads, TileShape<D, TEAMS>::kCtas)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const TileParams p) {
  using T = TileShape<D, TEAMS>;
  constexpr int kTeams = T::kTeams, kRows = T::kRows, BN = T::BN, kHalves = T::kHalves;
  constexpr int kThreads = T::kThreads;
  extern __shared__ __align__(1024) uint8_t smem[];  // (no room for an alignment slack)
  uint8_t* sm_q = smem;
  uint8_t* sm_kv = smem + T::kRingOff;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::kBarOff);
  uint64_t* full = bars;                     // [kSlots] a tile has landed
  uint64_t* empty = bars + T::kSlots;        // [kSlots] its products are done
  uint64_t* s_full = bars + 2 * T::kSlots;   // [team][2] scores ready
  uint64_t* p_full = s_full + 4;             // [team][2] weights stored, O rescaled
  uint64_t* o_done = p_full + 4;             // [team][2] product with V done
  uint64_t* q_full = o_done + 4;
  uint64_t* drain = q_full + 1;
  uint64_t* landed = drain + 1;              // [kProducers] a copy's landing (with sm_i[7])
  int* sm_i = reinterpret_cast<int*>(smem + T::kBarOff + 384);
  // sm_i: [0] TMEM address, [1] sequence, [2] row tile, [3] min lo, [4] max hi,
  // [5] max lo, [6] min hi, [7] a row sees nothing: there may be tokens between min lo
  // and max hi that no row sees,
  // [8..32) warp sums of the tile search; then [8..16) a bit per query of the piece, set when
  // a row sees its token (used with [7] only)
  uint32_t* sm_tmem = reinterpret_cast<uint32_t*>(sm_i);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int N = p.num_seqs, G = p.G;
  auto report = [&](int bits) { atomicOr(p.status, bits); };

  if (smem_addr(smem) & 1023) {  // never expected: the swizzle needs 1024-byte tiles
    griddep_wait();
    if (tid == 0) report(kTileStatusConfig);
    return;
  }
  if (tid == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  griddep_wait();
  // (after the wait: a dependent launch that needs nothing of this one may then go on
  // without waiting itself, since the work before both is complete)
  griddep_launch_dependents();

  // ---- which piece: tiles are numbered through the sequences, those with the most
  // tokens to walk first where the batch is small enough to rank, and within one
  // from its last rows (causally the longest walk) to its first
  const int split = (int)(blockIdx.x % p.splits);
  const int g = (int)(blockIdx.x / p.splits % p.H_kv);
  const int want = (int)(blockIdx.x / ((unsigned)p.splits * p.H_kv));
  // rows of sequence s, and the first of them (clamped into [0, total_q])
  auto rows_at = [&](int s, int& first) -> int {
    first = min(max(__ldg(p.qo_indptr + s), 0), p.total_q);
    return max(min(__ldg(p.qo_indptr + s + 1), p.total_q) - first, 0);
  };
  auto tiles_of = [&](int s) -> int {
    int first;
    return (int)(((long long)rows_at(s, first) * G + kRows - 1) / kRows);
  };
  // row offsets that fall, or pass total_q, are reported (such rows are not written)
  auto check_rows = [&](int s) {
    if (p.num_blocks <= 0 || blockIdx.x != 0) return;
    const int a = __ldg(p.qo_indptr + s), b = __ldg(p.qo_indptr + s + 1);
    if (a < 0 || b < a || b > p.total_q) report(kTileStatusBadLength);
  };
  if (tid == 0) {
    sm_i[1] = -1;
    sm_i[3] = 0x7fffffff;
    sm_i[4] = -1;
    sm_i[5] = 0;
    sm_i[6] = 0x7fffffff;
    sm_i[7] = 0;
    for (int i = 0; i < T::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);  // a team's warps
      mbar_init(&o_done[i], 1);
    }
    mbar_init(q_full, kTeams * 8);
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (N <= kRankedSeqs) {
    int2* rank = reinterpret_cast<int2*>(smem);  // (tokens, tiles) of each sequence
    int tokens = 0, tiles = 0;
    if (tid < N) {
      // what the sequence's last row sees, which is near what each of its pieces walks
      int first;
      const int rows = rows_at(tid, first), L = __ldg(p.seq_lens + tid);
      check_rows(tid);
      int from = p.window > 0 ? L - p.window : 0;
      if (p.doc_starts != nullptr && rows > 0)
        from = max(from, __ldg(p.doc_starts + first + rows - 1));
      from = min(max(from, 0), max(L, 0));
      tokens = max(L, 0) - from;
      if (p.prefix_lens != nullptr) tokens += min(max(__ldg(p.prefix_lens + tid), 0), from);
      tiles = (int)(((long long)rows * G + kRows - 1) / kRows);
      rank[tid] = make_int2(tokens, tiles);
    }
    __syncthreads();
    if (tid < N) {
      int before = 0;
#pragma unroll 4
      for (int u = 0; u < N; ++u) {
        const int2 x = rank[u];
        if (x.x > tokens || (x.x == tokens && u < tid)) before += x.y;
      }
      if (want >= before && want < before + tiles) {
        sm_i[1] = tid;
        sm_i[2] = tiles - 1 - (want - before);
      }
    }
    __syncthreads();
  } else {
    const int per = (N + kThreads - 1) / kThreads;
    const int s0 = min(N, tid * per), s1 = min(N, s0 + per);
    int local = 0;
    for (int s = s0; s < s1; ++s) {
      local += tiles_of(s);
      check_rows(s);
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sm_i[8 + warp] = incl;
    __syncthreads();
    int before = incl - local;
    for (int w = 0; w < warp; ++w) before += sm_i[8 + w];
    if (want >= before && want < before + local) {
      int s = s0;
      for (;;) {
        const int n = tiles_of(s);
        if (want < before + n || s + 1 >= s1) break;
        before += n;
        ++s;
      }
      sm_i[1] = s;
      // (clamped: offsets that overlap without end may wrap the sums)
      sm_i[2] = min(max(tiles_of(s) - 1 - (want - before), 0), max(tiles_of(s) - 1, 0));
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
  const bool both = kTeams == 2 && n_rows > 128;  // a row tile per warpgroup

  // ---- this thread's row (softmax threads) and the tokens it sees
  // Row r of a tile belongs to the warps with warp % 4 = r / 32, whose part of the
  // tensor memory that is.
  constexpr int kTeamWarps = T::kTeams * 8, kMmaWarp = kTeamWarps + T::kProducers;
  const int team = warp >> 3;              // kTeams and up: the other roles
  const int half = (warp >> 2) & 1;        // which columns of the row
  const int r128 = (warp & 3) * 32 + lane;
  const int rr = row0 + (both ? team * 128 : 0) + r128;
  const bool softmax_thread = warp < kTeamWarps;
  const int qi = rr / G;
  const bool valid = softmax_thread && (long long)rr < (long long)q_len * G && rr < row0 + kRows;
  long long q_row = -1;                    // row of q / out viewed as rows of D
  int lo = 0, hi = 0x7fffffff, pos = 0, head = 0;
  if (valid) {  // (a row's two threads agree on everything but their columns)
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
    } else if (p.causal) {
      sm_i[7] = 1;
    }
    atomicMax(&sm_i[5], lo);
    atomicMin(&sm_i[6], hi);
  }
  // ---- the query rows, swizzled for the products (128-byte rows, 16-byte chunk c
  // of row r at c ^ (r % 8)); the threads of a row (four with one row tile for two
  // teams) share the work
  if (softmax_thread) {
    const int sharers = both ? 2 : 2 * kTeams, chunks = D / 8 / sharers;
    const int c0 = (both ? half : 2 * team + half) * chunks;
    uint8_t* tile = sm_q + (both ? team * T::kQTileBytes : 0);
#pragma unroll 4
    for (int c = c0; c < c0 + chunks; ++c) {
      const uint4 v = valid ? __ldg(reinterpret_cast<const uint4*>(p.q + q_row * D) + c)
                            : make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(tile + (c >> 3) * (128 * 128) + r128 * 128 +
                                (((c & 7) ^ (r128 & 7)) << 4)) = v;
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
  }
  if (tid < 8) sm_i[8 + tid] = 0;
  __syncthreads();
  const int min_lo = sm_i[3], max_hi = sm_i[4];
  // tiles beginning in [clean_lo, clean_hi] are seen whole by every row
  const int clean_lo = sm_i[5], clean_hi = sm_i[6] - (BN - 1);

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
  // First token of this part's tile j, from its last to its first: under a distance
  // bias the scores fall that way, so the maximum is found at once and O is not
  // rescaled at every tile.
  auto token_of = [&](int j) -> int {
    const int k = k1 - 1 - j;
    return (k < head_tiles ? k : k + skip) * BN;
  };
  const long long part_rows = (long long)p.total_q * p.H_q;
  if (n <= 0) {  // nothing to see here: a zero row, or an empty state
    if (valid && half == 0 && (both || team == 0)) {
      if (p.single) {
        uint4* o = reinterpret_cast<uint4*>(p.out + q_row * D);
        for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
      } else {
        p.part_ml[split * part_rows + q_row] = make_float2(-INFINITY, 0.f);
      }
    }
    return;
  }

  if (warp == kMmaWarp) tmem_alloc(sm_tmem, T::kTmemColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sm_tmem;

  // A team's step is one score tile: every token tile with two row tiles, else (two
  // teams on one row tile) every other one.
  const int stride = kTeams == 2 && !both ? 2 : 1;  // token tiles from step to step
  // Items of the ring, in the order the products first use them: the K tiles of
  // every team's first kBufs steps, then a V tile and the K tile `ahead` + 1 further on.
  const int ahead = T::kBufs * stride - 1;
  auto item_k = [&](int j) { return j + max(0, j - ahead); };
  auto item_v = [&](int j) { return j + min(n, j + 1 + ahead); };
  constexpr int slots = T::kSlots, kBufs = T::kBufs;
  auto buf_of = [&](int t, int i) -> int { return kBufs * t + (kBufs == 2 ? i & 1 : 0); };
  auto slot_off = [&](int slot) -> int { return T::kRingOff + slot * T::kSlotBytes; };

  if (warp >= kTeamWarps && warp < kMmaWarp) {
    // =================================================================== producer
    const uint64_t policy = l2_evict_first_policy();
    const int pages = BN / p.BS, boxes = pages * kHalves;  // at most 16 boxes: one per lane
    const int page = lane % pages, half_col = lane / pages;
    // This warp's items are first, first + kProducers, ...; the K or V tile of each:
    const int first = warp - kTeamWarps, lead = min(n, ahead + 1), mixed = 2 * (n - lead);
    auto tile_of = [&](int it, bool& is_v) -> int {
      const int u = it - lead;
      is_v = u >= 0 && (u >= mixed || !(u & 1));
      return u < 0 ? it : u >= mixed ? n - lead + (u - mixed) : is_v ? u >> 1 : ahead + 1 + (u >> 1);
    };
    auto block_of = [&](int it) -> int {  // this lane's page, -1: no row of it is seen
      if (it >= 2 * n || lane >= boxes) return -1;
      bool is_v;
      const int t0 = token_of(tile_of(it, is_v)) + page * p.BS;
      const bool seen = t0 < pre || (t0 <= max_hi && t0 + p.BS > min_lo);
      if (!seen) return -1;
      const int pb = __ldg(p.block_tables + (size_t)s * p.maxb + t0 / p.BS);
      if (p.num_blocks > 0 && (pb < 0 || (long long)pb >= p.num_blocks))
        report(kTileStatusBadBlock);  // the copy's bounds check reads it as zeros
      return pb;
    };
    // Tokens inside [min_lo, max_hi] that no row sees.  Rows that see up to themselves cover
    // what lies between the first and the last of them, so only tokens of rows which see
    // nothing can be such.  Their V rows are zeroed here, between a tile's landing
    // and its arrival at `full`: one copy at a time, but only in these rare pieces, and
    // nothing of it in the loops of the other warps (the same in the softmax loop: four
    // capped prompt chunks 478 -> 492 us).
    const bool between = sm_i[7] != 0;
    const int pos0 = len - q_len + row0 / G;  // the token of the piece's first query
    uint32_t land_phase = 0;
    if (between) {  // (every warp sets all the bits, and its own barrier up)
      if (lane == 0) {
        mbar_init(&landed[first], 1);
        fence_barrier_init();
        fence_proxy_async_shared();
      }
      const int last = (row0 + n_rows - 1) / G - row0 / G;
      for (int k = lane; k <= last; k += 32) {
        int from = p.window > 0 ? (int)max(0LL, (long long)pos0 + k - p.window + 1) : 0;
        if (p.doc_starts != nullptr)
          from = max(from, min(__ldg(p.doc_starts + qo + row0 / G + k), len));
        if (from > pos0 + k) continue;
        const int a = max(from - pos0, 0);
        for (int w = a >> 5; w <= k >> 5; ++w)
          atomicOr(&sm_i[8 + w], (int)(bits_from(a - 32 * w) & ~bits_from(k + 1 - 32 * w)));
      }
      __syncwarp();
    }
    auto zero_between = [&](uint8_t* v, int t0) {
      for (int row = 0; row < BN; ++row) {
        const int t = t0 + row, k = t - pos0;
        if (t < pre || t > max_hi || k < 0 || (sm_i[8 + (k >> 5)] >> (k & 31) & 1)) continue;
        if (lane < kHalves * 8)
          *reinterpret_cast<uint4*>(v + (lane >> 3) * (BN * 128) + row * 128 + (lane & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_shared();
    };
    bool ok = true;
    int slot = first, end = first;  // end: one stride past the last item copied
    uint32_t phase = 0;
    int pb = block_of(first);
    for (int it = first; it < 2 * n; it += T::kProducers) {
      const int pb_next = block_of(it + T::kProducers);
      bool is_v;
      const int tile = tile_of(it, is_v);
      ok = ok && tile_wait(&empty[slot], phase ^ 1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint64_t* bar = between ? &landed[first] : &full[slot];
      if (lane == 0) mbar_arrive_expect_tx(bar, T::kSlotBytes);
      __syncwarp();
      if (lane < boxes)  // a block id of -1 is out of the map's bounds: zeros
        tma_load_4d(smem + slot_off(slot) + half_col * (BN * 128) + page * p.BS * 128,
                    is_v ? &tm_v : &tm_k, bar, 0, g * p.BS, half_col, pb < 0 ? -1 : pb, policy);
      if (between) {
        ok = __all_sync(0xffffffffu, tile_wait(bar, land_phase));
        land_phase ^= 1u;
        if (!ok) break;
        if (is_v) zero_between(smem + slot_off(slot), token_of(tile));
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[slot]);
      }
      slot += T::kProducers;
      if (slot >= slots) {
        slot -= slots;
        phase ^= 1u;
      }
      pb = pb_next;
      end = it + T::kProducers;
    }
    if (!ok && lane == 0) report(kTileStatusTimeout);
    // no copy may be in flight when the CTA exits: this warp's last ones
    for (int it = end - T::kProducers; it >= first && it > end - T::kProducers - slots;
         it -= T::kProducers)
      if (!mbar_wait(&full[it % slots], (uint32_t)((it / slots) & 1)) && lane == 0)
        report(kTileStatusTimeout);
  } else if (warp == kMmaWarp) {
    // ==================================================================== products
    // The warp walks the steps together, with warp-uniform operands, and one lane
    // issues: the products take their operands from uniform registers.
    {
      // (a reduction's result is uniform to the compiler)
      const uint32_t lead = elect_one();
      const bool two = __reduce_max_sync(0xffffffffu, (uint32_t)both) != 0;  // two row tiles
      const int n_tiles = (int)__reduce_max_sync(0xffffffffu, (uint32_t)n);
      const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
      constexpr uint32_t kDescS = instr_desc(128, BN, false), kDescO = instr_desc(128, D, true);
      bool ok = mbar_wait(q_full, 0);
      const uint32_t q_desc = desc_lo(smem_addr(smem), 16);
      const uint32_t v_lead = ((uint32_t)(BN * 128 - 16) >> 4) << 16;  // K-major to MN-major lead
      // The next K tile's and the next V tile's place in the ring: both advance
      // through the items in order.
      int k_slot = 0, v_slot = 0, item = 0;
      uint32_t phase = 0;
      // A wait's round trip is long in this kernel (200 to 600 cycles: barrier
      // operations queue behind the exponentials of the other warps), so each is
      // looked at as soon as the one before it has been used, and waited for only
      // where that look came too early.
      bool seen = mbar_test_wait(&full[0], 0u);
      auto next_item = [&]() -> int {  // waits for the next item, returns its slot
        if (!seen && ok) ok = tile_wait(&full[item], phase);
        const int slot = item;
        if (++item == slots) {
          item = 0;
          phase ^= 1u;
        }
        seen = mbar_test_wait(&full[item], phase);
        return slot;
      };
      const int steps_of = two || kTeams == 1 ? 1 : 2;  // token tiles of one round
      // Step i of team t on token tile j.
      auto scores = [&](int t, int i, int j) {  // S[t][i & 1] = Q K_j^T
        if (!two || t == 0) k_slot = next_item();
        const uint32_t qd = q_desc + (two && t == 1 ? T::kQTileBytes >> 4 : 0);
        const uint32_t kd = q_desc + (slot_off(k_slot) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(lead, tm + buf_of(t, i) * BN,
                 qd + (((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4),
                 kd + (((kk >> 2) * (BN * 128) + (kk & 3) * 32) >> 4), kDescS, kk > 0);
        mma_commit(lead, &s_full[buf_of(t, i)]);
        if (!two || t == 1) mma_commit(lead, &empty[k_slot]);
      };
      auto values = [&](int t, int i, int j) {  // O[t] = O[t] + P[t][i & 1] V_j
        if (!two || t == 0) v_slot = next_item();
        // (after a timeout the walk goes on without waiting: what it then multiplies is
        // in bounds, and the call has reported)
        if (ok) ok = tile_wait(&p_full[buf_of(t, i)], (uint32_t)(i / kBufs) & 1u);
        tc_fence_after();
        const uint32_t vd = q_desc + v_lead + (slot_off(v_slot) >> 4);
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          mma_ts(lead, tm + T::kOCol + t * D, tm + buf_of(t, i) * BN + kk * 8,
                 vd + (kk * 2048 >> 4), kDescO, i > 0 || kk > 0);
        // (with one buffer only the last product's completion is waited for: a step's
        // scores are issued behind the product before)
        if (kBufs == 2 || j + steps_of >= n_tiles) mma_commit(lead, &o_done[buf_of(t, i)]);
        if (!two || t == 1) mma_commit(lead, &empty[v_slot]);
      };
      // kBufs steps of scores ahead, each buffer's next scores behind the product that
      // reads the weights over its last ones (products run in the order of issue).
      // Every item is waited for in the ring's order: with two row tiles the second
      // team's turn uses the tiles of the first's.
      for (int i = 0; i < kBufs; ++i)
        for (int t = 0; t < kTeams; ++t) {
          const int j = steps_of * i + (steps_of == 2 ? t : 0);
          if (j < n_tiles) scores(t, i, j);
        }
      for (int i = 0; steps_of * i < n_tiles; ++i) {
        for (int t = 0; t < kTeams; ++t) {
          const int j = steps_of * i + (steps_of == 2 ? t : 0);
          if (j >= n_tiles) break;
          values(t, i, j);
          if (j + kBufs * steps_of < n_tiles) scores(t, i + kBufs, j + kBufs * steps_of);
        }
      }
      mma_commit(lead, drain);
      if (!mbar_wait(drain, 0)) ok = false;
      if (!ok && lead) report(kTileStatusTimeout);
    }
    __syncwarp();
  } else {
    // ===================================================================== softmax
    // A thread's 32 or 64 columns.  With 64 registers are scarce (96 a thread): capped
    // scores, whose polynomial wants some, are read in two blocks, and the first one a
    // second time for its weights instead of being kept (four capped prompt chunks 507
    // -> 485 us; plain ones lose by it, 401 -> 427).
    constexpr int kCols = T::kCols, kBlocks = kCols / 32;
    constexpr bool kReload = kBlocks == 2 && MOD == kTileCapped;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_addr =
        tmem + lane_base + T::kOCol + (kTeams == 2 ? team * D : 0) + half * (D / 2);
    float* sm_max = reinterpret_cast<float*>(smem + T::kMaxOff) + team * kBufs * 256;
    const uint32_t pair_bar = 1 + team * 4 + (warp & 3);  // the two warps of 32 rows
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, tile_wait(bar, parity)) != 0;
    };
    float m = -INFINITY, l = 0.f;  // l: over this thread's columns
    bool ok = true;
    const float slope = MOD == kTileGeneral && valid && p.slopes != nullptr
                            ? __ldg(p.slopes + head) * 1.4426950408889634f
                            : 0.f;
    CapSeries cap = {};
    if constexpr (MOD == kTileCapped) cap = cap_series(p.cap_in, p.cap_log2);
    const int last_seen = max(max_hi, pre - 1);
    // A warp none of whose rows is the piece's only keeps step: what is then in its
    // rows of the weights reaches its rows of O alone, which nobody stores.
    const bool idle = !__any_sync(0xffffffffu, valid);
    const int my_steps = stride == 2 ? (n + 1 - team) / 2 : n;
    for (int i = 0; i < my_steps; ++i) {
      const int buf = buf_of(team, i), j = stride == 2 ? 2 * i + team : i, t0 = token_of(j);
      const int c0 = t0 + half * kCols;  // token of this thread's first column
      const uint32_t s_addr = tmem + lane_base + buf * BN;
      ok = ok && warp_wait(&s_full[buf], (uint32_t)(i / kBufs) & 1u);
      if (ok) tc_fence_after();
      if (!idle) {
      // ---- Unseen tokens: a bit per column, from the interval ends.
      bool ragged = false;
      uint32_t seen[kBlocks];
      auto find_seen = [&] {
        if (t0 >= clean_lo && t0 <= clean_hi) return;
        const bool whole = (c0 >= lo && c0 + kCols - 1 <= hi) || c0 + kCols <= pre;
        ragged = !__all_sync(0xffffffffu, whole);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
          seen[b] = (bits_from(lo - c0 - 32 * b) & ~bits_from(hi + 1LL - c0 - 32 * b)) |
                    ~bits_from(pre - c0 - 32 * b);
      };
      auto sees = [&](int b, int c) { return (seen[b] >> c & 1u) != 0; };
      // ---- this thread's scores (a timeout leaves what is there: the walk goes on
      // without waiting, so that the row's threads stay together)
      float x[kReload ? 1 : kBlocks][32];
      auto load = [&](int b) {
        tmem_ld_begin(s_addr + half * kCols + b * 32, x[kReload ? 0 : b]);
        tmem_ld_end(x[kReload ? 0 : b]);
      };
      if constexpr (kReload || kBlocks == 1) {
        if constexpr (!kReload) load(0);
      } else {
        tmem_ld_begin(s_addr + half * kCols, reinterpret_cast<float (&)[64]>(x));
        tmem_ld_end(reinterpret_cast<float (&)[64]>(x));
      }
      if constexpr (MOD == kTileGeneral) {
        // the whole transformation here, in place: with a bias the order of the raw
        // scores says nothing
        const float d0 = (float)(pos - c0), base = -slope * d0;
        // -slope |pos - t| is linear over the columns where no token lies past the
        // query, which is everywhere but on a causal diagonal and beyond
        const bool behind = __all_sync(0xffffffffu, pos >= c0 + kCols - 1 || slope == 0.f);
        auto each_pair = [&](auto&& f) {  // column pairs (c, c + 1)
#pragma unroll
          for (int c = 0; c < kCols; c += 2) {
            float* y = &x[c >> 5][c & 31];
            const float2 v = f(make_float2(y[0], y[1]), c);
            y[0] = v.x;
            y[1] = v.y;
          }
        };
        const float2 slope2 = make_float2(slope, slope), base2 = make_float2(base, base);
        auto bias = [&](int c) {
          return fma2(slope2, make_float2((float)c, (float)(c + 1)), base2);
        };
        if (p.cap_log2 > 0.f) {
          float mx0 = -INFINITY, mx1 = -INFINITY, mn0 = INFINITY, mn1 = INFINITY;
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            const float* y = &x[c >> 5][c & 31];
            mx0 = max3(mx0, y[0], y[1]);
            mx1 = max3(mx1, y[2], y[3]);
            mn0 = min3(mn0, y[0], y[1]);
            mn1 = min3(mn1, y[2], y[3]);
          }
          const CapSeries cap = cap_series(p.cap_in, p.cap_log2);
          if (__all_sync(0xffffffffu, fmaxf(fmaxf(mx0, mx1), -fminf(mn0, mn1)) < cap.reach)) {
            const float2 a0 = make_float2(cap.a0, cap.a0), a1 = make_float2(cap.a1, cap.a1);
            const float2 a2 = make_float2(cap.a2, cap.a2);
            each_pair([&](float2 y, int) {
              const float2 z = mul2(y, y);
              return mul2(y, fma2(z, fma2(z, a2, a1), a0));
            });
          } else {
            each_pair([&](float2 y, int) {
              return make_float2(cap_score(y.x, p.cap_in, p.cap_log2),
                                 cap_score(y.y, p.cap_in, p.cap_log2));
            });
          }
          if (behind) each_pair([&](float2 y, int c) { return add2(y, bias(c)); });
        } else {
          const float2 f = make_float2(p.scale_log2, p.scale_log2);
          if (behind)
            each_pair([&](float2 y, int c) { return fma2(y, f, bias(c)); });
          else
            each_pair([&](float2 y, int) { return mul2(y, f); });
        }
        if (!behind) {
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            x[c >> 5][c & 31] = fmaf(-slope, fabsf(d0 - (float)c), x[c >> 5][c & 31]);
        }
      }
      find_seen();
      // (capped scores are left alone, as the polynomial wants them finite: out of the
      // maximum here, and given no weight below)
      if (MOD != kTileCapped && ragged) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          if (!sees(c >> 5, c & 31)) x[c >> 5][c & 31] = -INFINITY;
      }
      // ---- running maximum, raised only past kTileLazyMax.  Scaling by a positive
      // factor and the cap keep the order: there only the maximum is transformed.
      float mx = -INFINITY, mn = INFINITY;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        if constexpr (kReload) load(b);
        const float (&y)[32] = x[kReload ? 0 : b];
        if (MOD == kTileCapped && ragged) {
#pragma unroll
          for (int c = 0; c < 32; ++c) mx = sees(b, c) ? fmaxf(mx, y[c]) : mx;
        } else {
          float mx0 = mx, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            mx0 = max3(mx0, y[c], y[c + 1]);
            mx1 = max3(mx1, y[c + 2], y[c + 3]);
            mx2 = max3(mx2, y[c + 4], y[c + 5]);
            mx3 = max3(mx3, y[c + 6], y[c + 7]);
          }
          mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
        }
        if constexpr (MOD == kTileCapped) {
          float mn1 = INFINITY;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            mn = min3(mn, y[c], y[c + 1]);
            mn1 = min3(mn1, y[c + 2], y[c + 3]);
          }
          mn = fminf(mn, mn1);
        }
      }
      const float own_max = mx;
      // the other half's; its thread has read its scores by then, so the packed
      // weights may overwrite them.  (With one score buffer a thread comes here again
      // only when all have finished this step; with two, the buffers of the exchange
      // take turns, and a thread writes one again only after its pair's barrier of
      // the step between.)
      float* exchange = sm_max + (buf - buf_of(team, 0)) * 256;
      exchange[half * 128 + r128] = mx;
      named_barrier(pair_bar, 64);
      mx = fmaxf(mx, exchange[(half ^ 1) * 128 + r128]);
      if constexpr (MOD == kTilePlain) mx *= p.scale_log2;  // (-inf stays: the factor is positive)
      if constexpr (MOD == kTileCapped)
        mx = mx == -INFINITY ? mx : cap_score(mx, p.cap_in, p.cap_log2);
      float alpha = 1.f;
      if (mx > m + kTileLazyMax) {
        alpha = fast_exp2(m - mx);
        m = mx;
        l *= alpha;
      }
      const float sub = m == -INFINITY ? 0.f : m;  // a row that has seen nothing: weights 0
      // ---- weights 2^(x - m), packed
      float2 sum = make_float2(0.f, 0.f);
      const float2 sub2 = make_float2(-sub, -sub);
      auto weigh = [&](auto masked, auto&& exponent) {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
          const int b = kReload ? kBlocks - 1 - k : k;
          const float (&y)[32] = x[kReload ? 0 : b];
          uint32_t w[16];
#pragma unroll
          for (int e2 = 0; e2 < 16; ++e2) {
            float2 e = exponent(make_float2(y[2 * e2], y[2 * e2 + 1]));
            if constexpr (decltype(masked)::value) {
              if (!sees(b, 2 * e2)) e.x = -INFINITY;
              if (!sees(b, 2 * e2 + 1)) e.y = -INFINITY;
            }
            e.x = fast_exp2(e.x);
            e.y = fast_exp2(e.y);
            sum = add2(sum, e);
            w[e2] = pack_bf16x2(e.x, e.y);
          }
          // (the first block's scores again, before the weights over them: those of the
          // second take the place of its last 16)
          if constexpr (kReload)
            if (b > 0) load(b - 1);
          tmem_st(s_addr + half * (kCols / 2) + b * 16, w);
        }
      };
      if constexpr (MOD == kTileCapped) {
        // (of a ragged tile own_max leaves the unseen scores out: what the polynomial
        // makes of them is not used.  A NaN is carried neither here nor there; the
        // polynomial keeps it.)
        if (__all_sync(0xffffffffu, fmaxf(own_max, -mn) < cap.reach)) {
          const float2 a0 = make_float2(cap.a0, cap.a0), a1 = make_float2(cap.a1, cap.a1);
          const float2 a2 = make_float2(cap.a2, cap.a2);
          auto series = [&](float2 s) {
            const float2 z = mul2(s, s);
            return fma2(s, fma2(z, fma2(z, a2, a1), a0), sub2);
          };
          // (two loops: as a condition inside one the selection costs every tile)
          if (ragged)
            weigh(std::true_type(), series);
          else
            weigh(std::false_type(), series);
        } else {
          if (!ragged) {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) seen[b] = 0xffffffffu;
          }
          weigh(std::true_type(), [&](float2 s) {
            return make_float2(cap_score(s.x, p.cap_in, p.cap_log2) - sub,
                               cap_score(s.y, p.cap_in, p.cap_log2) - sub);
          });
        }
      } else {
        const float f = MOD == kTilePlain ? p.scale_log2 : 1.f;
        weigh(std::false_type(), [&](float2 s) { return fma2(s, make_float2(f, f), sub2); });
      }
      l += sum.x + sum.y;
      tmem_st_wait();
      // ---- O, rescaled where the maximum rose, once the step before is in it (each
      // thread its half of the columns)
      if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        if constexpr (kBufs == 2)
          ok = ok && warp_wait(&o_done[buf_of(team, i - 1)], (uint32_t)((i - 1) >> 1) & 1u);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
          float o[32];
          tmem_ld_begin(o_addr + c, o);
          tmem_ld_end(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= alpha;
          tmem_st(o_addr + c, o);
        }
        tmem_st_wait();
      }
      }
      // ---- V rows of this tile that no row of the piece sees (the first step on a
      // tile zeroes them; the product of the other row tile comes after its own)
      if ((t0 < clean_lo || t0 > clean_hi) && (!both || team == 0) &&
          (t0 + BN - 1 > last_seen || (t0 < min_lo && t0 + BN > pre))) {
        const int item = item_v(j);
        ok = ok && warp_wait(&full[item % slots], (uint32_t)((item / slots) & 1));
        uint8_t* v = smem + slot_off(item % slots);
        for (int c = half * 128 + r128; ok && c < BN * kHalves * 8; c += 256) {
          const int row = (c >> 3) % BN, t = t0 + row;
          if (t > last_seen || (t < min_lo && t >= pre))
            *reinterpret_cast<uint4*>(v + (c >> 3) / BN * (BN * 128) + row * 128 +
                                      (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_shared();
      }
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&p_full[buf]);
    }
    // ---- the last product of this team (the one before it has completed: the last
    // scores were issued behind it)
    if (my_steps > 0) {
      const int last = my_steps - 1;
      ok = ok && warp_wait(&o_done[buf_of(team, last)],
                           kBufs == 2 ? (uint32_t)(last >> 1) & 1u : 0u);
    }
    if (!ok && lane == 0) report(kTileStatusTimeout);
    tc_fence_after();
    // ---- the row's sum from its two threads
    {
      float* exchange = sm_max;
      named_barrier(pair_bar, 64);  // every read of the maxima is done
      exchange[half * 128 + r128] = l;
      named_barrier(pair_bar, 64);
      l = half == 0 ? l + exchange[128 + r128] : exchange[r128] + l;
    }
    // a NaN score counts in the sum, not in the maximum: the maximum takes it over, so that
    // the state is not taken for an empty one
    if (l != l) m = l;
    // ---- one row tile: the second team hands its state over through the ring (idle
    // once both have seen their last product), [D][128] floats, then (m, l)
    const bool merge = stride == 2 && n > 1;
    float* sm_o = reinterpret_cast<float*>(sm_kv) + half * (D / 2) * 128;
    float2* sm_ml = reinterpret_cast<float2*>(sm_kv + D * 128 * 4);
    float f_own = 1.f, f_other = 0.f;
    if (merge) {
      named_barrier(9, kTeams * 256);
      if (team == 1) {
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
          float o[32];
          tmem_ld_begin(o_addr + c, o);
          tmem_ld_end(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) sm_o[(c + i) * 128 + r128] = o[i];
        }
        if (half == 0) sm_ml[r128] = make_float2(m, l);
      }
      named_barrier(9, kTeams * 256);
      if (team == 0) {
        const float2 y = sm_ml[r128];
        const float top = fmaxf(m, y.x);
        f_own = m == -INFINITY ? 0.f : fast_exp2(m - top);
        f_other = y.x == -INFINITY ? 0.f : fast_exp2(y.x - top);
        l = l * f_own + (f_other != 0.f ? y.y * f_other : 0.f);
        m = l != l ? l : top;
      }
    }
    if (both || team == 0) {
      const float inv = p.single ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        float o[32];
        tmem_ld_begin(o_addr + c, o);
        tmem_ld_end(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (merge)
            o[i] = o[i] * f_own + (f_other != 0.f ? sm_o[(c + i) * 128 + r128] * f_other : 0.f);
          o[i] *= inv;
        }
        if (valid) {
          const int col = half * (D / 2) + c;
          if (p.single) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + q_row * D + col);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]),
                                  pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                                  pack_bf16x2(o[8 * i + 4], o[8 * i + 5]),
                                  pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
          } else {
            float4* dst =
                reinterpret_cast<float4*>(p.part_o + (split * part_rows + q_row) * D + col);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
      }
      if (valid && half == 0 && !p.single)
        p.part_ml[split * part_rows + q_row] = make_float2(m, l);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, T::kTmemColumns);
  }
}

template <int D, int TEAMS, int MOD>
cudaError_t launch_tile_as(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                           cudaStream_t stream) {
  using T = TileShape<D, TEAMS>;
  static std::atomic<bool> limit_raised[64];
  auto kernel = paged_tile_kernel<D, TEAMS, MOD>;
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

template <int D, int TEAMS>
cudaError_t launch_tile(const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                        cudaStream_t stream) {
  if (p.slopes != nullptr || !(p.scale_log2 > 0.f))
    return launch_tile_as<D, TEAMS, kTileGeneral>(tk, tv, p, stream);
  return p.cap_log2 > 0.f ? launch_tile_as<D, TEAMS, kTileCapped>(tk, tv, p, stream)
                          : launch_tile_as<D, TEAMS, kTilePlain>(tk, tv, p, stream);
}

}  // namespace pagedattn
