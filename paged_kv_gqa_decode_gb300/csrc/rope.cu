// Norms of query and key heads, their rotation by position, and the append of the K and
// V rows by slot (include/paged_attn.h, paged_kv_rope_append_slots), in one pass:
//
//     y = x / sqrt(mean_d(x_d^2) + eps) * w             (no norm: y = x)
//     (a, b) -> (a c - b s, b c + a s)                  for the R / 2 rotated pairs
//
// pair i being elements (i, i + R / 2), or (2i, 2i + 1), and (c, s) = cos_sin[p, i] at
// the row's position p on the pair's axis.  Everything is float32 from the load to the
// one rounding at the store; an FP8 cache row is quantized from those float32 values, so
// K is rounded once there too.
//
// What bounds it: memory.  A lane holds 16 elements of a head, two chunks of 16 bytes that
// are each other's partners in the rotation, so that it needs no exchange, and D / 16
// lanes (a group) a head.  The coefficients of a row are made once for several heads: with
// the norm's weights folded in, z = r (x[a] (w[a] c) - x[b] (w[b] s)), r the root's reciprocal.
//
// Two kernels.  With few bf16 rows (a decode step) a group reads kHeads heads of one row
// straight into its registers.  With many, registers are what limits the bytes in flight
// (8192 rows of 32 + 2 x 8 heads of 128: 50 us however the heads and CTAs were set), so
// there each warp streams units of 4 KB through a ring of its own in shared memory by bulk
// copies that it issues itself, and no warp waits for another.
#include <atomic>
#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "rope.h"
#include "tcgen05.cuh"

namespace pagedattn {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // heads of one row that a group of lanes takes (few rows)
// bf16 rows are many from this many input bytes an SM on, if units hold half of their 4 KB on
// average (32 + 2 x 8 heads of 128, few / many: 512 rows 4.2 / 4.3 us, 1024 6.7 / 5.9, 8192 40.6 /
// 37.4; but 4 + 2 x 2 heads of 64, whose units are short, 8192 8.0 / 15.4).  FP8 rows always
// are: the quantization in four heads' copies is too long a code for a short kernel (8 + 2 x 2
// heads of 128, few / many: 64 rows 4.9 / 3.5, 1024 5.1 / 5.5, 8192 23.2 / 22.6; 24 + 2 x 4 of
// 256, 64 rows 5.5 / 4.0, 8192 77 / 47).
constexpr long long kManyBytes = 64 << 10;
constexpr float kE4m3Max = 448.f;
constexpr int kBadSlot = 1, kBadPosition = 2, kTimeout = 4;

// Two chunks of eight bf16 as pairs of float32.
__device__ __forceinline__ void unpack(const uint4& u, float2 (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack(const float2 (&x)[4]) {
  return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                    pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
}
__device__ __forceinline__ uint2 to_e4m3(const float2 (&x)[4], float f) {
  uint32_t b[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    b[i >> 2] |= (uint32_t)__nv_cvt_float_to_fp8((i & 1 ? x[i >> 1].y : x[i >> 1].x) / f,
                                                 __NV_SATFINITE, __NV_E4M3)
                 << (8 * (i & 3));
  return make_uint2(b[0], b[1]);
}
template <int N>
__device__ __forceinline__ void load_floats(const float* src, float* x) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4*>(x + i) = __ldg(reinterpret_cast<const float4*>(src + i));
}

// The row's cosines and sines, times the norm's weights: z0 = r (x0 a0 + x1 b0), z1 = r (x1
// a1 + x0 b1) with x0, x1 the first and second elements of a lane's eight pairs.
struct Coefficients {
  float2 a0[4], a1[4], b0[4], b1[4];
};

// What a lane holds: chunks c0 and c1 of a head hold the first and second elements of the
// same eight pairs, or (INTER, and what does not turn) are neighbours.
template <bool INTER>
struct Place {
  int l, c0, c1;
  bool turns;
  __device__ __forceinline__ Place(int lane, int R) {
    l = lane;
    turns = l < (R >> 4);
    c0 = turns && !INTER ? l : 2 * l;
    c1 = turns && !INTER ? l + (R >> 4) : 2 * l + 1;
  }
};

// The axes of a lane's eight pairs, the same for every row: nearly always one, or two where a
// section ends in between; `many` where they change oftener.
struct Axes {
  int lo, hi;       // of the first and the last pair
  uint32_t use_hi;  // bit i: pair i is on the last one's
  bool two, many;
};
__device__ __forceinline__ int axis_of(const RopeParams& p, int i) {
  return min(max(__ldg(p.freq_axis + i), 0), p.axes - 1);
}
template <bool INTER>
__device__ __forceinline__ Axes axes_of(const RopeParams& p, const Place<INTER>& at) {
  Axes x = {0, 0, 0u, false, false};
  if (p.freq_axis == nullptr || !at.turns) return x;
  x.lo = axis_of(p, 8 * at.l);
  x.hi = axis_of(p, 8 * at.l + 7);
  x.two = x.lo != x.hi;
  for (int i = 0; i < 8; ++i) {
    const int a = axis_of(p, 8 * at.l + i);
    if (a == x.hi) x.use_hi |= 1u << i;
    if (a != x.lo && a != x.hi) x.many = true;
  }
  return x;
}
// Positions of a row on a lane's two axes, as places in the table.
struct Positions {
  int lo, hi;
};
__device__ __forceinline__ int position(const RopeParams& p, int axis, long long row) {
  return __ldg(p.positions + (long long)axis * p.rows + row);
}
template <bool INTER>
__device__ __forceinline__ Positions positions_of(const RopeParams& p, const Place<INTER>& at,
                                                  const Axes& x, long long row, bool rotate) {
  Positions y = {0, 0};
  if (!rotate || !at.turns) return y;
  y.lo = position(p, x.lo, row);
  y.hi = x.two ? position(p, x.hi, row) : y.lo;
  return y;
}
__device__ __forceinline__ const float* table_row(const RopeParams& p, int pos, bool some) {
  if ((pos < 0 || pos >= p.max_positions) && p.status != nullptr && some)
    atomicOr(p.status, kBadPosition);
  return p.cos_sin + (long long)min(max(pos, 0), p.max_positions - 1) * p.R;
}

template <bool INTER>
__device__ __forceinline__ Coefficients coefficients(const RopeParams& p, const Place<INTER>& at,
                                                     const Axes& x, const Positions& pos,
                                                     long long row, const float* norm, bool rotate,
                                                     bool some) {
  Coefficients k;
  const int half = p.R >> 1, i0 = 8 * at.l;  // (i0: the first of its eight pairs)
  float c[8], s[8], w[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[0][i] = w[1][i] = 1.f;
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (rotate) {
    const float* from = table_row(p, pos.lo, some) + i0;
    load_floats<8>(from, c);
    load_floats<8>(from + half, s);
    if (x.two) {
      float c2[8], s2[8];
      from = table_row(p, pos.hi, some) + i0;
      load_floats<8>(from, c2);
      load_floats<8>(from + half, s2);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (x.use_hi >> i & 1u) {
          c[i] = c2[i];
          s[i] = s2[i];
        }
    }
    if (x.many) {
#pragma unroll 1
      for (int i = 1; i < 7; ++i) {
        const int a = axis_of(p, i0 + i);
        if (a == x.lo || a == x.hi) continue;
        from = table_row(p, position(p, a, row), some) + i0 + i;
        const float ci = __ldg(from), si = __ldg(from + half);
#pragma unroll
        for (int j = 1; j < 7; ++j)
          if (j == i) {
            c[j] = ci;
            s[j] = si;
          }
      }
    }
  }
  if (norm != nullptr) {
    load_floats<8>(norm + 8 * at.c0, w[0]);
    load_floats<8>(norm + 8 * at.c1, w[1]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // the weights of the pair's elements: (w[0][i], w[1][i]), or of neighbours
    const float wa = INTER ? w[i >> 2][2 * (i & 3)] : w[0][i];
    const float wb = INTER ? w[i >> 2][2 * (i & 3) + 1] : w[1][i];
    (i & 1 ? k.a0[i >> 1].y : k.a0[i >> 1].x) = wa * c[i];
    (i & 1 ? k.b0[i >> 1].y : k.b0[i >> 1].x) = -(wb * s[i]);
    (i & 1 ? k.a1[i >> 1].y : k.a1[i >> 1].x) = wb * c[i];
    (i & 1 ? k.b1[i >> 1].y : k.b1[i >> 1].x) = wa * s[i];
  }
  return k;
}

// Swaps the second of a pair of float2 with the first of the other: pairs (a, b) side by side to
// first and second elements apart, and back.
__device__ __forceinline__ void transpose2(float2& u, float2& v) {
  const float t = u.y;
  u.y = v.x;
  v.x = t;
}

// Norm and rotation of one head, and its store.  kind: 0 q, 1 k, 2 v; at_row: cache row of
// the first KV head, -1 for none.  The whole warp walks along (`write`: this group's head is one).
template <int D, bool FP8, bool INTER>
__device__ __forceinline__ void head(const RopeParams& p, const Place<INTER>& at,
                                     const Coefficients& k, uint4 raw0, uint4 raw1, bool normed,
                                     bool rotate, int kind, long long row, int h,
                                     long long at_row, bool write) {
  constexpr int kLanes = D / 16;
  float2 x[2][4], z[2][4];
  unpack(raw0, x[0]);
  unpack(raw1, x[1]);
  float r = 1.f;
  const bool any_norm = __any_sync(0xffffffffu, normed);
  if (any_norm) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = fma2(x[0][i], x[0][i], fma2(x[1][i], x[1][i], sum));
    float all = sum.x + sum.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (normed) r = rsqrtf(all * (1.f / D) + p.eps);
  }
  // (INTER: after the exchange x[c][i] and x[c][i + 1] hold the first and second elements of
  // pairs 4 c + i, 4 c + i + 1, whose coefficients are at 2 c + i / 2)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 &u = INTER ? x[i >> 1][2 * (i & 1)] : x[0][i], &v = INTER ? x[i >> 1][2 * (i & 1) + 1] : x[1][i];
    if constexpr (INTER) transpose2(u, v);
    float2 &y = INTER ? z[i >> 1][2 * (i & 1)] : z[0][i], &t = INTER ? z[i >> 1][2 * (i & 1) + 1] : z[1][i];
    y = mul2(u, k.a0[i]);
    t = mul2(v, k.a1[i]);
    if (rotate) {  // (not multiplied by a sine of zero: an infinity stays one)
      y = fma2(v, k.b0[i], y);
      t = fma2(u, k.b1[i], t);
    }
    if (any_norm) {
      y = mul2(y, make_float2(r, r));
      t = mul2(t, make_float2(r, r));
    }
    if constexpr (INTER) transpose2(y, t);
  }
  if (kind == 0) {
    if (write) {
      uint4* to = reinterpret_cast<uint4*>(p.q_out + (row * p.H_q + h) * D);
      to[at.c0] = pack(z[0]);
      to[at.c1] = pack(z[1]);
    }
  }
  if constexpr (!FP8) {
    if (kind != 0 && write && at_row >= 0) {
      __nv_bfloat16* cache = static_cast<__nv_bfloat16*>(kind == 1 ? p.k_cache : p.v_cache);
      uint4* to = reinterpret_cast<uint4*>(cache + (at_row + (long long)h * p.BS) * D);
      to[at.c0] = kind == 1 ? pack(z[0]) : raw0;
      to[at.c1] = kind == 1 ? pack(z[1]) : raw1;
    }
  } else if (kind != 0) {  // (the whole warp's: FP8 caches are written by the kernel for many rows)
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top = fmaxf(top, fmaxf(fabsf(z[0][i].x), fabsf(z[0][i].y)));
      top = fmaxf(top, fmaxf(fabsf(z[1][i].x), fabsf(z[1][i].y)));
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (write && at_row >= 0) {
      const float f = top > 0.f ? top / kE4m3Max : 1.f;
      const long long to = at_row + (long long)h * p.BS;
      uint2* dst = reinterpret_cast<uint2*>(
          static_cast<uint8_t*>(kind == 1 ? p.k_cache : p.v_cache) + to * D);
      dst[at.c0] = to_e4m3(z[0], f);
      dst[at.c1] = to_e4m3(z[1], f);
      if (at.l == 0) (kind == 1 ? p.k_scale : p.v_scale)[to] = f;
    }
  }
}

// Heads h0 .. of one tensor of a row: `heads` of them at most in an item.
struct Item {
  long long row;
  int kind, h0, heads;  // q, k, v; the first head and how many
};
__device__ __forceinline__ Item item_of(const RopeParams& p, long long item, int each) {
  const int q_parts = (p.H_q + each - 1) / each, kv_parts = (p.H_kv + each - 1) / each;
  const int parts = q_parts + 2 * kv_parts;
  Item x;
  // (32-bit division where it fits: the 64-bit one is a long sequence)
  x.row = item <= 0xffffffffLL ? (long long)((uint32_t)item / (uint32_t)parts) : item / parts;
  int part = (int)(item - x.row * parts);
  x.kind = part < q_parts ? 0 : part < q_parts + kv_parts ? 1 : 2;
  part -= x.kind == 0 ? 0 : x.kind == 1 ? q_parts : q_parts + kv_parts;
  x.h0 = part * each;
  x.heads = min(each, (x.kind == 0 ? p.H_q : p.H_kv) - x.h0);
  return x;
}
__device__ __forceinline__ const __nv_bfloat16* source(const RopeParams& p, const Item& x) {
  return (x.kind == 0   ? p.q + x.row * p.q_stride
          : x.kind == 1 ? p.k + x.row * p.k_stride
                        : p.v + x.row * p.v_stride) +
         (long long)x.h0 * p.D;
}
__device__ __forceinline__ long long cache_row(const RopeParams& p, const Item& x, bool some) {
  if (x.kind == 0) return -1;
  const long long slots = p.num_blocks * p.BS;
  const long long slot = __ldg(reinterpret_cast<const long long*>(p.slot_map) + x.row);
  if (slot >= slots && p.status != nullptr && some) atomicOr(p.status, kBadSlot);
  if (slot < 0 || slot >= slots) return -1;
  return (slot >> (p.BS == 32 ? 5 : 4)) * p.H_kv * p.BS + (slot & (p.BS - 1));
}
__device__ __forceinline__ const float* norm_of(const RopeParams& p, int kind) {
  return kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : nullptr;
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) paged_kv_rope_few_kernel(const RopeParams p) {
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes;
  griddep_wait();
  griddep_launch_dependents();  // (after the wait: what is ahead of this launch is complete)
  const int lane = threadIdx.x & 31, group = lane / kLanes;
  const Place<INTER> at(lane % kLanes, p.R);
  const Axes axes = axes_of(p, at);
  const long long items =
      (long long)p.rows * ((p.H_q + kHeads - 1) / kHeads + 2 * ((p.H_kv + kHeads - 1) / kHeads));
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  for (long long first = ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kGroups;
       first < items; first += warps * kGroups) {
    // (a group without an item walks along: the shuffles are the whole warp's)
    const bool some = first + group < items;
    const Item x = item_of(p, some ? first + group : first, kHeads);
    const uint4* src = reinterpret_cast<const uint4*>(source(p, x));
    uint4 raw[kHeads][2];
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {  // (plain loads: q_out may be q)
      raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
      if (u < x.heads) {
        raw[u][0] = src[u * (D / 8) + at.c0];
        raw[u][1] = src[u * (D / 8) + at.c1];
      }
    }
    const long long at_row = cache_row(p, x, some);
    const float* norm = norm_of(p, x.kind);
    const bool rotate = at.turns && x.kind != 2;
    const Positions pos = positions_of(p, at, axes, x.row, rotate);
    const Coefficients k = coefficients(p, at, axes, pos, x.row, norm, rotate, some);
#pragma unroll
    for (int u = 0; u < kHeads; ++u)
      head<D, false, INTER>(p, at, k, raw[u][0], raw[u][1], norm != nullptr, rotate, x.kind, x.row,
                          x.h0 + u, at_row, some && u < x.heads);
  }
}

// Many rows.  A warp takes a run of consecutive units and keeps kStages of them in flight: its
// lane 0 issues the copy of a unit as soon as the warp has read the one in that place.
// 8192 rows of 32 + 2 x 8 heads of 128, three axes: 38.5 us, 5.3 TB/s (16 warps with 3 stages
// 39.3, 12 warps with 4 stages of 4 KB 47, 8 with 3 of 8 KB 57: warps count for more than
// bytes in flight, and what is left of the L1 holds the table rows).
constexpr int kStreamWarps = 16, kStages = 2, kUnitBytes = 4096;
constexpr size_t kStreamSmem = (size_t)kStreamWarps * kStages * (kUnitBytes + 8);

template <int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(kStreamWarps * 32, 1)
    paged_kv_rope_many_kernel(const RopeParams p) {
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes, kUnitHeads = kUnitBytes / (2 * D);
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane / kLanes;
  uint8_t* ring = smem + warp * kStages * kUnitBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStreamWarps * kStages * kUnitBytes) +
                   warp * kStages;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();  // (after the wait: what is ahead of this launch is complete)
  const Place<INTER> at(lane % kLanes, p.R);
  const Axes axes = axes_of(p, at);
  const long long units = (long long)p.rows * ((p.H_q + kUnitHeads - 1) / kUnitHeads +
                                               2 * ((p.H_kv + kUnitHeads - 1) / kUnitHeads));
  const long long warps = (long long)gridDim.x * kStreamWarps;
  const long long me = (long long)blockIdx.x * kStreamWarps + warp;
  const long long first = units * me / warps, last = units * (me + 1) / warps;
  // the unit behind x (no division: one for the first unit of a warp)
  auto behind = [&](Item x) -> Item {
    x.h0 += kUnitHeads;
    if (x.h0 >= (x.kind == 0 ? p.H_q : p.H_kv)) {
      x.h0 = 0;
      if (++x.kind == 3) {
        x.kind = 0;
        ++x.row;
      }
    }
    x.heads = min(kUnitHeads, (x.kind == 0 ? p.H_q : p.H_kv) - x.h0);
    return x;
  };
  auto issue = [&](const Item& x, int stage) {
    if (lane == 0) {
      const uint32_t bytes = (uint32_t)x.heads * D * 2;
      mbar_arrive_expect_tx(&full[stage], bytes);
#ifdef PAGED_ATTN_WAIT_TEST
      if (x.kind == 0 && x.row == p.test_skip_row) return;  // (armed and never filled)
#endif
      bulk_load(ring + stage * kUnitBytes, source(p, x), bytes, &full[stage]);
    }
  };
  const int n = (int)(last - first);  // (units of a warp: far fewer than 2^31)
  if (n <= 0) return;
  Item x = item_of(p, first, kUnitHeads), ahead = x;
  for (int i = 0; i < kStages; ++i) {
    if (i < n) issue(ahead, i);
    ahead = behind(ahead);
  }
  int stage = 0;
  uint32_t phase = 0;
  // (a row's positions are read while the unit before is worked on; the coefficients stay
  // while row and tensor do)
  Positions pos = positions_of(p, at, axes, x.row, true);
  Coefficients k;
  bool fresh = true;
  for (int i = 0; i < n; ++i) {
    const long long at_row = cache_row(p, x, true);
    const float* norm = norm_of(p, x.kind);
    const bool rotate = at.turns && x.kind != 2;
    if (fresh) k = coefficients(p, at, axes, pos, x.row, norm, rotate, true);
    const Item next = behind(x);
    if (next.row != x.row && i + 1 < n) pos = positions_of(p, at, axes, next.row, true);
    if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase))) {
      // never expected: no copy may be in flight when the CTA exits, the one that is late included
      for (int j = 0; j < kStages && i + j < n; ++j)
        mbar_wait(&full[(stage + j) % kStages], stage + j >= kStages ? phase ^ 1u : phase);
      if (p.status != nullptr && lane == 0) atomicOr(p.status, kTimeout);
      return;
    }
    const uint4* tile = reinterpret_cast<const uint4*>(ring + stage * kUnitBytes);
    if (FP8 || x.kind != 2) {
      for (int u0 = 0; u0 < x.heads; u0 += kGroups) {
        const int u = u0 + group;
        const bool write = u < x.heads;
        uint4 raw0 = make_uint4(0u, 0u, 0u, 0u), raw1 = raw0;
        if (write) {
          raw0 = tile[u * (D / 8) + at.c0];
          raw1 = tile[u * (D / 8) + at.c1];
        }
        head<D, FP8, INTER>(p, at, k, raw0, raw1, norm != nullptr, rotate, x.kind, x.row, x.h0 + u,
                            at_row, write);
      }
    } else if (at_row >= 0) {  // V as it is
      uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v_cache) +
                                           (at_row + (long long)x.h0 * p.BS) * D);
      for (int c = lane; c < x.heads * (D / 8); c += 32)
        to[(c / (D / 8)) * p.BS * (D / 8) + c % (D / 8)] = tile[c];
    }
    __syncwarp();  // the unit is read
    if (i + kStages < n) issue(ahead, stage);
    ahead = behind(ahead);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
    fresh = next.row != x.row || next.kind != x.kind;
    x = next;
  }
}

template <int D, bool FP8, bool INTER>
cudaError_t launch_kernel(const RopeParams& p, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // may be scheduled while the kernel before it ends
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const long long row_bytes = (long long)(p.H_q + 2 * p.H_kv) * D * 2;
  constexpr int kUnitHeads = kUnitBytes / (2 * D);
  const int units = (p.H_q + kUnitHeads - 1) / kUnitHeads + 2 * ((p.H_kv + kUnitHeads - 1) / kUnitHeads);
  if (FP8 || (p.rows * row_bytes >= kManyBytes * sms && row_bytes >= units * (kUnitBytes / 2))) {
    static std::atomic<bool> limit_raised[64];
    auto kernel = paged_kv_rope_many_kernel<D, FP8, INTER>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !limit_raised[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)kStreamSmem);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) limit_raised[dev].store(true, std::memory_order_release);
    }
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(kStreamWarps * 32);
    cfg.dynamicSmemBytes = kStreamSmem;
    return cudaLaunchKernelEx(&cfg, kernel, p);
  }
  if constexpr (!FP8) {
    const int parts = (p.H_q + kHeads - 1) / kHeads + 2 * ((p.H_kv + kHeads - 1) / kHeads);
    const long long lanes = (long long)p.rows * parts * (D / 16);
    const long long want = (lanes + kThreads - 1) / kThreads, most = (long long)sms * 8;
    cfg.gridDim = dim3((unsigned)(want < most ? want : most));
    cfg.blockDim = dim3(kThreads);
    return cudaLaunchKernelEx(&cfg, paged_kv_rope_few_kernel<D, INTER>, p);
  }
  return cudaErrorInvalidValue;  // (not reached)
}

template <int D>
cudaError_t launch_as(const RopeParams& p, int sms, cudaStream_t stream) {
  if (p.k_scale != nullptr) {
    if constexpr (D >= 128)
      return p.interleaved ? launch_kernel<D, true, true>(p, sms, stream)
                           : launch_kernel<D, true, false>(p, sms, stream);
    return cudaErrorInvalidValue;
  }
  return p.interleaved ? launch_kernel<D, false, true>(p, sms, stream)
                       : launch_kernel<D, false, false>(p, sms, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, int sms, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  return p.D == 64    ? launch_as<64>(p, sms, stream)
         : p.D == 128 ? launch_as<128>(p, sms, stream)
                      : launch_as<256>(p, sms, stream);
}

}  // namespace pagedattn
