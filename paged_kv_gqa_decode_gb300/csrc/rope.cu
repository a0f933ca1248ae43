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
// What bounds it: memory.  D / 8 lanes hold one head, 16 bytes each, so the norm is a
// few shuffles and pairs of halves meet by one more; such a group of lanes takes up to
// kHeads heads of one row, whose position, cosines and sines it reads once, and all of
// whose loads are in flight together.
#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "rope.h"

namespace pagedattn {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // heads of one row that a group of lanes takes
constexpr float kE4m3Max = 448.f;
constexpr int kBadSlot = 1, kBadPosition = 2;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <int N>
__device__ __forceinline__ void load_floats(const float* src, float* x) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4*>(x + i) = __ldg(reinterpret_cast<const float4*>(src + i));
}

template <int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(kThreads) paged_kv_rope_append_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8;            // lanes of a group
  constexpr int kGroups = 32 / kLanes;     // groups of a warp
  constexpr int kPairs = INTER ? 4 : 8;    // cosines of a lane
  griddep_wait();
  griddep_launch_dependents();  // (after the wait: what is ahead of this launch is complete)
  const int lane = threadIdx.x & 31, l = lane % kLanes, group = lane / kLanes;
  const int half = p.R >> 1;
  // this lane's part of the rotation: elements 8 l .. 8 l + 7, pairs from i0 on
  const bool turns = 8 * l < p.R;
  const bool upper = !INTER && 8 * l >= half;  // holds the second elements of its pairs
  const int i0 = INTER ? 4 * l : upper ? 8 * l - half : 8 * l;
  const int partner = group * kLanes + (turns ? (upper ? l - (half >> 3) : l + (half >> 3)) : l);
  const int q_parts = (p.H_q + kHeads - 1) / kHeads, kv_parts = (p.H_kv + kHeads - 1) / kHeads;
  const int parts = q_parts + 2 * kv_parts;
  const long long items = (long long)p.rows * parts;
  const long long slots = p.num_blocks * p.BS;
  const int shift = p.BS == 32 ? 5 : 4;
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  for (long long first = ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kGroups;
       first < items; first += warps * kGroups) {
    // (a group without an item walks along: the shuffles are the whole warp's)
    const bool some = first + group < items;
    const long long item = some ? first + group : first;
    const int row = items <= 0xffffffffLL ? (int)((uint32_t)item / (uint32_t)parts)
                                          : (int)(item / parts);
    int part = (int)(item - (long long)row * parts);
    const int kind = part < q_parts ? 0 : part < q_parts + kv_parts ? 1 : 2;  // q, k, v
    part -= kind == 0 ? 0 : kind == 1 ? q_parts : q_parts + kv_parts;
    const int heads = kind == 0 ? p.H_q : p.H_kv, h0 = part * kHeads;
    const __nv_bfloat16* src = kind == 0   ? p.q + row * p.q_stride
                               : kind == 1 ? p.k + row * p.k_stride
                                           : p.v + row * p.v_stride;
    uint4 raw[kHeads];
    const long long slot =
        kind == 0 ? 0 : __ldg(reinterpret_cast<const long long*>(p.slot_map) + row);
#pragma unroll
    for (int u = 0; u < kHeads; ++u)
      // (plain loads: q_out may be q)
      raw[u] = h0 + u < heads ? *(reinterpret_cast<const uint4*>(src + (h0 + u) * D) + l)
                              : make_uint4(0u, 0u, 0u, 0u);
    // ---- the row's cosines and sines
    float c[kPairs], s[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
    }
    const bool rotate = turns && kind != 2;
    if (rotate) {
      auto position = [&](int axis) -> int {
        const int x = __ldg(p.positions + (long long)axis * p.rows + row);
        if ((x < 0 || x >= p.max_positions) && p.status != nullptr && some)
          atomicOr(p.status, kBadPosition);
        return min(max(x, 0), p.max_positions - 1);
      };
      int axis[kPairs];
      bool one = true;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) axis[i] = 0;
      if (p.freq_axis != nullptr) {
#pragma unroll
        for (int i = 0; i < kPairs; i += 4) {
          const int4 a = __ldg(reinterpret_cast<const int4*>(p.freq_axis + i0 + i));
          axis[i] = a.x;
          axis[i + 1] = a.y;
          axis[i + 2] = a.z;
          axis[i + 3] = a.w;
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          axis[i] = min(max(axis[i], 0), p.axes - 1);
          one = one && axis[i] == axis[0];
        }
      }
      if (one) {
        const float* at = p.cos_sin + (long long)position(axis[0]) * p.R + i0;
        load_floats<kPairs>(at, c);
        load_floats<kPairs>(at + half, s);
      } else {  // pairs of several axes in these 8 elements
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float* at = p.cos_sin + (long long)position(axis[i]) * p.R + i0 + i;
          c[i] = __ldg(at);
          s[i] = __ldg(at + half);
        }
      }
      if (upper) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) s[i] = -s[i];
      }
    }
    const float* norm = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : nullptr;
    const bool normed = norm != nullptr;
    float w[8];
    if (normed) load_floats<8>(norm + 8 * l, w);
    const bool any_norm = __any_sync(0xffffffffu, normed);
    long long at_row = -1;  // cache row of head 0
    if (kind != 0) {
      if (slot >= 0 && slot < slots)
        at_row = (slot >> shift) * p.H_kv * p.BS + (slot & (p.BS - 1));
      else if (slot >= slots && p.status != nullptr && some)
        atomicOr(p.status, kBadSlot);
    }
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + u;
      float x[8];
      unpack8(raw[u], x);
      if (any_norm) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (normed) {
          const float f = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= f * w[i];
        }
      }
      if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[2 * i], b = x[2 * i + 1];
          // (selected, not multiplied by one and zero: an infinity stays one)
          x[2 * i] = rotate ? a * c[i] - b * s[i] : a;
          x[2 * i + 1] = rotate ? b * c[i] + a * s[i] : b;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float other = __shfl_sync(0xffffffffu, x[i], partner);
          x[i] = rotate ? x[i] * c[i] - other * s[i] : x[i];
        }
      }
      const bool write = some && h < heads;
      const uint4 packed = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                      pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      if (kind == 0) {
        if (write)
          *(reinterpret_cast<uint4*>(p.q_out + ((long long)row * p.H_q + h) * D) + l) = packed;
      }
      if constexpr (!FP8) {
        if (kind != 0 && write && at_row >= 0) {
          __nv_bfloat16* cache = static_cast<__nv_bfloat16*>(kind == 1 ? p.k_cache : p.v_cache);
          *(reinterpret_cast<uint4*>(cache + (at_row + (long long)h * p.BS) * D) + l) =
              kind == 1 ? packed : raw[u];
        }
      } else {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (kind != 0 && write && at_row >= 0) {
          const float f = top > 0.f ? top / kE4m3Max : 1.f;
          uint32_t b[2] = {0u, 0u};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            b[i >> 2] |= (uint32_t)__nv_cvt_float_to_fp8(x[i] / f, __NV_SATFINITE, __NV_E4M3)
                         << (8 * (i & 3));
          const long long to = at_row + (long long)h * p.BS;
          uint8_t* cache = static_cast<uint8_t*>(kind == 1 ? p.k_cache : p.v_cache);
          *(reinterpret_cast<uint2*>(cache + to * D) + l) = make_uint2(b[0], b[1]);
          if (l == 0) (kind == 1 ? p.k_scale : p.v_scale)[to] = f;
        }
      }
    }
  }
}

template <int D>
cudaError_t launch_as(const RopeParams& p, const cudaLaunchConfig_t& cfg) {
  if (p.k_scale != nullptr) {
    if constexpr (D >= 128)
      return p.interleaved
                 ? cudaLaunchKernelEx(&cfg, paged_kv_rope_append_kernel<D, true, true>, p)
                 : cudaLaunchKernelEx(&cfg, paged_kv_rope_append_kernel<D, true, false>, p);
    return cudaErrorInvalidValue;
  }
  return p.interleaved
             ? cudaLaunchKernelEx(&cfg, paged_kv_rope_append_kernel<D, false, true>, p)
             : cudaLaunchKernelEx(&cfg, paged_kv_rope_append_kernel<D, false, false>, p);
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, int sms, cudaStream_t stream) {
  const int parts = (p.H_q + kHeads - 1) / kHeads + 2 * ((p.H_kv + kHeads - 1) / kHeads);
  const long long lanes = (long long)p.rows * parts * (p.D / 8);
  if (lanes == 0) return cudaSuccess;
  const long long want = (lanes + kThreads - 1) / kThreads, most = (long long)sms * 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(want < most ? want : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // may be scheduled while the kernel before it ends
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.D == 64 ? launch_as<64>(p, cfg) : p.D == 128 ? launch_as<128>(p, cfg)
                                                        : launch_as<256>(p, cfg);
}

}  // namespace pagedattn
