// C ABI of the paged-KV GQA decode library (include/paged_attn.h): argument
// validation, launch planning (grid, pipeline depth, workspace), TMA tensor
// maps, and the per-device workspace the plain entry point owns.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <memory>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "append.h"
#include "assign.h"
#include "launch.h"
#include "paged_attn.h"
#include "tile.h"

namespace pagedattn {
namespace {

thread_local int g_last_cuda_error = 0;
thread_local int g_launch_flags = 0;  // paged_attn_set_launch_flags
// paged_attn_set_checks: pool size and device status word for every call of
// this thread (0 / null: no checks)
thread_local long long g_check_blocks = 0;
thread_local int32_t* g_check_status = nullptr;
#ifdef PAGED_ATTN_WAIT_TEST
thread_local int g_test_skip_unit = -1;
thread_local int g_test_skip_publish = 0;
#endif

constexpr int kMaxSeqsPerLaunch = 4096;
constexpr size_t kWsAlign = 256;
constexpr int kAppendApartPieces = 4;  // (s, g) pieces per CTA from which the append runs apart
constexpr int kMaxMultiRows = 256;      // multi-token decode: max q_len * G (16 pieces of 16 rows)
constexpr long long kRingBytesPerSm = 128 << 10;            // K/V rings of one SM, few pieces per CTA
constexpr long long kRingBytesPerSmManyPieces = 160 << 10;  // ... two or more pieces per CTA
constexpr long long kRingBytesPerSmThreeCtas = 150 << 10;   // three FP8 CTAs: 12 stages each

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int cuda_fail(int err) {
  g_last_cuda_error = err;
  return PAGED_ATTN_ERR_CUDA;
}

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int validate_sizes(int num_seqs, int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
                   int block_size) {
  if (H_kv <= 0 || H_q <= 0 || H_q % H_kv != 0 || H_q / H_kv > 16) return PAGED_ATTN_ERR_HEADS;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PAGED_ATTN_ERR_HEAD_DIM;
  if (block_size != 16 && block_size != 32) return PAGED_ATTN_ERR_BLOCK_SIZE;
  if (num_seqs < 0 || max_blocks_per_seq <= 0) return PAGED_ATTN_ERR_SIZES;
  // lengths up to max_blocks_per_seq * block_size must fit int32; table rows must be indexable
  if ((long long)max_blocks_per_seq * block_size > 0x7fffffffLL) return PAGED_ATTN_ERR_SIZES;
  if ((long long)H_kv * block_size > 0x7fffffffLL) return PAGED_ATTN_ERR_SIZES;
  return PAGED_ATTN_OK;
}

struct DeviceInfo {
  int sms = 0;
  int max_smem = 0;     // opt-in dynamic shared memory per block
  int smem_per_sm = 0;  // shared memory per multiprocessor
};

struct OwnedWorkspace {
  void* ptr = nullptr;
  size_t bytes = 0;
};

// Per-device state, indexed by device ordinal (guarded by g_mu; g_ws by g_ws_mu).
constexpr int kMaxDevices = 64;
std::mutex g_mu;
DeviceInfo g_info[kMaxDevices];
OwnedWorkspace g_ws[kMaxDevices];
void* g_static_scratch_ptr[kMaxDevices];  // address of the static scratch array

int current_device(int* dev) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (*dev < 0 || *dev >= kMaxDevices) return cuda_fail(cudaErrorInvalidDevice);
  return PAGED_ATTN_OK;
}

int device_info(DeviceInfo* out, int* dev_out = nullptr) {
  int dev = 0;
  int rc = current_device(&dev);
  if (rc != PAGED_ATTN_OK) return rc;
  if (dev_out) *dev_out = dev;
  thread_local DeviceInfo tl_info[kMaxDevices];  // this thread's copy of g_info
  if (tl_info[dev].sms > 0) {
    *out = tl_info[dev];
    return PAGED_ATTN_OK;
  }
  cudaError_t e;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_info[dev].sms > 0) {
    *out = tl_info[dev] = g_info[dev];
    return PAGED_ATTN_OK;
  }
  DeviceInfo di;
  if ((e = cudaDeviceGetAttribute(&di.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return cuda_fail(e);
  if ((e = cudaDeviceGetAttribute(&di.max_smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) !=
      cudaSuccess)
    return cuda_fail(e);
  if ((e = cudaDeviceGetAttribute(&di.smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor,
                                  dev)) != cudaSuccess)
    return cuda_fail(e);
  g_info[dev] = tl_info[dev] = di;
  *out = di;
  return PAGED_ATTN_OK;
}

// The end of a workspace's status word and combine counters, which must be zero
// between calls: whatever else a call puts into a workspace begins here.
size_t counters_end(const DeviceInfo& di) {
  return kWsAlign + round_up((size_t)di.sms * kMaxCtasPerSm * 4, kWsAlign);
}

// Everything a launch needs that depends only on sizes and the device.
struct Plan {
  int D, BS, G;
  bool g16;
  bool fp8;     // FP8 caches
  bool xp;      // x-packed K / D-major V caches (bf16)
  bool mod;     // score options (or a state output)
  int rows;     // query rows of one piece: G, or a multi-token chunk (8 or 16)
  int qchunks;  // multi-token decode: pieces per (sequence, KV head); 0: single token
  int chunk;    // sequences per launch
  int stages;   // pipeline depth
  size_t smem;  // dynamic shared memory per CTA
  int grid;     // persistent CTAs
  size_t off_counters, off_partials, ws_bytes;
};

// G: query rows of one piece; qchunks > 0: multi-token decode (room for chunk + 1
// row offsets and the page prefixes of qchunks passes).
// qchunks < 0: decode with score options (room for two values per sequence).
template <int D, int BS, bool FP8>
bool plan_smem(int G, int chunk, int max_smem, long long ring_cap, int qchunks, int* stages,
               size_t* smem) {
  using L = SmemLayout<D, BS, FP8>;
  const int qo_entries = qchunks > 0 ? chunk + 1 : qchunks < 0 ? 2 * chunk : 0;
  const int walks = qchunks > 0 ? qchunks : 1;
  const L none{0, G, chunk, qo_entries, walks};
  const long long fixed = none.total() + 2048;  // + alignment slack and static shared memory
  const long long per_stage = L::kStageBytes + L::kScaleBytes + 16;
  long long st = (max_smem - fixed) / per_stage;
  if (st > kMaxStages) st = kMaxStages;
  if (st > ring_cap / L::kStageBytes) st = ring_cap / L::kStageBytes;
  // At least one slot per consumer warp (slot s belongs to warp s % 4).
  if (st < kConsumerWarps) return false;
  const L lay{(int)st, G, chunk, qo_entries, walks};
  *stages = (int)st;
  *smem = (size_t)lay.total() + 1024;
  return *smem + 256 <= (size_t)max_smem;  // + the kernel's static shared memory
}

template <bool FP8>
bool plan_smem_d(int D, int BS, int G, int chunk, int max_smem, long long ring_cap,
                 int qchunks, int* stages, size_t* smem) {
  if (D == 64) {
    if constexpr (FP8) return false;  // FP8 caches need head_dim 128 or 256
    else
      return BS == 16 ? plan_smem<64, 16, false>(G, chunk, max_smem, ring_cap, qchunks, stages, smem)
                      : plan_smem<64, 32, false>(G, chunk, max_smem, ring_cap, qchunks, stages, smem);
  }
  if (D == 128)
    return BS == 16 ? plan_smem<128, 16, FP8>(G, chunk, max_smem, ring_cap, qchunks, stages, smem)
                    : plan_smem<128, 32, FP8>(G, chunk, max_smem, ring_cap, qchunks, stages, smem);
  return BS == 16 ? plan_smem<256, 16, FP8>(G, chunk, max_smem, ring_cap, qchunks, stages, smem)
                  : plan_smem<256, 32, FP8>(G, chunk, max_smem, ring_cap, qchunks, stages, smem);
}

bool plan_smem_any(int D, int BS, bool fp8, int G, int chunk, int max_smem, long long ring_cap,
                   int qchunks, int* stages, size_t* smem) {
  return fp8 ? plan_smem_d<true>(D, BS, G, chunk, max_smem, ring_cap, qchunks, stages, smem)
             : plan_smem_d<false>(D, BS, G, chunk, max_smem, ring_cap, qchunks, stages, smem);
}

// rows > 0: multi-token decode with `rows` query rows per piece and `qchunks`
// pieces per (sequence, KV head).  mod: decode with score options.
int make_plan(int num_seqs, int H_q, int H_kv, int D, int BS, const DeviceInfo& di, Plan* pl,
              bool fp8 = false, int rows = 0, int qchunks = 0, bool mod = false) {
  pl->D = D;
  pl->fp8 = fp8;
  pl->xp = false;
  pl->mod = mod;
  pl->BS = BS;
  pl->G = H_q / H_kv;
  pl->rows = rows > 0 ? rows : pl->G;
  pl->qchunks = rows > 0 ? qchunks : 0;
  pl->g16 = pl->rows > 8;
  const int chunk0 =
      num_seqs < kMaxSeqsPerLaunch ? (num_seqs > 0 ? num_seqs : 1) : kMaxSeqsPerLaunch;
  // Two CTAs per SM (two independent pipelines) when their shared memory fits,
  // else one.  Keep at least 4 pipeline stages where possible by launching
  // fewer sequences at a time.
  bool ok = false;
  int chunk = chunk0;
  for (int occ = ctas_per_sm(D, pl->g16, BS, fp8); occ >= 1 && !ok; --occ) {
    int budget = di.smem_per_sm / occ - 1024;  // 1 KB per CTA is reserved by the system
    if (budget > di.max_smem) budget = di.max_smem;
    chunk = chunk0;
    for (;;) {
      // Bytes in flight per SM: past about 128 KB the memory system delivers no
      // more and a deeper ring measured slower (LLaMA-shaped batch, 8 KB pages, two
      // CTAs per SM: 8 stages 51.4 us, 10 52.2, 12 53.3); CTAs that cross many
      // (s, g) pieces gain from a deeper ring that absorbs the stall at each
      // piece end (ragged 256-sequence batch: 8 stages 617 us, 10 608).
      // Three FP8 CTAs per SM: 12 stages each (8 measured slower on the
      // LLaMA-shaped batch, 32.7 against 31.0 us; 16 do not fit).
      const long long pieces = (long long)chunk * H_kv * (pl->qchunks > 0 ? pl->qchunks : 1);
      const long long ring_cap =
          (occ >= 3                           ? kRingBytesPerSmThreeCtas
           : pieces >= 2LL * di.sms * occ ? kRingBytesPerSmManyPieces
                                          : kRingBytesPerSm) /
          occ;
      if (plan_smem_any(D, BS, fp8, pl->rows, chunk, budget, ring_cap, mod ? -1 : pl->qchunks,
                        &pl->stages, &pl->smem) &&
          (pl->stages >= 4 || chunk <= 64)) {
        ok = true;
        pl->grid = di.sms * occ;
        break;
      }
      if (chunk <= 1) break;
      chunk = (chunk + 1) / 2;
    }
  }
  if (!ok) return PAGED_ATTN_ERR_SIZES;
  pl->chunk = chunk;
  // [0, 256): status word; then one combine counter per CTA of the largest grid
  // any launch on this device uses (kMaxCtasPerSm CTAs per SM); then the
  // partial states.
  // The counter region depends on the device only (not on this launch's grid,
  // which is one CTA per SM for some shapes), so a workspace reused by calls of
  // any size always finds it zero: partials never land on it.
  pl->off_counters = kWsAlign;
  pl->off_partials = counters_end(di);
  pl->ws_bytes = pl->off_partials +
                 round_up((size_t)pl->grid * 2 * pl->rows * (size_t)(D + 4) * 4, kWsAlign);
  return PAGED_ATTN_OK;
}

// make_plan through a small per-thread cache: the plan depends only on the
// sizes, the variant and the device, so a decode loop plans once.
int cached_plan(int num_seqs, int H_q, int H_kv, int D, int BS, int dev, const DeviceInfo& di,
                Plan* pl, bool fp8 = false, int rows = 0, int qchunks = 0, bool mod = false) {
  struct Entry {
    int key[9];
    Plan plan;
    bool used;
  };
  constexpr int kEntries = 16;
  thread_local Entry tl_plans[kEntries] = {};
  const int key[9] = {num_seqs, H_q, H_kv, D, BS, (fp8 ? 1 : 0) + (mod ? 2 : 0), rows,
                      qchunks, dev};
  uint32_t h = 2166136261u;
  for (int k : key) h = (h ^ (uint32_t)k) * 16777619u;
  Entry& e = tl_plans[h % kEntries];
  if (e.used && std::memcmp(e.key, key, sizeof key) == 0) {
    *pl = e.plan;
    return PAGED_ATTN_OK;
  }
  int rc = make_plan(num_seqs, H_q, H_kv, D, BS, di, pl, fp8, rows, qchunks, mod);
  if (rc != PAGED_ATTN_OK) return rc;
  std::memcpy(e.key, key, sizeof key);
  e.plan = *pl;
  e.used = true;
  return PAGED_ATTN_OK;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int get_encoder(EncodeTiledFn* fn) {
  static EncodeTiledFn cached = nullptr;
  static cudaError_t cached_err = cudaSuccess;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    cached_err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                  cudaEnableDefault, &q);
    if (cached_err == cudaSuccess && q == cudaDriverEntryPointSuccess)
      cached = reinterpret_cast<EncodeTiledFn>(p);
    else if (cached_err == cudaSuccess)
      cached_err = cudaErrorSymbolNotFound;
  });
  if (!cached) return cuda_fail(cached_err);
  *fn = cached;
  return PAGED_ATTN_OK;
}

// 4-D view of a cache: (column within a 64-column half, row within a block =
// kv_head * BS + slot, half, block id).  A page of one KV head is the box
// {64, BS, D / 64, 1} at (0, g * BS, 0, block); it lands in shared memory as
// [half][row][128 bytes] with the 128-byte swizzle the kernel's ldmatrix
// addressing expects.
int encode_cache_map(const void* base, int D, int BS, int H_kv, long long num_blocks,
                     CUtensorMap* map, bool fp8 = false) {
  EncodeTiledFn enc = nullptr;
  int rc = get_encoder(&enc);
  if (rc != PAGED_ATTN_OK) return rc;
  const int elem = fp8 ? 1 : 2;          // bytes per element
  const cuuint64_t inner = 128 / elem;   // elements in a 128-byte half of a row
  const cuuint64_t halves = (cuuint64_t)D * elem / 128;
  const cuuint64_t row_bytes = (cuuint64_t)D * elem;
  const cuuint64_t block_bytes = row_bytes * (cuuint64_t)H_kv * BS;
  cuuint64_t nb = (cuuint64_t)num_blocks;
  if (num_blocks <= 0) {
    // pool size unknown: any non-negative int32 block id is addressable, as long
    // as the described extent stays below 2^40 bytes
    nb = ((cuuint64_t)1 << 40) / block_bytes;
    if (nb > 0x7fffffffULL) nb = 0x7fffffffULL;
  }
  const cuuint64_t dims[4] = {inner, (cuuint64_t)H_kv * BS, halves, nb};
  const cuuint64_t strides[3] = {row_bytes, 128, block_bytes};
  const cuuint32_t box[4] = {(cuuint32_t)inner, (cuuint32_t)BS, (cuuint32_t)halves, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   4, const_cast<void*>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cuda_fail((int)r);
  return PAGED_ATTN_OK;
}

// The same view with a box of one 128-byte column half of a page, {64, BS, 1, 1}:
// the row-tile kernel stacks the halves of several pages.
int encode_half_map(const void* base, int D, int BS, int H_kv, long long num_blocks,
                    CUtensorMap* map) {
  EncodeTiledFn enc = nullptr;
  int rc = get_encoder(&enc);
  if (rc != PAGED_ATTN_OK) return rc;
  const cuuint64_t row_bytes = (cuuint64_t)D * 2;
  const cuuint64_t block_bytes = row_bytes * (cuuint64_t)H_kv * BS;
  cuuint64_t nb = (cuuint64_t)num_blocks;
  if (num_blocks <= 0) {
    nb = ((cuuint64_t)1 << 40) / block_bytes;
    if (nb > 0x7fffffffULL) nb = 0x7fffffffULL;
  }
  const cuuint64_t dims[4] = {64, (cuuint64_t)H_kv * BS, (cuuint64_t)D / 64, nb};
  const cuuint64_t strides[3] = {row_bytes, 128, block_bytes};
  const cuuint32_t box[4] = {64, (cuuint32_t)BS, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cuda_fail((int)r);
  return PAGED_ATTN_OK;
}

// x-packed caches.  A page of one KV head is contiguous in both (K [num_blocks,
// H_kv, D / 8, BS, 8], V [num_blocks, H_kv, D, BS]) and the kernel bulk-copies
// it, except V pages of 32 tokens, read through the 4-D view (BS, D, H_kv,
// block) of V: the box {BS, D, 1, 1} lands as [D][BS] with the 64-byte swizzle.
// The K map of the launch is unused and set to the same view.
int encode_xpacked_maps(const void* v, int D, int BS, int H_kv, long long num_blocks,
                        CUtensorMap* tk, CUtensorMap* tv) {
  EncodeTiledFn enc = nullptr;
  int rc = get_encoder(&enc);
  if (rc != PAGED_ATTN_OK) return rc;
  const cuuint64_t head_bytes = (cuuint64_t)D * BS * 2;
  const cuuint64_t block_bytes = head_bytes * (cuuint64_t)H_kv;
  cuuint64_t nb = (cuuint64_t)num_blocks;
  if (num_blocks <= 0) {
    nb = ((cuuint64_t)1 << 40) / block_bytes;
    if (nb > 0x7fffffffULL) nb = 0x7fffffffULL;
  }
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const cuuint64_t vdims[4] = {(cuuint64_t)BS, (cuuint64_t)D, (cuuint64_t)H_kv, nb};
  const cuuint64_t vstrides[3] = {(cuuint64_t)BS * 2, head_bytes, block_bytes};
  const cuuint32_t vbox[4] = {(cuuint32_t)BS, (cuuint32_t)D, 1, 1};
  CUresult r = enc(tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(v), vdims,
                   vstrides, vbox, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   BS == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cuda_fail((int)r);
  *tk = *tv;
  return PAGED_ATTN_OK;
}

cudaError_t launch_dim(int D, int BS, bool g16, bool fp8, bool xp, bool mod,
                       const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p,
                       int grid, size_t smem, cudaStream_t st) {
#ifdef PAGED_ATTN_WAIT_TEST
  // the test build carries the single-token bf16 head_dim-128 kernels only
  if (p.qo_indptr != nullptr || xp || fp8 || mod || D != 128) return cudaErrorNotSupported;
  return launch_decode_d128(BS, g16, tk, tv, p, grid, smem, st);
#else
  if (mod && fp8)
    return D == 128 ? launch_decode_fp8_mod_d128(BS, g16, tk, tv, p, grid, smem, st)
                    : launch_decode_fp8_mod_d256(BS, g16, tk, tv, p, grid, smem, st);
  if (mod) {
    if (D == 64) return launch_decode_mod_d64(BS, g16, tk, tv, p, grid, smem, st);
    if (D == 128) return launch_decode_mod_d128(BS, g16, tk, tv, p, grid, smem, st);
    return launch_decode_mod_d256(BS, g16, tk, tv, p, grid, smem, st);
  }
  if (p.qo_indptr != nullptr) {
    if (D == 64) return launch_decode_multi_d64(BS, g16, tk, tv, p, grid, smem, st);
    if (D == 128) return launch_decode_multi_d128(BS, g16, tk, tv, p, grid, smem, st);
    return launch_decode_multi_d256(BS, g16, tk, tv, p, grid, smem, st);
  }
  if (xp) {
    if (D == 64) return launch_decode_xp_d64(BS, g16, tk, tv, p, grid, smem, st);
    if (D == 128) return launch_decode_xp_d128(BS, g16, tk, tv, p, grid, smem, st);
    return launch_decode_xp_d256(BS, g16, tk, tv, p, grid, smem, st);
  }
  if (fp8)
    return D == 128 ? launch_decode_fp8_d128(BS, g16, tk, tv, p, grid, smem, st)
                    : launch_decode_fp8_d256(BS, g16, tk, tv, p, grid, smem, st);
  if (D == 64) return launch_decode_d64(BS, g16, tk, tv, p, grid, smem, st);
  if (D == 128) return launch_decode_d128(BS, g16, tk, tv, p, grid, smem, st);
  return launch_decode_d256(BS, g16, tk, tv, p, grid, smem, st);
#endif
}

int check_pointers(const void* q, const void* k, const void* v, const void* out,
                   const int32_t* bt, const int32_t* sl) {
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(bt) ||
      !aligned16(sl))
    return PAGED_ATTN_ERR_POINTER;
  return PAGED_ATTN_OK;
}

// The tensor maps of a call through a per-thread direct-mapped cache: a map
// depends only on the base address and the sizes it describes, so a decode
// loop over the same caches encodes each once.
enum MapKind { kMapBf16 = 0, kMapFp8 = 1, kMapXpackedV = 2, kMapHalf = 3 };

int cached_map(const void* base, int D, int BS, int H_kv, long long num_blocks, MapKind kind,
               CUtensorMap* out) {
  struct Entry {
    CUtensorMap map;
    const void* base;
    long long num_blocks;
    int D, BS, H_kv, kind;
    bool used;
  };
  constexpr int kEntries = 256;
  thread_local std::unique_ptr<Entry[]> tl_maps;
  if (!tl_maps) tl_maps.reset(new Entry[kEntries]());
  const uint64_t a = reinterpret_cast<uintptr_t>(base);
  const uint64_t h = (a >> 8) * 0x9E3779B97F4A7C15ull ^ ((uint64_t)kind << 1) ^
                     ((uint64_t)D * 31 + (uint64_t)BS * 7 + (uint64_t)H_kv);
  Entry& e = tl_maps[(h >> 32) % kEntries];
  if (e.used && e.base == base && e.num_blocks == num_blocks && e.D == D && e.BS == BS &&
      e.H_kv == H_kv && e.kind == kind) {
    *out = e.map;
    return PAGED_ATTN_OK;
  }
  CUtensorMap m;
  int rc;
  if (kind == kMapXpackedV) {
    CUtensorMap unused;
    rc = encode_xpacked_maps(base, D, BS, H_kv, num_blocks, &unused, &m);
  } else if (kind == kMapHalf) {
    rc = encode_half_map(base, D, BS, H_kv, num_blocks, &m);
  } else {
    rc = encode_cache_map(base, D, BS, H_kv, num_blocks, &m, kind == kMapFp8);
  }
  if (rc != PAGED_ATTN_OK) return rc;
  e.map = m;
  e.base = base;
  e.num_blocks = num_blocks;
  e.D = D;
  e.BS = BS;
  e.H_kv = H_kv;
  e.kind = kind;
  e.used = true;
  *out = m;
  return PAGED_ATTN_OK;
}

// Everything one decode call hands to its launches.
struct Operands {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  void* out;
  const int32_t* bt;
  const int32_t* seq_lens;
  int num_seqs, H_q, H_kv, maxb;
  float scale;
  void* ws;                         // workspace (status word, counters, partials)
  int32_t* status = nullptr;        // caller status word (null: the workspace's)
  long long num_blocks = 0;         // > 0: block ids checked against the pool
  bool early = false;               // early-prologue launch (caller's guarantee holds)
  const void* k_new = nullptr;      // fused cache append (bf16)
  const void* v_new = nullptr;
  const float* k_scale = nullptr;   // FP8 row floats
  const float* v_scale = nullptr;
  const int32_t* qo_indptr = nullptr;  // multi-token decode
  int total_q = 0;
  int causal = 1;
  // score options
  float softcap = 0.f;
  const float* slopes = nullptr;
  int window = 0;
  const int32_t* prefix_lens = nullptr;
  const int32_t* doc_starts = nullptr;
  bool independent = false;  // needs nothing of the launch just ahead (DecodeParams)
  float* state = nullptr;  // softmax states [num_seqs * H_q][D + 4] instead of the output
};

// The calling thread's device-side checks (paged_attn_set_checks), if any.
void apply_checks(Operands* o) {
  if (g_check_blocks > 0) {
    o->num_blocks = g_check_blocks;
    o->status = g_check_status;
  }
}

// The early prologue applies when the caller asked for it on this thread and
// nothing the library itself launched just before writes what the producer
// reads ahead of the wait.
bool early_requested() { return (g_launch_flags & PAGED_ATTN_FLAG_EARLY_PROLOGUE) != 0; }

// Runs the whole operation in chunks of plan.chunk sequences on `stream`.
int run(const Plan& pl, const Operands& o, cudaStream_t stream) {
  CUtensorMap tk, tv;
  int rc;
  if (pl.xp) {
    rc = cached_map(o.v_cache, pl.D, pl.BS, o.H_kv, o.num_blocks, kMapXpackedV, &tv);
    if (rc != PAGED_ATTN_OK) return rc;
    tk = tv;  // unused by the x-packed kernel
  } else {
    const MapKind kind = pl.fp8 ? kMapFp8 : kMapBf16;
    rc = cached_map(o.k_cache, pl.D, pl.BS, o.H_kv, o.num_blocks, kind, &tk);
    if (rc != PAGED_ATTN_OK) return rc;
    rc = cached_map(o.v_cache, pl.D, pl.BS, o.H_kv, o.num_blocks, kind, &tv);
    if (rc != PAGED_ATTN_OK) return rc;
  }
  uint8_t* wsb = static_cast<uint8_t*>(o.ws);
  for (int s0 = 0; s0 < o.num_seqs; s0 += pl.chunk) {
    const int n = o.num_seqs - s0 < pl.chunk ? o.num_seqs - s0 : pl.chunk;
    DecodeParams p;
    // multi-token decode: q and out rows are found through qo_indptr (absolute)
    const size_t row0 = o.qo_indptr ? 0 : (size_t)s0;
    p.q = static_cast<const __nv_bfloat16*>(o.q) + row0 * o.H_q * pl.D;
    p.out = static_cast<__nv_bfloat16*>(o.out) + row0 * o.H_q * pl.D;
    p.qo_indptr = o.qo_indptr ? o.qo_indptr + s0 : nullptr;
    p.rows = pl.rows;
    p.chunks = pl.qchunks > 0 ? pl.qchunks : 1;
    p.total_q = o.total_q;
    p.causal = o.causal;
    p.block_tables = o.bt + (size_t)s0 * o.maxb;
    p.seq_lens = o.seq_lens + s0;
    p.num_seqs = n;
    p.H_q = o.H_q;
    p.H_kv = o.H_kv;
    p.G = pl.G;
    p.maxb = o.maxb;
    p.stages = pl.stages;
    p.scale_log2 = o.scale * 1.4426950408889634f;
    p.status = o.status ? o.status : reinterpret_cast<int32_t*>(wsb);
    p.counters = reinterpret_cast<int32_t*>(wsb + pl.off_counters);
    p.partials = reinterpret_cast<float*>(wsb + pl.off_partials);
    p.num_blocks = o.num_blocks;
    p.early = o.early ? 1 : 0;
    p.cap_log2 = o.softcap * 1.4426950408889634f;
    p.cap_in = o.softcap > 0.f ? o.scale / o.softcap : 0.f;
    p.slopes = o.slopes;
    p.window = o.window;
    p.prefix_lens = o.prefix_lens ? o.prefix_lens + s0 : nullptr;
    p.doc_starts = o.doc_starts ? o.doc_starts + s0 : nullptr;
    p.independent = o.independent && s0 == 0 ? 1 : 0;
    p.state = o.state ? o.state + (size_t)s0 * o.H_q * (pl.D + 4) : nullptr;
    p.k_new = o.k_new ? static_cast<const __nv_bfloat16*>(o.k_new) + (size_t)s0 * o.H_kv * pl.D
                      : nullptr;
    p.v_new = o.v_new ? static_cast<const __nv_bfloat16*>(o.v_new) + (size_t)s0 * o.H_kv * pl.D
                      : nullptr;
    p.k_cache = static_cast<__nv_bfloat16*>(const_cast<void*>(o.k_cache));
    p.v_cache = static_cast<__nv_bfloat16*>(const_cast<void*>(o.v_cache));
    p.k_scale = o.k_scale;
    p.v_scale = o.v_scale;
#ifdef PAGED_ATTN_WAIT_TEST
    p.test_skip_unit = g_test_skip_unit;
    p.test_skip_publish = g_test_skip_publish;
#endif
    cudaError_t e =
        launch_dim(pl.D, pl.BS, pl.g16, pl.fp8, pl.xp, pl.mod, tk, tv, p,
                   pl.grid + p.independent, pl.smem, stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return PAGED_ATTN_OK;
}

// Guards the library-owned workspaces.  A call that uses one holds it until its launches
// are enqueued: another host thread's larger call releases the buffer in stream order,
// which must come after them.
std::mutex g_ws_mu;
using WorkspaceHold = std::unique_lock<std::mutex>;

// Grows a workspace to at least `bytes`, zero-filled.  Earlier calls on this stream may
// still use the old buffer: it is released in stream order, and the new one is made so
// (the device's default pool).  No device-wide sync.
int grow(OwnedWorkspace* w, size_t bytes, cudaStream_t stream) {
  if (w->bytes >= bytes) return PAGED_ATTN_OK;
  cudaError_t e;
  if (w->ptr) {
    if ((e = cudaFreeAsync(w->ptr, stream)) != cudaSuccess) return cuda_fail(e);
    *w = OwnedWorkspace();
  }
  void* p = nullptr;
  if ((e = cudaMallocAsync(&p, bytes, stream)) != cudaSuccess) return cuda_fail(e);
  if ((e = cudaMemsetAsync(p, 0, bytes, stream)) != cudaSuccess) {
    cudaFreeAsync(p, stream);
    return cuda_fail(e);
  }
  w->ptr = p;
  w->bytes = bytes;
  return PAGED_ATTN_OK;
}

// The library-owned workspace of the current device, grown to at least `bytes` (calls on
// other streams overlapping this one race on it, as the header says).
int owned_workspace(size_t bytes, cudaStream_t stream, void** out, WorkspaceHold* hold) {
  int dev = 0;
  int rc = current_device(&dev);
  if (rc != PAGED_ATTN_OK) return rc;
  *hold = WorkspaceHold(g_ws_mu);
  if ((rc = grow(&g_ws[dev], bytes, stream)) != PAGED_ATTN_OK) return rc;
  *out = g_ws[dev].ptr;
  return PAGED_ATTN_OK;
}

// The workspace of a call that takes an optional one: the caller's, or one that the
// library keeps for the call's stream (apart from owned_workspace, whose buffer captured
// graphs of the other entry points may hold), so that calls on different streams need
// nothing of each other.  A stream being captured must bring its own: a graph must not
// keep a buffer that a later, larger call releases.
// Streams are told apart by their id, which is never given out twice (a handle may be).
struct StreamWorkspace {
  unsigned long long stream;
  unsigned long long last_use;
  OwnedWorkspace w;
};
constexpr int kStreamWorkspaces = 64;
struct StreamWorkspaces {
  int count = 0;
  unsigned long long uses = 0;
  StreamWorkspace entry[kStreamWorkspaces];
};
StreamWorkspaces g_opt_ws[kMaxDevices];  // guarded by g_ws_mu

// The entry of a stream, made where there is none: past kStreamWorkspaces streams the
// least recently used one's is taken over, once the device has finished all work.
int stream_workspace(StreamWorkspaces& all, unsigned long long id, cudaStream_t stream,
                     OwnedWorkspace** out) {
  StreamWorkspace* x = nullptr;
  for (int k = 0; k < all.count && x == nullptr; ++k)
    if (all.entry[k].stream == id) x = &all.entry[k];
  if (x == nullptr && all.count < kStreamWorkspaces) {
    x = &all.entry[all.count++];
    *x = StreamWorkspace();
    x->stream = id;
  }
  if (x == nullptr) {
    x = &all.entry[0];
    for (StreamWorkspace& y : all.entry)
      if (y.last_use < x->last_use) x = &y;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess && x->w.ptr) e = cudaFreeAsync(x->w.ptr, stream);
    if (e != cudaSuccess) return cuda_fail(e);
    *x = StreamWorkspace();
    x->stream = id;
  }
  x->last_use = ++all.uses;
  *out = &x->w;
  return PAGED_ATTN_OK;
}

int optional_workspace(void* workspace, size_t workspace_bytes, size_t need, cudaStream_t stream,
                       void** out, WorkspaceHold* hold) {
  if (workspace != nullptr) {
    if ((reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) != 0 || workspace_bytes < need)
      return PAGED_ATTN_ERR_WORKSPACE;
    *out = workspace;
    return PAGED_ATTN_OK;
  }
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(stream, &cap);
  if (e != cudaSuccess) return cuda_fail(e);
  if (cap != cudaStreamCaptureStatusNone) return PAGED_ATTN_ERR_WORKSPACE;
  int dev = 0;
  int rc = current_device(&dev);
  if (rc != PAGED_ATTN_OK) return rc;
  unsigned long long id = 0;
  if ((e = cudaStreamGetId(stream, &id)) != cudaSuccess) return cuda_fail(e);
  *hold = WorkspaceHold(g_ws_mu);
  OwnedWorkspace* w = nullptr;
  if ((rc = stream_workspace(g_opt_ws[dev], id, stream, &w)) != PAGED_ATTN_OK) return rc;
  if ((rc = grow(w, need, stream)) != PAGED_ATTN_OK) return rc;
  *out = w->ptr;
  return PAGED_ATTN_OK;
}

// Scratch for paged_attn_decode_static: a fixed array every GPU that loads the
// library holds until the process exits, so that entry point never allocates.
constexpr size_t kStaticScratchBytes = size_t(4) << 20;  // 4 MiB
static __device__ __align__(256) unsigned char g_static_scratch[kStaticScratchBytes];

// Device address of g_static_scratch on the current device, looked up once per
// device (in host code the array's name is only a stand-in, not an address).
int static_scratch_address(void** out) {
  int dev = 0;
  int rc = current_device(&dev);
  if (rc != PAGED_ATTN_OK) return rc;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_static_scratch_ptr[dev] != nullptr) {
    *out = g_static_scratch_ptr[dev];
    return PAGED_ATTN_OK;
  }
  void* ptr = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&ptr, g_static_scratch);
  if (e != cudaSuccess) return cuda_fail(e);
  g_static_scratch_ptr[dev] = ptr;
  *out = ptr;
  return PAGED_ATTN_OK;
}

int common_checks(const void* q, const void* k, const void* v, const void* out, const int32_t* bt,
                  const int32_t* sl, int num_seqs, int H_q, int H_kv, int head_dim,
                  int max_blocks_per_seq, int block_size, float scale) {
  int rc = validate_sizes(num_seqs, H_q, H_kv, head_dim, max_blocks_per_seq, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  if (!std::isfinite(scale)) return PAGED_ATTN_ERR_SCALE;
  if (num_seqs == 0) return PAGED_ATTN_OK;
  return check_pointers(q, k, v, out, bt, sl);
}

// A decode call's operands with the caller's pointers and sizes.
Operands operands(const void* q, const void* k_cache, const void* v_cache, void* out,
                  const int32_t* bt, const int32_t* sl, int num_seqs, int H_q, int H_kv,
                  int max_blocks_per_seq, float scale) {
  Operands o;
  o.q = q;
  o.k_cache = k_cache;
  o.v_cache = v_cache;
  o.out = out;
  o.bt = bt;
  o.seq_lens = sl;
  o.num_seqs = num_seqs;
  o.H_q = H_q;
  o.H_kv = H_kv;
  o.maxb = max_blocks_per_seq;
  o.scale = scale;
  o.ws = nullptr;
  return o;
}

// Plans a decode launch on the current device and runs it in the library-owned
// workspace (o.ws null) or the one given.  rows > 0: multi-token pieces.
int plan_and_run(Operands& o, int head_dim, int block_size, bool fp8, bool xp, int rows,
                 int qchunks, cudaStream_t st) {
  int dev = 0;
  DeviceInfo di;
  int rc = device_info(&di, &dev);
  if (rc != PAGED_ATTN_OK) return rc;
  Plan pl;
  rc = cached_plan(o.num_seqs, o.H_q, o.H_kv, head_dim, block_size, dev, di, &pl, fp8, rows,
                   qchunks);
  if (rc != PAGED_ATTN_OK) return rc;
  pl.xp = xp;  // same shared-memory plan as the bf16 layout
  WorkspaceHold hold;
  if (o.ws == nullptr && (rc = owned_workspace(pl.ws_bytes, st, &o.ws, &hold)) != PAGED_ATTN_OK)
    return rc;
  return run(pl, o, st);
}

// Score options as the entry points take them (arrays 4-byte aligned or null).
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

int mods_checks(float scale, long long max_tokens, float softcap, const float* slopes,
                int window, const int32_t* prefix_lens, const int32_t* doc_starts) {
  // token positions a tile past the last one stay inside int32
  if (max_tokens > 0x7fffff00LL) return PAGED_ATTN_ERR_SIZES;
  // (what the score arithmetic needs: scale / softcap and softcap log2(e) far inside float32)
  if (softcap != 0.f &&
      !(softcap >= 1e-30f && softcap <= 1e30f && std::fabs(scale / softcap) <= 1e30f))
    return PAGED_ATTN_ERR_MODS;
  if (window < 0) return PAGED_ATTN_ERR_MODS;
  if (!aligned4(slopes) || !aligned4(prefix_lens) || !aligned4(doc_starts))
    return PAGED_ATTN_ERR_POINTER;
  return PAGED_ATTN_OK;
}

// A decode call with score options, its arguments checked.
int decode_mods_impl(Operands& o, int head_dim, int block_size, bool fp8, void* workspace,
                     size_t workspace_bytes, cudaStream_t st) {
  apply_checks(&o);
  int dev = 0;
  DeviceInfo di;
  int rc = device_info(&di, &dev);
  if (rc != PAGED_ATTN_OK) return rc;
  Plan pl;
  rc = cached_plan(o.num_seqs, o.H_q, o.H_kv, head_dim, block_size, dev, di, &pl, fp8, 0, 0, true);
  if (rc != PAGED_ATTN_OK) return rc;
  WorkspaceHold hold;
  rc = optional_workspace(workspace, workspace_bytes, pl.ws_bytes, st, &o.ws, &hold);
  if (rc != PAGED_ATTN_OK) return rc;
  return run(pl, o, st);
}

// Row-tile attention (multi-token decode with score options, shared prefixes).
constexpr int kMaxSplits = 32;  // the merge gives one lane to each part

// Row tiles a launch provides for (an upper bound that needs no device value).
long long tile_bound(int total_q, int num_seqs, int G, int teams) {
  return (long long)total_q * G / (128 * teams) + num_seqs;
}

// Parts of each piece's token range: one when the pieces fill the places there are
// for CTAs (two on an SM for the one-team kernels of head_dim 64 and 128), else as many as
// make 1.75 CTAs a place, so that the longest parts end near the others (fewer
// leave SMs idle behind a long sequence, more pay each CTA's 4 us of start and end:
// verification of five tokens, 272 pieces, 1 / 2 / 3 / 6 parts 64 / 51 / 57 / 75 us;
// where pieces fill the places parts only cost: a chunk of 1200 tokens, 160 pieces,
// 1 / 2 / 3 parts 70 / 102 / 124 us, two head_dim 256 chunks, 156 pieces, 127 / 140 /
// 167 us).
// `beside`: another launch runs at the same time (shared prefixes: the sequences'
// own tokens), for which SMs are left: 1.25 CTAs an SM (64 chats over three prompts, 40
// pieces, 2 / 3 / 4 / 5 / 6 / 8 / 12 parts 71 / 55 / 46 / 47.5 / 51 / 47 / 45.6 us).
// The part count bounds what the kernel uses (it never makes parts of fewer than
// two tiles).  num_seqs > 0, so there is at least one piece.
int tile_splits(int D, int total_q, int num_seqs, int H_q, int H_kv, int sms,
                bool beside = false) {
  const int G = H_q / H_kv, teams = tile_teams(D, (long long)total_q * G, num_seqs, H_kv, sms);
  const long long places = (D < 256 && teams == 1 ? 2 : 1) * (long long)sms;
  const long long pieces = tile_bound(total_q, num_seqs, G, teams) * H_kv;
  if (pieces >= (beside ? sms : places)) return 1;
  const long long want = beside ? 5LL * sms / 4 : 7 * places / 4;
  const long long s = (want + pieces / 2) / pieces;
  return s > kMaxSplits ? kMaxSplits : (int)s;
}

// Workspace of the partial states: (m, l) of every part and row, then their o.
size_t tile_part_bytes(int D, int total_q, int H_q, int splits) {
  const size_t rows = (size_t)splits * total_q * H_q;
  return round_up(rows * 8, kWsAlign) + round_up(rows * D * 4, kWsAlign);
}

// Validates what the row-tile kernel's index arithmetic needs.
bool tile_sizes_ok(int total_q, int num_seqs, int H_q, int H_kv, int D) {
  return (long long)total_q * (H_q / H_kv) < 0x7ffffff0LL &&
         tile_bound(total_q, num_seqs, H_q / H_kv, 1) * H_kv < 0x7fffffffLL / kMaxSplits &&
         (long long)total_q * H_q * D < (1LL << 40);
}

int launch_tiles(int D, const TileParams& p, const void* k_cache, const void* v_cache,
                 cudaStream_t st) {
  CUtensorMap tk, tv;
  int rc = cached_map(k_cache, D, p.BS, p.H_kv, p.num_blocks, kMapHalf, &tk);
  if (rc != PAGED_ATTN_OK) return rc;
  rc = cached_map(v_cache, D, p.BS, p.H_kv, p.num_blocks, kMapHalf, &tv);
  if (rc != PAGED_ATTN_OK) return rc;
#ifdef PAGED_ATTN_WAIT_TEST
  (void)st;
  return cuda_fail(cudaErrorNotSupported);  // not in the test build
#else
  const cudaError_t e = D == 64    ? launch_tile_d64(tk, tv, p, st)
                        : D == 128 ? launch_tile_d128(tk, tv, p, st)
                                   : launch_tile_d256(tk, tv, p, st);
  return e == cudaSuccess ? PAGED_ATTN_OK : cuda_fail(e);
#endif
}

int launch_merge_parts(const MergeParams& p, cudaStream_t st) {
#ifdef PAGED_ATTN_WAIT_TEST
  (void)p, (void)st;
  return cuda_fail(cudaErrorNotSupported);
#else
  const cudaError_t e = launch_merge(p, st);
  return e == cudaSuccess ? PAGED_ATTN_OK : cuda_fail(e);
#endif
}

// The parameters common to both uses.
TileParams tile_params(int D, int sms, const void* q, void* out, const int32_t* bt, const int32_t* lens,
                       const int32_t* qo, int num_seqs, int total_q, int H_q, int H_kv, int maxb,
                       int BS, float scale, float softcap, const float* slopes) {
  TileParams t = {};
  t.q = static_cast<const __nv_bfloat16*>(q);
  t.out = static_cast<__nv_bfloat16*>(out);
  t.block_tables = bt;
  t.seq_lens = lens;
  t.qo_indptr = qo;
  t.num_seqs = num_seqs;
  t.total_q = total_q;
  t.H_q = H_q;
  t.H_kv = H_kv;
  t.G = H_q / H_kv;
  t.teams = tile_teams(D, (long long)total_q * t.G, num_seqs, H_kv, sms);
  t.maxb = maxb;
  t.BS = BS;
  t.scale_log2 = scale * 1.4426950408889634f;
  t.cap_log2 = softcap * 1.4426950408889634f;
  t.cap_in = softcap > 0.f ? scale / softcap : 0.f;
  t.slopes = slopes;
  t.num_blocks = g_check_blocks;
  return t;
}

void set_parts(TileParams* t, uint8_t* base) {
  const size_t rows = (size_t)t->splits * t->total_q * t->H_q;
  t->part_ml = reinterpret_cast<float2*>(base);
  t->part_o = reinterpret_cast<float*>(base + round_up(rows * 8, kWsAlign));
}

AppendParams append_params(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                           const int32_t* bt, const int32_t* sl, int num_seqs, int H_kv,
                           int head_dim, int max_blocks_per_seq, int block_size) {
  AppendParams a;
  a.k_new = static_cast<const __nv_bfloat16*>(k_new);
  a.v_new = static_cast<const __nv_bfloat16*>(v_new);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = nullptr;
  a.v_scale = nullptr;
  a.block_tables = bt;
  a.seq_lens = sl;
  a.qo_indptr = nullptr;
  a.num_seqs = num_seqs;
  a.total_q = 0;
  a.H_kv = H_kv;
  a.D = head_dim;
  a.maxb = max_blocks_per_seq;
  a.BS = block_size;
  a.num_blocks = g_check_blocks;
  a.status = g_check_blocks > 0 ? g_check_status : nullptr;
  return a;
}

int sms_of_device(int* sms) {
  DeviceInfo di;
  int rc = device_info(&di);
  if (rc == PAGED_ATTN_OK) *sms = di.sms;
  return rc;
}

int multi_checks(const void* q, const void* k_cache, const void* v_cache, const void* out,
                 const int32_t* qo_indptr, const int32_t* bt, const int32_t* sl, int num_seqs,
                 int total_q, int max_q_len, int H_q, int H_kv, int head_dim,
                 int max_blocks_per_seq, int block_size, float scale) {
  int rc = validate_sizes(num_seqs, H_q, H_kv, head_dim, max_blocks_per_seq, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  if (!std::isfinite(scale)) return PAGED_ATTN_ERR_SCALE;
  const int G = H_q / H_kv;
  if (total_q < 0 || max_q_len < 1 || (long long)max_q_len * G > kMaxMultiRows ||
      (long long)total_q * H_q * head_dim >= (1LL << 40))
    return PAGED_ATTN_ERR_SIZES;
  if (num_seqs == 0) return PAGED_ATTN_OK;
  rc = check_pointers(q, k_cache, v_cache, out, bt, sl);
  if (rc != PAGED_ATTN_OK) return rc;
  if (!aligned16(qo_indptr)) return PAGED_ATTN_ERR_POINTER;
  return PAGED_ATTN_OK;
}

int decode_multi_impl(const void* q, const void* k_cache, const void* v_cache, void* out,
                      const int32_t* qo_indptr, const int32_t* bt, const int32_t* sl,
                      int num_seqs, int total_q, int max_q_len, int H_q, int H_kv, int head_dim,
                      int max_blocks_per_seq, int block_size, float scale, int causal, bool early,
                      cudaStream_t st) {
  Operands o = operands(q, k_cache, v_cache, out, bt, sl, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.qo_indptr = qo_indptr;
  o.total_q = total_q;
  o.causal = causal ? 1 : 0;
  o.early = early;
  apply_checks(&o);
  // one n8 MMA tile of rows when a KV head's q_len * G rows fit, else pieces of 16
  const int G = H_q / H_kv;
  const int rows = max_q_len * G <= 8 ? 8 : 16;
  const int qchunks = (max_q_len * G + rows - 1) / rows;
  return plan_and_run(o, head_dim, block_size, false, false, rows, qchunks, st);
}

int fp8_checks(const void* q, const void* k8, const void* v8, const void* k_scale,
               const void* v_scale, const void* out, const int32_t* bt, const int32_t* sl,
               int num_seqs, int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
               int block_size, float scale) {
  int rc = common_checks(q, k8, v8, out, bt, sl, num_seqs, H_q, H_kv, head_dim,
                         max_blocks_per_seq, block_size, scale);
  if (rc != PAGED_ATTN_OK) return rc;
  if (head_dim == 64) return PAGED_ATTN_ERR_HEAD_DIM;  // FP8 pages need 128-byte rows
  if (num_seqs == 0) return PAGED_ATTN_OK;
  if (!aligned16(k_scale) || !aligned16(v_scale)) return PAGED_ATTN_ERR_POINTER;
  return PAGED_ATTN_OK;
}

}  // namespace
}  // namespace pagedattn

using namespace pagedattn;

extern "C" {

int paged_attn_decode(const void* q, const void* k_cache, const void* v_cache, void* out,
                      const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                      int H_q, int H_kv, int head_dim, int max_blocks_per_seq, int block_size,
                      float scale, void* stream) {
  int rc = common_checks(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                         head_dim, max_blocks_per_seq, block_size, scale);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.early = early_requested();
  apply_checks(&o);
  return plan_and_run(o, head_dim, block_size, false, false, 0, 0,
                      static_cast<cudaStream_t>(stream));
}

int paged_attn_decode_multi(const void* q, const void* k_cache, const void* v_cache, void* out,
                            const int32_t* qo_indptr, const int32_t* block_tables,
                            const int32_t* seq_lens, int num_seqs, int total_q, int max_q_len,
                            int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
                            int block_size, float scale, void* stream) {
  return paged_attn_decode_multi_ex(q, k_cache, v_cache, out, qo_indptr, block_tables, seq_lens,
                                    num_seqs, total_q, max_q_len, H_q, H_kv, head_dim,
                                    max_blocks_per_seq, block_size, scale, 1, stream);
}

int paged_attn_decode_multi_ex(const void* q, const void* k_cache, const void* v_cache,
                               void* out, const int32_t* qo_indptr, const int32_t* block_tables,
                               const int32_t* seq_lens, int num_seqs, int total_q, int max_q_len,
                               int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
                               int block_size, float scale, int is_causal, void* stream) {
  int rc = multi_checks(q, k_cache, v_cache, out, qo_indptr, block_tables, seq_lens, num_seqs,
                        total_q, max_q_len, H_q, H_kv, head_dim, max_blocks_per_seq, block_size,
                        scale);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  return decode_multi_impl(q, k_cache, v_cache, out, qo_indptr, block_tables, seq_lens, num_seqs,
                           total_q, max_q_len, H_q, H_kv, head_dim, max_blocks_per_seq,
                           block_size, scale, is_causal, early_requested(),
                           static_cast<cudaStream_t>(stream));
}

int paged_attn_decode_xpacked(const void* q, const void* k_cache, const void* v_cache, void* out,
                              const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                              int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
                              int block_size, float scale, void* stream) {
  int rc = common_checks(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                         head_dim, max_blocks_per_seq, block_size, scale);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.early = early_requested();
  apply_checks(&o);
  return plan_and_run(o, head_dim, block_size, false, true, 0, 0,
                      static_cast<cudaStream_t>(stream));
}

int paged_attn_decode_fp8(const void* q, const void* k_cache, const void* v_cache,
                          const float* k_scale, const float* v_scale, void* out,
                          const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                          int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
                          int block_size, float scale, void* stream) {
  int rc = fp8_checks(q, k_cache, v_cache, k_scale, v_scale, out, block_tables, seq_lens,
                      num_seqs, H_q, H_kv, head_dim, max_blocks_per_seq, block_size, scale);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.k_scale = k_scale;
  o.v_scale = v_scale;
  o.early = early_requested();
  apply_checks(&o);
  return plan_and_run(o, head_dim, block_size, true, false, 0, 0,
                      static_cast<cudaStream_t>(stream));
}

int paged_attn_append_decode(const void* q, const void* k_new, const void* v_new, void* k_cache,
                             void* v_cache, void* out, const int32_t* block_tables,
                             const int32_t* seq_lens, int num_seqs, int H_q, int H_kv,
                             int head_dim, int max_blocks_per_seq, int block_size, float scale,
                             void* stream) {
  int rc = common_checks(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                         head_dim, max_blocks_per_seq, block_size, scale);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  if (!aligned16(k_new) || !aligned16(v_new)) return PAGED_ATTN_ERR_POINTER;
  int dev = 0;
  DeviceInfo di;
  if ((rc = device_info(&di, &dev)) != PAGED_ATTN_OK) return rc;
  Plan pl;
  if ((rc = cached_plan(num_seqs, H_q, H_kv, head_dim, block_size, dev, di, &pl)) !=
      PAGED_ATTN_OK)
    return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  apply_checks(&o);
  WorkspaceHold hold;
  if ((rc = owned_workspace(pl.ws_bytes, st, &o.ws, &hold)) != PAGED_ATTN_OK) return rc;
  // Fused, the warp that reads a piece's last page patches the new rows into it,
  // a small cost per piece on that CTA's path.  When CTAs average kAppendApartPieces
  // or more (s, g) pieces, the CTA crossing the most short sequences sets the
  // kernel's end and a separate append launch ahead of the decode is cheaper
  // (ragged 256-sequence batch: decode 619 us, fused 630, apart 622; LLaMA-shaped
  // batch: decode 51.3, fused 51.6, apart 53.4).  Both give the same bits.
  if ((long long)num_seqs * H_kv >= (long long)kAppendApartPieces * pl.grid) {
    AppendParams a = append_params(k_new, v_new, k_cache, v_cache, block_tables, seq_lens,
                                   num_seqs, H_kv, head_dim, max_blocks_per_seq, block_size);
    cudaError_t e = launch_append(a, di.sms, st);
    if (e != cudaSuccess) return cuda_fail(e);
    // The append just written is what the decode's producer reads first: the
    // decode waits for it before any global access (no early prologue).
    o.early = false;
    return run(pl, o, st);
  }
  // Fused: the new rows are patched into the pages in shared memory, whatever
  // the producer's copy brought, so the early prologue stays as requested.
  o.early = early_requested();
  o.k_new = k_new;
  o.v_new = v_new;
  return run(pl, o, st);
}

int paged_kv_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                    const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int H_kv,
                    int head_dim, int max_blocks_per_seq, int block_size, void* stream) {
  // the decode's size rules with a one-head query group
  int rc = validate_sizes(num_seqs, H_kv, H_kv, head_dim, max_blocks_per_seq, block_size);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(block_tables) || !aligned16(seq_lens))
    return PAGED_ATTN_ERR_POINTER;
  int sms = 0;
  if ((rc = sms_of_device(&sms)) != PAGED_ATTN_OK) return rc;
  AppendParams a = append_params(k_new, v_new, k_cache, v_cache, block_tables, seq_lens, num_seqs,
                                 H_kv, head_dim, max_blocks_per_seq, block_size);
  cudaError_t e = launch_append(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PAGED_ATTN_OK : cuda_fail(e);
}

int paged_kv_append_multi(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                          const int32_t* qo_indptr, const int32_t* block_tables,
                          const int32_t* seq_lens, int num_seqs, int total_q, int H_kv,
                          int head_dim, int max_blocks_per_seq, int block_size, void* stream) {
  int rc = validate_sizes(num_seqs, H_kv, H_kv, head_dim, max_blocks_per_seq, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  if (total_q < 0 || (long long)total_q * H_kv * head_dim >= (1LL << 40))
    return PAGED_ATTN_ERR_SIZES;
  if (num_seqs == 0 || total_q == 0) return PAGED_ATTN_OK;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(qo_indptr) || !aligned16(block_tables) || !aligned16(seq_lens))
    return PAGED_ATTN_ERR_POINTER;
  int sms = 0;
  if ((rc = sms_of_device(&sms)) != PAGED_ATTN_OK) return rc;
  AppendParams a = append_params(k_new, v_new, k_cache, v_cache, block_tables, seq_lens, num_seqs,
                                 H_kv, head_dim, max_blocks_per_seq, block_size);
  a.qo_indptr = qo_indptr;
  a.total_q = total_q;
  cudaError_t e = launch_append(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PAGED_ATTN_OK : cuda_fail(e);
}

int paged_attn_append_decode_multi(const void* q, const void* k_new, const void* v_new,
                                   void* k_cache, void* v_cache, void* out,
                                   const int32_t* qo_indptr, const int32_t* block_tables,
                                   const int32_t* seq_lens, int num_seqs, int total_q,
                                   int max_q_len, int H_q, int H_kv, int head_dim,
                                   int max_blocks_per_seq, int block_size, float scale,
                                   int is_causal, void* stream) {
  int rc = multi_checks(q, k_cache, v_cache, out, qo_indptr, block_tables, seq_lens, num_seqs,
                        total_q, max_q_len, H_q, H_kv, head_dim, max_blocks_per_seq, block_size,
                        scale);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  if (!aligned16(k_new) || !aligned16(v_new)) return PAGED_ATTN_ERR_POINTER;
  int sms = 0;
  if ((rc = sms_of_device(&sms)) != PAGED_ATTN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (total_q > 0) {
    AppendParams a = append_params(k_new, v_new, k_cache, v_cache, block_tables, seq_lens,
                                   num_seqs, H_kv, head_dim, max_blocks_per_seq, block_size);
    a.qo_indptr = qo_indptr;
    a.total_q = total_q;
    cudaError_t e = launch_append(a, sms, st);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  // the decode reads the rows just appended: plain launch (no early prologue)
  return decode_multi_impl(q, k_cache, v_cache, out, qo_indptr, block_tables, seq_lens, num_seqs,
                           total_q, max_q_len, H_q, H_kv, head_dim, max_blocks_per_seq,
                           block_size, scale, is_causal, false, st);
}

int paged_kv_append_fp8(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                        float* k_scale, float* v_scale, const int32_t* block_tables,
                        const int32_t* seq_lens, int num_seqs, int H_kv, int head_dim,
                        int max_blocks_per_seq, int block_size, void* stream) {
  int rc = validate_sizes(num_seqs, H_kv, H_kv, head_dim, max_blocks_per_seq, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  if (head_dim == 64) return PAGED_ATTN_ERR_HEAD_DIM;  // as the FP8 decode
  if (num_seqs == 0) return PAGED_ATTN_OK;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(k_scale) || !aligned16(v_scale) || !aligned16(block_tables) ||
      !aligned16(seq_lens))
    return PAGED_ATTN_ERR_POINTER;
  int sms = 0;
  if ((rc = sms_of_device(&sms)) != PAGED_ATTN_OK) return rc;
  AppendParams a = append_params(k_new, v_new, k_cache, v_cache, block_tables, seq_lens, num_seqs,
                                 H_kv, head_dim, max_blocks_per_seq, block_size);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  cudaError_t e = launch_append_fp8(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PAGED_ATTN_OK : cuda_fail(e);
}

int paged_attn_append_decode_fp8(const void* q, const void* k_new, const void* v_new,
                                 void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                 void* out, const int32_t* block_tables, const int32_t* seq_lens,
                                 int num_seqs, int H_q, int H_kv, int head_dim,
                                 int max_blocks_per_seq, int block_size, float scale,
                                 void* stream) {
  int rc = fp8_checks(q, k_cache, v_cache, k_scale, v_scale, out, block_tables, seq_lens,
                      num_seqs, H_q, H_kv, head_dim, max_blocks_per_seq, block_size, scale);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  if (!aligned16(k_new) || !aligned16(v_new)) return PAGED_ATTN_ERR_POINTER;
  int dev = 0;
  DeviceInfo di;
  if ((rc = device_info(&di, &dev)) != PAGED_ATTN_OK) return rc;
  Plan pl;
  if ((rc = cached_plan(num_seqs, H_q, H_kv, head_dim, block_size, dev, di, &pl, true)) !=
      PAGED_ATTN_OK)
    return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.k_scale = k_scale;
  o.v_scale = v_scale;
  apply_checks(&o);
  WorkspaceHold hold;
  if ((rc = owned_workspace(pl.ws_bytes, st, &o.ws, &hold)) != PAGED_ATTN_OK) return rc;
  // As for bf16 caches: fused (each piece's last page quantized and patched in
  // shared memory, then stored) unless CTAs average kAppendApartPieces or more
  // pieces, when the append runs as its own launch and the decode after it is
  // a plain launch.
  // The fused form is compiled for head_dim 128 only (at 256 its code would cost
  // the page loop a register spill).
  if (head_dim != 128 ||
      (long long)num_seqs * H_kv >= (long long)kAppendApartPieces * pl.grid) {
    AppendParams a = append_params(k_new, v_new, k_cache, v_cache, block_tables, seq_lens,
                                   num_seqs, H_kv, head_dim, max_blocks_per_seq, block_size);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    cudaError_t e = launch_append_fp8(a, di.sms, st);
    if (e != cudaSuccess) return cuda_fail(e);
    o.early = false;  // the decode reads the rows just appended
    return run(pl, o, st);
  }
  o.early = early_requested();
  o.k_new = k_new;
  o.v_new = v_new;
  return run(pl, o, st);
}

int paged_attn_decode_mods(const void* q, const void* k_cache, const void* v_cache, void* out,
                           const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                           int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
                           int block_size, float scale, float softcap,
                           const float* alibi_slopes, int window, const int32_t* prefix_lens,
                           const int32_t* doc_starts, void* workspace, size_t workspace_bytes,
                           void* stream) {
  int rc = common_checks(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                         head_dim, max_blocks_per_seq, block_size, scale);
  if (rc == PAGED_ATTN_OK)
    rc = mods_checks(scale, (long long)max_blocks_per_seq * block_size, softcap, alibi_slopes,
                     window, prefix_lens, doc_starts);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.softcap = softcap;
  o.slopes = alibi_slopes;
  o.window = window;
  o.prefix_lens = prefix_lens;
  o.doc_starts = doc_starts;
  return decode_mods_impl(o, head_dim, block_size, false, workspace, workspace_bytes,
                          static_cast<cudaStream_t>(stream));
}

int paged_attn_decode_fp8_mods(const void* q, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, void* out,
                               const int32_t* block_tables, const int32_t* seq_lens,
                               int num_seqs, int H_q, int H_kv, int head_dim,
                               int max_blocks_per_seq, int block_size, float scale, float softcap,
                               const float* alibi_slopes, int window, const int32_t* prefix_lens,
                               const int32_t* doc_starts, void* workspace, size_t workspace_bytes,
                               void* stream) {
  int rc = fp8_checks(q, k_cache, v_cache, k_scale, v_scale, out, block_tables, seq_lens,
                      num_seqs, H_q, H_kv, head_dim, max_blocks_per_seq, block_size, scale);
  if (rc == PAGED_ATTN_OK)
    rc = mods_checks(scale, (long long)max_blocks_per_seq * block_size, softcap, alibi_slopes,
                     window, prefix_lens, doc_starts);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.k_scale = k_scale;
  o.v_scale = v_scale;
  o.softcap = softcap;
  o.slopes = alibi_slopes;
  o.window = window;
  o.prefix_lens = prefix_lens;
  o.doc_starts = doc_starts;
  return decode_mods_impl(o, head_dim, block_size, true, workspace, workspace_bytes,
                          static_cast<cudaStream_t>(stream));
}

size_t paged_attn_multi_mods_workspace_bytes(int num_seqs, int total_q, int H_q, int H_kv,
                                             int head_dim, int max_blocks_per_seq,
                                             int block_size) {
  if (validate_sizes(num_seqs, H_q, H_kv, head_dim, max_blocks_per_seq, block_size) !=
          PAGED_ATTN_OK ||
      total_q < 0 || !tile_sizes_ok(total_q, num_seqs, H_q, H_kv, head_dim))
    return 0;
  DeviceInfo di;
  if (device_info(&di) != PAGED_ATTN_OK) return 0;
  if (num_seqs == 0 || total_q == 0) return counters_end(di);
  const int splits = tile_splits(head_dim, total_q, num_seqs, H_q, H_kv, di.sms);
  return counters_end(di) + (splits > 1 ? tile_part_bytes(head_dim, total_q, H_q, splits) : 0);
}

int paged_attn_decode_multi_mods(const void* q, const void* k_cache, const void* v_cache,
                                 void* out, const int32_t* qo_indptr,
                                 const int32_t* block_tables, const int32_t* seq_lens,
                                 int num_seqs, int total_q, int H_q, int H_kv, int head_dim,
                                 int max_blocks_per_seq, int block_size, float scale,
                                 int is_causal, float softcap, const float* alibi_slopes,
                                 int window, const int32_t* prefix_lens,
                                 const int32_t* doc_starts, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  int rc = validate_sizes(num_seqs, H_q, H_kv, head_dim, max_blocks_per_seq, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  if (!std::isfinite(scale)) return PAGED_ATTN_ERR_SCALE;
  if (total_q < 0 || !tile_sizes_ok(total_q, num_seqs, H_q, H_kv, head_dim))
    return PAGED_ATTN_ERR_SIZES;
  rc = mods_checks(scale, (long long)max_blocks_per_seq * block_size, softcap, alibi_slopes,
                   window, prefix_lens, doc_starts);
  if (rc != PAGED_ATTN_OK || num_seqs == 0 || total_q == 0) return rc;
  rc = check_pointers(q, k_cache, v_cache, out, block_tables, seq_lens);
  if (rc != PAGED_ATTN_OK) return rc;
  if (!aligned16(qo_indptr)) return PAGED_ATTN_ERR_POINTER;
  DeviceInfo di;
  if ((rc = device_info(&di)) != PAGED_ATTN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TileParams t = tile_params(head_dim, di.sms, q, out, block_tables, seq_lens, qo_indptr, num_seqs, total_q, H_q,
                             H_kv, max_blocks_per_seq, block_size, scale, softcap, alibi_slopes);
  t.causal = is_causal ? 1 : 0;
  t.window = window;
  t.prefix_lens = prefix_lens;
  t.doc_starts = doc_starts;
  t.splits = tile_splits(head_dim, total_q, num_seqs, H_q, H_kv, di.sms);
  t.single = t.splits == 1 ? 1 : 0;
  const size_t parts = t.single ? 0 : tile_part_bytes(head_dim, total_q, H_q, t.splits);
  void* ws = nullptr;
  WorkspaceHold hold;
  rc = optional_workspace(workspace, workspace_bytes, counters_end(di) + parts, st, &ws, &hold);
  if (rc != PAGED_ATTN_OK) return rc;
  t.status = g_check_blocks > 0 ? g_check_status : static_cast<int32_t*>(ws);
  if (!t.single) set_parts(&t, static_cast<uint8_t*>(ws) + counters_end(di));
  if ((rc = launch_tiles(head_dim, t, k_cache, v_cache, st)) != PAGED_ATTN_OK) return rc;
  if (t.single) return PAGED_ATTN_OK;
  MergeParams m = {};
  m.part_o = t.part_o;
  m.part_ml = t.part_ml;
  m.splits = t.splits;
  m.qo_indptr = qo_indptr;
  m.num_seqs = num_seqs;
  m.total_q = total_q;
  m.H_q = H_q;
  m.D = head_dim;
  m.out = t.out;
  return launch_merge_parts(m, st);
}

// Shared prefixes: the rows of a group's members over its prefix (row tiles),
// every sequence's own tokens (the decode kernel, its states as the output), then
// the merge of both.
namespace {
struct SharedPlan {
  Plan own;          // the decode over the sequences' own tokens
  int splits;        // parts of a prefix
  size_t off_state, off_parts, bytes;
};

int shared_plan(int num_seqs, int num_groups, int H_q, int H_kv, int head_dim, int block_size,
                SharedPlan* sp) {
  int dev = 0;
  DeviceInfo di;
  int rc = device_info(&di, &dev);
  if (rc != PAGED_ATTN_OK) return rc;
  rc = cached_plan(num_seqs, H_q, H_kv, head_dim, block_size, dev, di, &sp->own, false, 0, 0,
                   true);
  if (rc != PAGED_ATTN_OK) return rc;
  if (num_groups == 0) {  // the decode alone: no pieces, no states to merge
    sp->splits = 0;
    sp->off_state = sp->off_parts = sp->bytes = sp->own.ws_bytes;
    return PAGED_ATTN_OK;
  }
  sp->splits = tile_splits(head_dim, num_seqs, num_groups, H_q, H_kv, di.sms, true);
  sp->off_state = round_up(sp->own.ws_bytes, kWsAlign);
  sp->off_parts =
      sp->off_state + round_up((size_t)num_seqs * H_q * (head_dim + 4) * 4, kWsAlign);
  sp->bytes = sp->off_parts + tile_part_bytes(head_dim, num_seqs, H_q, sp->splits);
  return PAGED_ATTN_OK;
}

int shared_sizes(int num_seqs, int num_groups, int H_q, int H_kv, int head_dim,
                 int max_blocks_per_seq, int prefix_max_blocks, int block_size) {
  int rc = validate_sizes(num_seqs, H_q, H_kv, head_dim, max_blocks_per_seq, block_size);
  if (rc == PAGED_ATTN_OK)
    rc = validate_sizes(num_groups, H_q, H_kv, head_dim, prefix_max_blocks, block_size);
  if (rc == PAGED_ATTN_OK && !tile_sizes_ok(num_seqs, num_groups, H_q, H_kv, head_dim))
    rc = PAGED_ATTN_ERR_SIZES;
  return rc;
}
}  // namespace

size_t paged_attn_shared_workspace_bytes(int num_seqs, int num_groups, int H_q, int H_kv,
                                         int head_dim, int max_blocks_per_seq, int block_size) {
  if (shared_sizes(num_seqs, num_groups, H_q, H_kv, head_dim, max_blocks_per_seq, 1,
                   block_size) != PAGED_ATTN_OK)
    return 0;
  SharedPlan sp;
  return shared_plan(num_seqs, num_groups, H_q, H_kv, head_dim, block_size, &sp) == PAGED_ATTN_OK
             ? sp.bytes
             : 0;
}

int paged_attn_decode_shared(const void* q, const void* k_cache, const void* v_cache, void* out,
                             const int32_t* group_indptr, const int32_t* prefix_tables,
                             const int32_t* prefix_lens, int num_groups, int prefix_max_blocks,
                             const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                             int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
                             int block_size, float scale, float softcap,
                             const float* alibi_slopes, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int rc = shared_sizes(num_seqs, num_groups, H_q, H_kv, head_dim, max_blocks_per_seq,
                        prefix_max_blocks, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  if (!std::isfinite(scale)) return PAGED_ATTN_ERR_SCALE;
  const int most_blocks =
      max_blocks_per_seq > prefix_max_blocks ? max_blocks_per_seq : prefix_max_blocks;
  rc = mods_checks(scale, (long long)most_blocks * block_size, softcap, alibi_slopes, 0, nullptr,
                   nullptr);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  rc = check_pointers(q, k_cache, v_cache, out, block_tables, seq_lens);
  if (rc != PAGED_ATTN_OK) return rc;
  if (num_groups > 0 &&
      (!aligned16(group_indptr) || !aligned16(prefix_tables) || !aligned16(prefix_lens)))
    return PAGED_ATTN_ERR_POINTER;
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.softcap = softcap;
  o.slopes = alibi_slopes;
  if (num_groups == 0)
    return decode_mods_impl(o, head_dim, block_size, false, workspace, workspace_bytes,
                            static_cast<cudaStream_t>(stream));
  SharedPlan sp;
  rc = shared_plan(num_seqs, num_groups, H_q, H_kv, head_dim, block_size, &sp);
  if (rc != PAGED_ATTN_OK) return rc;
  DeviceInfo di;
  if ((rc = device_info(&di)) != PAGED_ATTN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  WorkspaceHold hold;
  rc = optional_workspace(workspace, workspace_bytes, sp.bytes, st, &o.ws, &hold);
  if (rc != PAGED_ATTN_OK) return rc;
  apply_checks(&o);
  uint8_t* base = static_cast<uint8_t*>(o.ws);
  TileParams t = tile_params(head_dim, di.sms, q, out, prefix_tables, prefix_lens, group_indptr, num_groups,
                             num_seqs, H_q, H_kv, prefix_max_blocks, block_size, scale, softcap,
                             alibi_slopes);
  t.tail_lens = seq_lens;
  t.tail_cap = max_blocks_per_seq * block_size;
  t.splits = sp.splits;
  t.status = o.status ? o.status : static_cast<int32_t*>(o.ws);
  set_parts(&t, base + sp.off_parts);
  if ((rc = launch_tiles(head_dim, t, k_cache, v_cache, st)) != PAGED_ATTN_OK) return rc;
  // The two passes over keys need nothing of each other and run side by side.
  o.independent = true;
  o.state = reinterpret_cast<float*>(base + sp.off_state);
  if ((rc = run(sp.own, o, st)) != PAGED_ATTN_OK) return rc;
  MergeParams m = {};
  m.part_o = t.part_o;
  m.part_ml = t.part_ml;
  m.splits = t.splits;
  m.qo_indptr = group_indptr;
  m.num_seqs = num_groups;
  m.total_q = num_seqs;
  m.H_q = H_q;
  m.D = head_dim;
  m.state = o.state;
  m.out = t.out;
  return launch_merge_parts(m, st);
}

size_t paged_attn_mods_workspace_bytes(int num_seqs, int H_q, int H_kv, int head_dim,
                                       int max_blocks_per_seq, int block_size) {
  if (validate_sizes(num_seqs, H_q, H_kv, head_dim, max_blocks_per_seq, block_size) !=
      PAGED_ATTN_OK)
    return 0;
  int dev = 0;
  DeviceInfo di;
  if (device_info(&di, &dev) != PAGED_ATTN_OK) return 0;
  size_t bytes = 0;
  for (int fp8 = 0; fp8 <= (head_dim == 64 ? 0 : 1); ++fp8) {
    Plan pl;
    if (cached_plan(num_seqs, H_q, H_kv, head_dim, block_size, dev, di, &pl, fp8 != 0, 0, 0,
                    true) != PAGED_ATTN_OK)
      return 0;
    if (pl.ws_bytes > bytes) bytes = pl.ws_bytes;
  }
  return bytes;
}

int paged_kv_assign(const int32_t* seq_lens, const int32_t* new_lens, int32_t* block_tables,
                    const int32_t* free_blocks, const int32_t* free_count, int32_t* seq_lens_out,
                    int32_t* qo_indptr, int64_t* slot_map, int32_t* free_count_out,
                    int32_t* refused, int num_seqs, int max_blocks_per_seq, int block_size,
                    int free_capacity, int max_new, void* stream) {
  int rc = validate_sizes(num_seqs, 1, 1, 64, max_blocks_per_seq, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  if (free_capacity < 0 || max_new < 0) return PAGED_ATTN_ERR_SIZES;
  // What a launch without sequences, new rows or free blocks never touches may be null.
  // (Without sequences there still are the padding slots and the counts to write.)
  if ((num_seqs > 0 && (!aligned16(seq_lens) || !aligned16(new_lens) ||
                        !aligned16(block_tables) || !aligned16(seq_lens_out))) ||
      !aligned16(qo_indptr) || free_count == nullptr ||
      !aligned4(free_count) || free_count_out == nullptr || !aligned4(free_count_out) ||
      !aligned4(refused) || (max_new > 0 && !aligned16(slot_map)) ||
      (free_capacity > 0 && !aligned16(free_blocks)))
    return PAGED_ATTN_ERR_POINTER;
  AssignParams a;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.block_tables = block_tables;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.seq_lens_out = seq_lens_out;
  a.qo_indptr = qo_indptr;
  a.slot_map = slot_map;
  a.free_count_out = free_count_out;
  a.refused = refused;
  a.num_seqs = num_seqs;
  a.maxb = max_blocks_per_seq;
  a.BS = block_size;
  a.free_capacity = free_capacity;
  a.max_new = max_new;
  a.num_blocks = g_check_blocks;
  a.status = g_check_blocks > 0 ? g_check_status : nullptr;
  cudaError_t e = launch_assign(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PAGED_ATTN_OK : cuda_fail(e);
}

int paged_kv_append_slots(const void* k_new, const void* v_new, long long k_stride,
                          long long v_stride, void* k_cache, void* v_cache,
                          const int64_t* slot_map, int rows, int H_kv, int head_dim,
                          int block_size, long long num_blocks, void* stream) {
  int rc = validate_sizes(0, H_kv, H_kv, head_dim, 1, block_size);
  if (rc != PAGED_ATTN_OK) return rc;
  const long long row = (long long)H_kv * head_dim;
  if (rows < 0 || num_blocks < 1 || num_blocks > 0x7fffffffLL || k_stride < row ||
      v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return PAGED_ATTN_ERR_SIZES;
  if (rows == 0) return PAGED_ATTN_OK;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(slot_map))
    return PAGED_ATTN_ERR_POINTER;
  int sms = 0;
  if ((rc = sms_of_device(&sms)) != PAGED_ATTN_OK) return rc;
  AppendSlotsParams a;
  a.k_new = static_cast<const __nv_bfloat16*>(k_new);
  a.v_new = static_cast<const __nv_bfloat16*>(v_new);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  a.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  a.slot_map = slot_map;
  a.rows = rows;
  a.H_kv = H_kv;
  a.D = head_dim;
  a.BS = block_size;
  a.num_blocks = num_blocks;
  a.status = g_check_blocks > 0 ? g_check_status : nullptr;
  cudaError_t e = launch_append_slots(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PAGED_ATTN_OK : cuda_fail(e);
}

size_t paged_attn_workspace_bytes(int num_seqs, int H_q, int H_kv, int head_dim,
                                  int max_blocks_per_seq, int block_size) {
  if (validate_sizes(num_seqs, H_q, H_kv, head_dim, max_blocks_per_seq, block_size) !=
      PAGED_ATTN_OK)
    return 0;
  int dev = 0;
  DeviceInfo di;
  if (device_info(&di, &dev) != PAGED_ATTN_OK) return 0;
  Plan pl;
  if (cached_plan(num_seqs, H_q, H_kv, head_dim, block_size, dev, di, &pl) != PAGED_ATTN_OK)
    return 0;
  return pl.ws_bytes;
}

int paged_attn_decode_ws(const void* q, const void* k_cache, const void* v_cache, void* out,
                         const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                         int H_q, int H_kv, int head_dim, int max_blocks_per_seq, int block_size,
                         float scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = common_checks(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                         head_dim, max_blocks_per_seq, block_size, scale);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) != 0)
    return PAGED_ATTN_ERR_WORKSPACE;
  int dev = 0;
  DeviceInfo di;
  if ((rc = device_info(&di, &dev)) != PAGED_ATTN_OK) return rc;
  Plan pl;
  if ((rc = cached_plan(num_seqs, H_q, H_kv, head_dim, block_size, dev, di, &pl)) !=
      PAGED_ATTN_OK)
    return rc;
  if (workspace_bytes < pl.ws_bytes) return PAGED_ATTN_ERR_WORKSPACE;
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.ws = workspace;
  o.early = early_requested();
  apply_checks(&o);
  return run(pl, o, static_cast<cudaStream_t>(stream));
}

int paged_attn_decode_checked(const void* q, const void* k_cache, const void* v_cache, void* out,
                              const int32_t* block_tables, const int32_t* seq_lens,
                              int num_seqs, int H_q, int H_kv, int head_dim,
                              int max_blocks_per_seq, int block_size, float scale,
                              long long num_blocks, int32_t* d_status, void* stream) {
  int rc = common_checks(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                         head_dim, max_blocks_per_seq, block_size, scale);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  if (num_blocks <= 0 || num_blocks > 0x7fffffffLL) return PAGED_ATTN_ERR_SIZES;
  if (d_status == nullptr || (reinterpret_cast<uintptr_t>(d_status) & 3) != 0)
    return PAGED_ATTN_ERR_POINTER;
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.num_blocks = num_blocks;
  o.status = d_status;
  o.early = early_requested();
  return plan_and_run(o, head_dim, block_size, false, false, 0, 0,
                      static_cast<cudaStream_t>(stream));
}

int paged_attn_decode_static(const void* q, const void* k_cache, const void* v_cache, void* out,
                             const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                             int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
                             int block_size, float scale, void* stream) {
  int rc = common_checks(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                         head_dim, max_blocks_per_seq, block_size, scale);
  if (rc != PAGED_ATTN_OK || num_seqs == 0) return rc;
  int dev = 0;
  DeviceInfo di;
  if ((rc = device_info(&di, &dev)) != PAGED_ATTN_OK) return rc;
  Plan pl;
  if ((rc = cached_plan(num_seqs, H_q, H_kv, head_dim, block_size, dev, di, &pl)) !=
      PAGED_ATTN_OK)
    return rc;
  if (pl.ws_bytes > kStaticScratchBytes) return PAGED_ATTN_ERR_STATIC_SCRATCH;
  void* ws = nullptr;
  if ((rc = static_scratch_address(&ws)) != PAGED_ATTN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // The array keeps whatever the previous call left; the status word and the
  // combine counters must start at zero.  The memset is a plain stream
  // operation ahead of the launch, which then waits for it before touching the
  // array (the early prologue only reads the caller's tables and caches early).
  cudaError_t e = cudaMemsetAsync(ws, 0, pl.off_partials, st);
  if (e != cudaSuccess) return cuda_fail(e);
  Operands o = operands(q, k_cache, v_cache, out, block_tables, seq_lens, num_seqs, H_q, H_kv,
                        max_blocks_per_seq, scale);
  o.ws = ws;
  o.early = early_requested();
  apply_checks(&o);
  return run(pl, o, st);
}

const char* paged_attn_status_string(int status) {
  switch (status) {
    case PAGED_ATTN_OK: return "ok";
    case PAGED_ATTN_ERR_POINTER: return "null or misaligned pointer";
    case PAGED_ATTN_ERR_HEADS: return "H_q must be a positive multiple of H_kv with H_q/H_kv <= 16";
    case PAGED_ATTN_ERR_HEAD_DIM: return "head_dim must be 64, 128 or 256";
    case PAGED_ATTN_ERR_BLOCK_SIZE: return "block_size must be 16 or 32";
    case PAGED_ATTN_ERR_SIZES: return "num_seqs, max_blocks_per_seq or num_blocks out of range";
    case PAGED_ATTN_ERR_CUDA: return "CUDA call failed (see paged_attn_last_cuda_error)";
    case PAGED_ATTN_ERR_WORKSPACE: return "workspace null, misaligned or too small";
    case PAGED_ATTN_ERR_SCALE: return "scale is not finite";
    case PAGED_ATTN_ERR_STATIC_SCRATCH:
      return "sizes need more scratch than paged_attn_decode_static's fixed 4 MiB array";
    case PAGED_ATTN_ERR_FLAGS: return "unknown launch flag bits";
    case PAGED_ATTN_ERR_MODS: return "softcap must be 0 or in [1e-30, 1e30], window >= 0";
    default: return "unknown status";
  }
}

int paged_attn_set_launch_flags(int flags) {
  if (flags & ~PAGED_ATTN_FLAG_EARLY_PROLOGUE) return PAGED_ATTN_ERR_FLAGS;
  g_launch_flags = flags;
  return PAGED_ATTN_OK;
}

int paged_attn_set_checks(long long num_blocks, int32_t* d_status) {
  if (num_blocks <= 0 && d_status == nullptr) {
    g_check_blocks = 0;
    g_check_status = nullptr;
    return PAGED_ATTN_OK;
  }
  if (num_blocks <= 0 || num_blocks > 0x7fffffffLL) return PAGED_ATTN_ERR_SIZES;
  if (d_status == nullptr || (reinterpret_cast<uintptr_t>(d_status) & 3) != 0)
    return PAGED_ATTN_ERR_POINTER;
  g_check_blocks = num_blocks;
  g_check_status = d_status;
  return PAGED_ATTN_OK;
}

int paged_attn_reset_workspace(void* stream) {
  int dev = 0;
  int rc = current_device(&dev);
  if (rc != PAGED_ATTN_OK) return rc;
  std::lock_guard<std::mutex> lk(g_ws_mu);
  auto zero = [&](const OwnedWorkspace& w) -> int {
    if (w.ptr == nullptr) return PAGED_ATTN_OK;
    cudaError_t e = cudaMemsetAsync(w.ptr, 0, w.bytes, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PAGED_ATTN_OK : cuda_fail(e);
  };
  rc = zero(g_ws[dev]);
  for (int k = 0; k < g_opt_ws[dev].count && rc == PAGED_ATTN_OK; ++k)
    rc = zero(g_opt_ws[dev].entry[k].w);
  return rc;
}

int paged_attn_last_cuda_error(void) { return g_last_cuda_error; }

int paged_attn_version(void) { return 300; }

#ifdef PAGED_ATTN_WAIT_TEST
// Test build only (not in include/paged_attn.h): the next decode launches of
// this thread leave unit `skip_unit` of CTA 0's range without a copy (-1: off)
// and, with skip_publish != 0, make every combiner wait for one more published
// part than exists, so the bounded waits run out.
__attribute__((visibility("default"))) int paged_attn_test_set_wait_faults(int skip_unit,
                                                                           int skip_publish) {
  g_test_skip_unit = skip_unit;
  g_test_skip_publish = skip_publish;
  return PAGED_ATTN_OK;
}
#endif

}  // extern "C"
