/*
 * paged_attn.h -- C ABI of the GB300 (sm_103a) paged-KV GQA decode attention library.
 *
 * The operation (every entry point below computes it):
 *
 *   "Paged Attention Kernel Architecture for BI-V100", section 1 (Problem
 *   Definition): for one new query token per sequence,
 *       out[s, h, :] = softmax_t( scale * q[s, h, :] . K_t ) . V_t,   t < seq_lens[s],
 *   where K_t / V_t are rows of a paged cache reached through a block table.
 *   Layout, length meaning and GQA head map follow the "Add Cuda Kernel"
 *   tutorial (RL.cu), include/kernels/attention.cuh, "Paged Attention - Decode":
 *       K_t = k_cache[block_tables[s, t / block_size], g, t % block_size, :]
 *       g   = h * H_kv / H_q          (H_q must be a multiple of H_kv; G = H_q / H_kv)
 *   The caller passes `scale` (the tutorial's launcher recomputed 1/sqrt(head_dim)
 *   and ignored its argument; here the argument is used as given).
 *
 * Tensors (DEVICE-ADDRESSABLE pointers, owned by the caller, densely packed
 * row-major, base addresses 16-byte aligned).  The caches (and their row floats)
 * must be device memory.  Every other tensor -- q, out, block_tables, seq_lens,
 * qo_indptr, the new K/V rows of the appends, status words -- may also be
 * pinned host memory (cudaMallocHost / cudaHostAlloc, which unified addressing
 * makes directly addressable from the device): the kernels then read and write
 * it over the host link (NVLink-C2C on GB300) inside the call, with no separate
 * copy, and the results are the same bits.  The library never dereferences any
 * of these pointers on the host.
 *   q            [num_seqs, H_q, head_dim]                      bf16   (read)
 *   k_cache      [num_blocks, H_kv, block_size, head_dim]       bf16   (read)
 *   v_cache      [num_blocks, H_kv, block_size, head_dim]       bf16   (read)
 *   out          [num_seqs, H_q, head_dim]                      bf16   (written)
 *   block_tables [num_seqs, max_blocks_per_seq]                 int32  (read)
 *   seq_lens     [num_seqs]                                     int32  (read)
 *
 * seq_lens[s] is the number of cached tokens the query attends to (the new
 * token's K/V must already be in the cache).  A length of 0 writes a zero row.
 * Lengths are clamped to [0, max_blocks_per_seq * block_size].  Only the
 * first ceil(seq_lens[s] / block_size) entries of a block-table row are read,
 * and only the rows t < seq_lens[s] of those blocks: slots past the end may
 * hold anything, NaN included.
 *
 * Supported: head_dim in {64, 128, 256}; block_size in {16, 32}; 1 <= G <= 16;
 * num_seqs >= 0 (0 is a no-op).  Arithmetic: bf16 inputs, fp32 accumulation
 * (tensor-core products of bf16 operands), bf16 output rounded to nearest even.
 *
 * Execution: every call is asynchronous on `stream` (a cudaStream_t; NULL is
 * the legacy default stream), never synchronises, and never allocates except
 * where an entry point says so.  Block ids outside the caller's pool are not
 * detected unless checks are on: paged_attn_decode_checked checks its own
 * call, and paged_attn_set_checks turns the same checks on for every later
 * call of the calling thread (all decode and append entry points).
 *
 * Errors: every entry point returns PAGED_ATTN_OK (0) or a negative
 * PAGED_ATTN_ERR_* code.  Argument errors are detected on the host before any
 * CUDA call.  Nothing aborts, throws or exits.
 */
#ifndef PAGED_ATTN_H_
#define PAGED_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Only the entry points below are exported from the shared library (it is built
 * with hidden default visibility), so several copies of it -- say, two versions
 * -- can live in one process without sharing any internal state. */
#if defined(__GNUC__)
#define PAGED_ATTN_API __attribute__((visibility("default")))
#else
#define PAGED_ATTN_API
#endif

#define PAGED_ATTN_OK 0
#define PAGED_ATTN_ERR_POINTER (-1)    /* null or not 16-byte aligned pointer */
#define PAGED_ATTN_ERR_HEADS (-2)      /* H_kv <= 0, H_q % H_kv != 0, or G > 16 */
#define PAGED_ATTN_ERR_HEAD_DIM (-3)   /* head_dim not in {64, 128, 256} */
#define PAGED_ATTN_ERR_BLOCK_SIZE (-4) /* block_size not in {16, 32} */
#define PAGED_ATTN_ERR_SIZES (-5)      /* num_seqs < 0, max_blocks_per_seq <= 0, or too large */
#define PAGED_ATTN_ERR_CUDA (-6)       /* a CUDA runtime/driver call failed; see paged_attn_last_cuda_error */
#define PAGED_ATTN_ERR_WORKSPACE (-7)  /* workspace pointer null/misaligned or smaller than required */
#define PAGED_ATTN_ERR_SCALE (-8)      /* scale is not finite */
#define PAGED_ATTN_ERR_STATIC_SCRATCH (-9) /* sizes exceed paged_attn_decode_static's scratch */
#define PAGED_ATTN_ERR_FLAGS (-10)     /* unknown bits in paged_attn_set_launch_flags */
#define PAGED_ATTN_ERR_MODS (-11)      /* softcap not 0 and outside [1e-30, 1e30] (or scale / softcap past 1e30), or window < 0 */
#define PAGED_ATTN_ERR_ROPE (-12)      /* rotary_dim, num_axes, max_positions or eps out of range */

/* Launch flags (paged_attn_set_launch_flags). */
#define PAGED_ATTN_FLAG_EARLY_PROLOGUE 1

/*
 * Decode attention (the operation above).
 *
 * Scratch: the split-KV partial states live in a per-device workspace that the
 * library owns.  The first call on a device (and any call that needs a larger
 * workspace than before) allocates it with cudaMallocAsync on `stream` from the
 * device's default memory pool and zero-fills it there (a smaller one is
 * released with cudaFreeAsync on `stream`, after the calls before it on that
 * stream); later calls allocate nothing.  Because the workspace is shared,
 * calls that may overlap on the GPU (different streams, same device) race:
 * give each concurrent stream its own workspace through paged_attn_decode_ws.
 */
PAGED_ATTN_API int paged_attn_decode(const void* q, const void* k_cache, const void* v_cache, void* out,
                      const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                      int H_q, int H_kv, int head_dim, int max_blocks_per_seq, int block_size,
                      float scale, void* stream);

/*
 * Bytes of caller-provided workspace that paged_attn_decode_ws needs for these
 * sizes on the CURRENT device (it depends on the device's SM count).  Returns 0
 * for unsupported sizes.
 */
PAGED_ATTN_API size_t paged_attn_workspace_bytes(int num_seqs, int H_q, int H_kv, int head_dim,
                                  int max_blocks_per_seq, int block_size);

/*
 * Same operation with a caller-owned device workspace of at least
 * paged_attn_workspace_bytes(...) bytes, 256-byte aligned.  The workspace
 * must be zero-filled before its first use; every call that returns
 * PAGED_ATTN_OK and completes on the GPU leaves its counter region (whose
 * place depends only on the device) zero again, so the same workspace serves
 * any later call on the same device that fits in it.  Calls sharing one
 * workspace must not overlap on the GPU.  Allocates nothing.
 */
PAGED_ATTN_API int paged_attn_decode_ws(const void* q, const void* k_cache, const void* v_cache, void* out,
                         const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                         int H_q, int H_kv, int head_dim, int max_blocks_per_seq, int block_size,
                         float scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Same operation with device-side input checks.  num_blocks is the size of the
 * caller's block pool.  A block id outside [0, num_blocks) in a used table
 * entry, or a sequence length outside [0, max_blocks_per_seq * block_size],
 * sets bit 0 (bad block) or bit 1 (bad length) of *d_status (a device int32
 * the caller zero-fills); bad blocks read as zero rows, bad lengths are
 * clamped, and no memory outside the pool is read.  Bit 2 reports that a
 * pipeline wait in the kernel ran out of its iteration limit and bit 3 that
 * the kernel rejected its launch configuration (library faults, never
 * expected; the output of such a call is undefined, the workspace stays
 * usable unless a combine wait ran out, in which case the workspace must be
 * zero-filled again before its next use: paged_attn_reset_workspace for the
 * library-owned one).  The
 * kernel writes *d_status only after the work ahead of it in the stream has
 * completed, so that work may zero-fill it.  Uses the library-owned workspace
 * like paged_attn_decode.
 */
PAGED_ATTN_API int paged_attn_decode_checked(const void* q, const void* k_cache, const void* v_cache, void* out,
                              const int32_t* block_tables, const int32_t* seq_lens,
                              int num_seqs, int H_q, int H_kv, int head_dim,
                              int max_blocks_per_seq, int block_size, float scale,
                              long long num_blocks, int32_t* d_status, void* stream);

/*
 * Same operation for callers that cannot allocate device memory.  There is no
 * counterpart in the reference pages; this entry point exists for callers whose
 * host framework owns all device memory -- a serving engine that reserves the
 * whole HBM for its KV-cache pool, or a plugin host that forbids allocation --
 * and for decode loops that cannot afford cudaMalloc's implicit device
 * synchronisation.  It calls no cudaMalloc, cudaFree or allocating library
 * routine: its scratch (split-KV partial states and combine counters) is a
 * fixed 4 MiB array compiled into the library, which every GPU that loads the
 * library holds until the process exits.  Sizes whose scratch would exceed
 * 4 MiB (those for which paged_attn_workspace_bytes() reports more) return
 * PAGED_ATTN_ERR_STATIC_SCRATCH before anything is launched (on a 152-SM
 * GB300 that is, for instance, head_dim 128 with 16 query heads per KV head;
 * the LLaMA-3-8B-, Qwen- and GQA-8-shaped decode batches all fit).
 *
 * The first call on each device looks up the array's device address (with
 * that device current) and caches it, so make that first call before any
 * stream capture.  Every call clears the array's status and counter region
 * on `stream` (a memset, not an allocation) and then shares the array: calls
 * that may overlap on the GPU (several streams, several host threads) race
 * on it and must be serialised by the caller.
 */
PAGED_ATTN_API int paged_attn_decode_static(const void* q, const void* k_cache, const void* v_cache, void* out,
                             const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                             int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
                             int block_size, float scale, void* stream);

/*
 * Device-side checks for every later call of the calling thread: with
 * num_blocks > 0, every decode and append entry point validates the block ids
 * it uses against [0, num_blocks) and reports into *d_status (a device int32,
 * 4-byte aligned, that the caller zero-fills) as paged_attn_decode_checked
 * does: bit 0 for a bad block id (a decode reads zero rows for it through the
 * tensor copies of the standard and FP8 layouts, block 0's rows through the
 * bulk copies of the x-packed layout; an append skips that row), bit 1 for a
 * bad length or a multi-token sequence with more query rows than the call
 * allows, bits 2 and 3 as there.  (0, NULL) turns the checks off.  Returns
 * PAGED_ATTN_ERR_SIZES for num_blocks outside [1, 2^31) and
 * PAGED_ATTN_ERR_POINTER for a null or misaligned d_status, changing nothing.
 */
PAGED_ATTN_API int paged_attn_set_checks(long long num_blocks, int32_t* d_status);

/*
 * The same operation over FP8 caches: the nvfp4-megamoe README's FP8 KV path
 * ("Stage D: FP8 Paged KV Gather", "FP8 KV Quantize/Dequant": e4m3 values,
 * dequantized with a scale per position during the gather).  k_cache / v_cache
 * hold e4m3 bytes (OCP E4M3: 1 sign, 4 exponent bits with bias 7, 3 mantissa
 * bits, no infinities) in the bf16 layout above, 1 byte per element, and
 *   k_scale, v_scale  [num_blocks, H_kv, block_size]  float32  (read)
 * give each cache row its dequant factor:
 *   K_t[d] = e4m3(k_cache[b, g, slot, d]) * k_scale[b, g, slot]   (V alike).
 * head_dim must be 128 or 256 (PAGED_ATTN_ERR_HEAD_DIM otherwise).  The
 * products run on f16 tensor cores: q is rounded to f16 (exact for bf16 values
 * of magnitude 2^-14 .. 65504), the probabilities times the V row factors are
 * rounded to f16; accumulation is fp32.  The probabilities are taken against a
 * running maximum that may trail the true one by up to a factor of 16 (so each
 * is at most 16): V row factors below 4094 (rows of magnitude below about
 * 1.8e6) keep the f16 products finite.  Workspace, allocation and errors as
 * paged_attn_decode; rows past a sequence's length may hold anything (NaN
 * bytes and factors included).
 */
PAGED_ATTN_API int paged_attn_decode_fp8(const void* q, const void* k_cache, const void* v_cache,
                                         const float* k_scale, const float* v_scale, void* out,
                                         const int32_t* block_tables, const int32_t* seq_lens,
                                         int num_seqs, int H_q, int H_kv, int head_dim,
                                         int max_blocks_per_seq, int block_size, float scale,
                                         void* stream);

/*
 * Multi-token decode: several new tokens per sequence query the cache at once
 * (speculative decoding, chunked prefill), the ragged query batch of AstrAI's
 * CUDA Kernels page ("Q Scheduling and KV Addressing": rows located through
 * qo_indptr; "Python Wrappers": is_causal).  Sequence s owns the query rows
 * qo_indptr[s] .. qo_indptr[s+1] - 1, its last q_len = qo_indptr[s+1] -
 * qo_indptr[s] tokens, which are already in the cache (seq_lens[s] counts
 * them).  Query i of sequence s attends the tokens t <= seq_lens[s] - q_len + i
 * (causal: its own position and everything before):
 *
 *   out[qo[s] + i, h, :] = softmax_t(scale * q[qo[s] + i, h, :] . K_t) . V_t,
 *                          t in [0, seq_lens[s] - q_len + i]
 *
 *   q, out      [total_q, H_q, head_dim]  bf16 (read / written)
 *   qo_indptr   [num_seqs + 1]  int32, device, 16-byte aligned: qo_indptr[0] = 0,
 *               non-decreasing, qo_indptr[num_seqs] = total_q
 *   max_q_len   the largest q_len (host value); max_q_len * (H_q / H_kv) <= 256
 *
 * Caches, tables, lengths, head_dim, block_size and scale as paged_attn_decode
 * (bf16 caches in the standard layout).  The q_len * G query rows of one KV
 * head are processed together, in pieces of 16 rows when they are more than 8:
 * every piece streams the KV head's pages once.  Rows whose query sees no token
 * (q_len > seq_len) and the rows of empty sequences are zero.  Query rows a
 * sequence does not own are not written.  Returns PAGED_ATTN_ERR_SIZES for
 * total_q < 0, max_q_len < 1 or max_q_len * G > 256; errors otherwise as
 * paged_attn_decode.  Uses the library-owned workspace.
 */
PAGED_ATTN_API int paged_attn_decode_multi(const void* q, const void* k_cache,
                                           const void* v_cache, void* out,
                                           const int32_t* qo_indptr,
                                           const int32_t* block_tables,
                                           const int32_t* seq_lens, int num_seqs, int total_q,
                                           int max_q_len, int H_q, int H_kv, int head_dim,
                                           int max_blocks_per_seq, int block_size, float scale,
                                           void* stream);

/*
 * paged_attn_decode_multi with the causal mask chosen by the caller (AstrAI's
 * CUDA Kernels page, "Python Wrappers": is_causal).  is_causal != 0 is
 * paged_attn_decode_multi; is_causal = 0 lets every query row of sequence s
 * attend all its tokens t < seq_lens[s]:
 *
 *   out[qo[s] + i, h, :] = softmax_t(scale * q[qo[s] + i, h, :] . K_t) . V_t,
 *                          t in [0, seq_lens[s])
 *
 * Everything else as paged_attn_decode_multi.
 */
PAGED_ATTN_API int paged_attn_decode_multi_ex(const void* q, const void* k_cache,
                                              const void* v_cache, void* out,
                                              const int32_t* qo_indptr,
                                              const int32_t* block_tables,
                                              const int32_t* seq_lens, int num_seqs,
                                              int total_q, int max_q_len, int H_q, int H_kv,
                                              int head_dim, int max_blocks_per_seq,
                                              int block_size, float scale, int is_causal,
                                              void* stream);

/*
 * The same operation over bf16 caches in the x-packed layout ("Paged Attention
 * Kernel Architecture for BI-V100", section 3, Paged K/V Gather: the key cache
 * split into 16-byte packs of x = 8 elements, the value cache head_dim-major):
 *
 *   k_cache  [num_blocks, H_kv, head_dim / 8, block_size, 8]  bf16  (read)
 *   v_cache  [num_blocks, H_kv, head_dim, block_size]         bf16  (read)
 *
 * so K_t[d] = k_cache[b, g, d / 8, t % block_size, d % 8] and
 * V_t[d] = v_cache[b, g, d, t % block_size] with b = block_tables[s, t / block_size].
 * Everything else (q, out, tables, lengths, sizes, scale, workspace, errors,
 * rows past a sequence's length) is as paged_attn_decode; the arithmetic is
 * the same, so the output equals paged_attn_decode's over the same values.
 */
PAGED_ATTN_API int paged_attn_decode_xpacked(const void* q, const void* k_cache,
                                             const void* v_cache, void* out,
                                             const int32_t* block_tables,
                                             const int32_t* seq_lens, int num_seqs, int H_q,
                                             int H_kv, int head_dim, int max_blocks_per_seq,
                                             int block_size, float scale, void* stream);

/*
 * Cache append ("reshape and cache") of one new token per sequence, the write
 * that precedes the decode: the paged-decode layout above counts the new token
 * in seq_lens ("context length including the new token"), so its K and V must
 * be in the cache when the decode runs; AstrAI's CUDA-kernels page (Backend
 * Layer) has the backend own that write.  For every sequence s with
 * L = seq_lens[s] >= 1 and every KV head g, with t = L - 1:
 *
 *   k_cache[block_tables[s, t / block_size], g, t % block_size, :] = k_new[s, g, :]
 *   v_cache[...same place...]                                      = v_new[s, g, :]
 *
 *   k_new, v_new  [num_seqs, H_kv, head_dim]  bf16  (read; device, 16-byte aligned)
 *   k_cache, v_cache                          bf16  (written at those rows only)
 *
 * Sequences with L = 0 or L > max_blocks_per_seq * block_size write nothing.
 * The block ids are not checked.  Sizes follow paged_attn_decode's rules
 * (head_dim 64/128/256, block_size 16/32); errors as above.  Asynchronous on
 * `stream`; allocates nothing.
 */
PAGED_ATTN_API int paged_kv_append(const void* k_new, const void* v_new, void* k_cache,
                                   void* v_cache, const int32_t* block_tables,
                                   const int32_t* seq_lens, int num_seqs, int H_kv, int head_dim,
                                   int max_blocks_per_seq, int block_size, void* stream);

/*
 * paged_kv_append followed by paged_attn_decode, fused into the decode launch:
 * the warp that processes the page holding a sequence's new token puts that
 * token's K and V rows into its copy of the page in shared memory (whatever
 * the cache held there is not used) and stores them to the cache, so the
 * append costs no extra launch and no extra pass over the cache.  The blocks
 * that receive the new tokens must not also be read by another sequence of
 * the same call (no copy-on-write sharing of a partly filled block).  When the
 * batch has many (sequence, KV head) pairs per SM (four or more per CTA of the
 * persistent grid), the per-piece patch would sit on the critical path of the
 * CTA crossing the most short sequences, and the call instead runs the append
 * as its own launch just ahead of the decode; the result is the same.  Same
 * arguments, workspace and errors as paged_attn_decode, plus k_new / v_new
 * ([num_seqs, H_kv, head_dim] bf16, 16-byte aligned).
 */
PAGED_ATTN_API int paged_attn_append_decode(const void* q, const void* k_new, const void* v_new,
                                            void* k_cache, void* v_cache, void* out,
                                            const int32_t* block_tables, const int32_t* seq_lens,
                                            int num_seqs, int H_q, int H_kv, int head_dim,
                                            int max_blocks_per_seq, int block_size, float scale,
                                            void* stream);

/*
 * Cache append of several new tokens per sequence, the write that precedes the
 * multi-token decode: the rows of k_new / v_new ([total_q, H_kv, head_dim]
 * bf16, 16-byte aligned) follow qo_indptr as the queries do (AstrAI's CUDA
 * Kernels page, "Q Scheduling and KV Addressing"): row qo_indptr[s] + i is
 * token t = seq_lens[s] - q_len + i of sequence s (q_len = qo_indptr[s+1] -
 * qo_indptr[s]; seq_lens counts the new tokens), and for every KV head g
 *
 *   k_cache[block_tables[s, t / block_size], g, t % block_size, :] = k_new[qo_indptr[s] + i, g, :]
 *
 * (v alike).  Rows with t < 0 (more new rows than the sequence holds), of a
 * sequence with a length outside [1, max_blocks_per_seq * block_size], or
 * outside [qo_indptr[0], qo_indptr[num_seqs]) write nothing.  Sizes and errors
 * as paged_kv_append, plus PAGED_ATTN_ERR_SIZES for total_q < 0.
 * Asynchronous on `stream`; allocates nothing.
 */
PAGED_ATTN_API int paged_kv_append_multi(const void* k_new, const void* v_new, void* k_cache,
                                         void* v_cache, const int32_t* qo_indptr,
                                         const int32_t* block_tables, const int32_t* seq_lens,
                                         int num_seqs, int total_q, int H_kv, int head_dim,
                                         int max_blocks_per_seq, int block_size, void* stream);

/*
 * paged_kv_append_multi followed by paged_attn_decode_multi_ex, as two
 * launches on `stream` (the decode waits for the append to complete before it
 * reads anything, whatever the launch flags).  Arguments as the two calls.
 */
PAGED_ATTN_API int paged_attn_append_decode_multi(const void* q, const void* k_new,
                                                  const void* v_new, void* k_cache,
                                                  void* v_cache, void* out,
                                                  const int32_t* qo_indptr,
                                                  const int32_t* block_tables,
                                                  const int32_t* seq_lens, int num_seqs,
                                                  int total_q, int max_q_len, int H_q, int H_kv,
                                                  int head_dim, int max_blocks_per_seq,
                                                  int block_size, float scale, int is_causal,
                                                  void* stream);

/*
 * Cache append into FP8 caches (quantize on write; nvfp4-megamoe README, "FP8
 * KV Quantize/Dequant" and "Paged KV cache read/write"): the new token's K and
 * V rows of every sequence and KV head, bf16 [num_seqs, H_kv, head_dim], are
 * quantized one row at a time and written where paged_kv_append writes:
 *
 *   f        = max_d |x[d]| / 448   in float32 (f = 1 for an all-zero row)
 *   byte[d]  = e4m3(x[d] / f)       float32 quotient, rounded to nearest even,
 *                                   saturated to +-448
 *   k_cache[b, g, slot, :] = byte,  k_scale[b, g, slot] = f   (v alike)
 *
 * so that paged_attn_decode_fp8 reads x[d] as e4m3(byte[d]) * f.  k_cache /
 * v_cache hold e4m3 bytes, k_scale / v_scale float32 [num_blocks, H_kv,
 * block_size]; head_dim 128 or 256 (PAGED_ATTN_ERR_HEAD_DIM otherwise).
 * Which sequences write, sizes, errors: as paged_kv_append.  Asynchronous on
 * `stream`; allocates nothing.
 */
PAGED_ATTN_API int paged_kv_append_fp8(const void* k_new, const void* v_new, void* k_cache,
                                       void* v_cache, float* k_scale, float* v_scale,
                                       const int32_t* block_tables, const int32_t* seq_lens,
                                       int num_seqs, int H_kv, int head_dim,
                                       int max_blocks_per_seq, int block_size, void* stream);

/*
 * paged_kv_append_fp8 followed by paged_attn_decode_fp8, fused into the decode
 * launch as paged_attn_append_decode is for bf16 caches: the warp that reads the
 * page holding a sequence's new token quantizes the new K and V rows exactly as
 * paged_kv_append_fp8 does, puts the bytes and row floats into its copy of the
 * page in shared memory and stores them to the cache.  For head_dim 256, or
 * with four or more (sequence, KV head) pairs per CTA of the persistent grid,
 * the append runs as its own launch and the decode after it is a plain launch
 * (whatever the launch flags).  The same bytes, floats and output either way.  Arguments as the two
 * calls; the blocks receiving new tokens must not also be read by another
 * sequence of the same call.
 */
PAGED_ATTN_API int paged_attn_append_decode_fp8(const void* q, const void* k_new,
                                                const void* v_new, void* k_cache, void* v_cache,
                                                float* k_scale, float* v_scale, void* out,
                                                const int32_t* block_tables,
                                                const int32_t* seq_lens, int num_seqs, int H_q,
                                                int H_kv, int head_dim, int max_blocks_per_seq,
                                                int block_size, float scale, void* stream);

/*
 * Decode with score options, for the layers whose scores are not the plain
 * scaled products.  The query of sequence s stands at position pos = L - 1 (L
 * = seq_lens[s], clamped as in paged_attn_decode) and
 *
 *   x(h, t) = scale * q[s, h, :] . K_t
 *   x       = softcap * tanh(x / softcap)            softcap > 0 (0: off)
 *   x       = x - alibi_slopes[h] * |pos - t|        alibi_slopes non-null
 *   out[s, h, :] = sum_t softmax_t(x) V_t over the tokens t < L that it sees:
 *       t < prefix_lens[s]   or
 *       t >= doc_starts[s]  and  (window == 0 or t > pos - window)
 *
 *   alibi_slopes  [H_q]       float32  (read; null: no distance bias)
 *   window        tokens the query sees at most, itself included (0: all)
 *   prefix_lens   [num_seqs]  int32    (read; null: 0) a prefix that every query
 *                 sees whatever the window and the documents (an attention sink,
 *                 a prefix language model's prefix)
 *   doc_starts    [num_seqs]  int32    (read; null: 0) the first token of the
 *                 document the query is in, in a sequence that packs several
 *
 * softcap is 0 or in [1e-30, 1e30], and max_blocks_per_seq * block_size at most
 * 2^31 - 256.  prefix_lens and doc_starts are clamped to [0, L].  A query that
 * sees no token gets a zero row.  Pages that hold no token the query sees are not read (their
 * table entries neither), and unseen rows of the pages that are may hold
 * anything, NaN included.  The arrays are 4-byte aligned device (or pinned
 * host) memory.  The cap is computed in float32 to about 1e-6 of the score, the
 * bias as one float32 multiply-add on top of it; everything else is
 * paged_attn_decode's.
 *
 * workspace: at least paged_attn_mods_workspace_bytes(...) bytes, 256-byte
 * aligned, zero-filled before its first use, not shared by calls that may
 * overlap (one workspace serves any calls of the _mods and _shared entry points
 * on a device, in any order); or null, for a workspace that the library keeps for
 * the call's stream, apart from paged_attn_decode's: calls on different streams, and
 * of the two kinds, may overlap.  It is allocated and grown as paged_attn_decode's;
 * past 64 streams a device the least recently used stream's is given up, after a
 * cudaDeviceSynchronize.  A stream that is being captured must pass one: with a
 * null workspace the call returns PAGED_ATTN_ERR_WORKSPACE there.  Launch flags do
 * not apply.
 */
PAGED_ATTN_API int paged_attn_decode_mods(const void* q, const void* k_cache,
                                          const void* v_cache, void* out,
                                          const int32_t* block_tables, const int32_t* seq_lens,
                                          int num_seqs, int H_q, int H_kv, int head_dim,
                                          int max_blocks_per_seq, int block_size, float scale,
                                          float softcap, const float* alibi_slopes, int window,
                                          const int32_t* prefix_lens, const int32_t* doc_starts,
                                          void* workspace, size_t workspace_bytes, void* stream);

/* The same over FP8 caches (paged_attn_decode_fp8: head_dim 128 or 256). */
PAGED_ATTN_API int paged_attn_decode_fp8_mods(
    const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
    const float* v_scale, void* out, const int32_t* block_tables, const int32_t* seq_lens,
    int num_seqs, int H_q, int H_kv, int head_dim, int max_blocks_per_seq, int block_size,
    float scale, float softcap, const float* alibi_slopes, int window,
    const int32_t* prefix_lens, const int32_t* doc_starts, void* workspace,
    size_t workspace_bytes, void* stream);

/* Bytes of workspace paged_attn_decode_mods and paged_attn_decode_fp8_mods need for
 * these sizes on the CURRENT device; 0 for unsupported sizes. */
PAGED_ATTN_API size_t paged_attn_mods_workspace_bytes(int num_seqs, int H_q, int H_kv,
                                                      int head_dim, int max_blocks_per_seq,
                                                      int block_size);

/*
 * Attention of several query tokens per sequence with score options: the
 * verification of drafted tokens, a chunk of a prompt, a whole prompt.  Any
 * number of query rows per sequence (paged_attn_decode_multi takes up to 256 per
 * KV head).  Sequence s owns the rows t = qo_indptr[s] + i, its last q_len =
 * qo_indptr[s+1] - qo_indptr[s] tokens, which are already in the cache; row i
 * stands at position pos = seq_lens[s] - q_len + i and sees the tokens t' < L with
 *
 *       t' < prefix_lens[s]   or
 *       t' >= doc_starts[t]  and  (window == 0 or t' > pos - window)
 *                            and  (is_causal == 0 or t' <= pos)
 *
 * with the scores of paged_attn_decode_mods, |pos - t'| the distance of the
 * bias.  q, out, qo_indptr and total_q as paged_attn_decode_multi, except that
 * doc_starts is [total_q] (one per row) and there is no max_q_len.  Rows that
 * see no token are zero; rows of q no sequence owns are not written.
 *
 * Without causality (is_causal = 0) the window and the document bound a query's view
 * on the left only: it sees everything from there to the sequence's end, later
 * documents included.  A bidirectional document mask over a packed sequence
 * is therefore not among these options.
 *
 * The query rows of a KV head are worked on in pieces of consecutive rows (up to 128 or
 * 256, as a call's sizes have it).  Pages ahead of all that a piece's rows see (its
 * prefix aside) and behind it are not read, nor their table entries.  Cache rows
 * that no query of the sequence sees may hold anything, NaN included; a cache row that
 * only some of a sequence's queries see must be finite for the others' sake.
 *
 * The products run on the 5th-generation tensor cores (bf16 operands, the
 * weights rounded to bf16, fp32 accumulation).  workspace: as
 * paged_attn_decode_mods, paged_attn_multi_mods_workspace_bytes(...) bytes.
 */
PAGED_ATTN_API int paged_attn_decode_multi_mods(
    const void* q, const void* k_cache, const void* v_cache, void* out,
    const int32_t* qo_indptr, const int32_t* block_tables, const int32_t* seq_lens,
    int num_seqs, int total_q, int H_q, int H_kv, int head_dim, int max_blocks_per_seq,
    int block_size, float scale, int is_causal, float softcap, const float* alibi_slopes,
    int window, const int32_t* prefix_lens, const int32_t* doc_starts, void* workspace,
    size_t workspace_bytes, void* stream);

PAGED_ATTN_API size_t paged_attn_multi_mods_workspace_bytes(int num_seqs, int total_q, int H_q,
                                                            int H_kv, int head_dim,
                                                            int max_blocks_per_seq,
                                                            int block_size);

/*
 * Attention of a tree of drafted tokens (speculative decoding with several
 * continuations at once): sequence s owns the rows t = qo_indptr[s] + i, its last q_len =
 * qo_indptr[s+1] - qo_indptr[s] tokens, which are already in the cache, and ctx =
 * seq_lens[s] - q_len tokens stand before the tree.  Row i sees
 *
 *       the cached tokens t' < ctx  with  t' < prefix_lens[s]  or
 *                                         (window == 0 or t' > pos - window)
 *       the drafted token j of its sequence (token ctx + j) where bit j % 32 of
 *       tree_mask[t, j / 32] is set
 *
 * and stands at pos = ctx + n - 1, n the drafted tokens it sees: in a tree, whose nodes see
 * themselves and their ancestors, as deep as the node is.  The scores are those of
 * paged_attn_decode_mods; the distance of the bias is |pos - t'| for a cached token and
 * the difference of the two rows' positions for a drafted one.  A mask without bits
 * leaves the cached tokens (a padding node; pos = ctx - 1); a row that sees nothing is zero.
 *
 * The window bounds cached tokens alone: a row sees each drafted token that it has a bit for,
 * however far above it the node stands.  So the call is right for a layer whose window is at
 * least as long as its trees are deep, and only there a chain is what
 * paged_attn_decode_multi_mods makes of it.  (Bits taken out for far ancestors move the
 * row's position, and with it the window over cached tokens and the bias.)
 *
 *   tree_mask   [total_q, mask_words]  int32 (read; 16-byte aligned): any bits, those
 *               from q_len on are not used
 *   mask_words  1 .. 8: a drafted token from 32 * mask_words on has no bit and is seen by no
 *               row (with paged_attn_set_checks on, it sets bit 1 of the status word)
 *
 * Cache rows that no row sees, those of padding nodes too, may hold anything, NaN
 * included; a row that only some of a sequence's rows see must be finite for the others'
 * sake.  Everything else as paged_attn_decode_multi_mods; workspace: as there,
 * paged_attn_tree_workspace_bytes(...) bytes.  Returns PAGED_ATTN_ERR_SIZES for mask_words
 * out of range.
 */
PAGED_ATTN_API int paged_attn_decode_tree(
    const void* q, const void* k_cache, const void* v_cache, void* out,
    const int32_t* qo_indptr, const int32_t* tree_mask, int mask_words,
    const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int total_q, int H_q,
    int H_kv, int head_dim, int max_blocks_per_seq, int block_size, float scale, float softcap,
    const float* alibi_slopes, int window, const int32_t* prefix_lens, void* workspace,
    size_t workspace_bytes, void* stream);

PAGED_ATTN_API size_t paged_attn_tree_workspace_bytes(int num_seqs, int total_q, int H_q,
                                                      int H_kv, int head_dim,
                                                      int max_blocks_per_seq, int block_size);

/*
 * Decode of a batch whose sequences share long prefixes (system prompts, a
 * document that many questions are about), each prefix read once for all its
 * sequences.  Sequences group_indptr[g] .. group_indptr[g+1] - 1 form group g
 * and begin with the prefix_lens[g] tokens that prefix_tables[g] leads to; their
 * own tokens follow, seq_lens[s] of them, in their own blocks:
 *
 *   x(h, t) over the prefix's tokens (positions 0 .. P - 1) and then the
 *   sequence's own (positions P .. P + seq_lens[s] - 1), P = prefix_lens[g]
 *   out[s, h, :] = softmax_t(x) . V_t
 *
 * with the scaled products, the cap and the distance bias of
 * paged_attn_decode_mods (the query stands at P + seq_lens[s] - 1).
 *
 *   group_indptr  [num_groups + 1]  int32, non-decreasing; a sequence in no group
 *                 has no prefix
 *   prefix_tables [num_groups, prefix_max_blocks]  int32 (read)
 *   prefix_lens   [num_groups]  int32 (read), clamped to [0, prefix_max_blocks *
 *                 block_size]: any length, not only whole blocks
 *   seq_lens      [num_seqs]  a sequence's own tokens, without the prefix (0 allowed)
 *
 * Everything else as paged_attn_decode; rows past a prefix's or a sequence's end
 * may hold anything.  A sequence without any token gets zero rows.  Three
 * launches: the prefixes and, side by side with them, the own tokens, then the
 * merge.  num_groups = 0 is paged_attn_decode_mods.  workspace: as there,
 * paged_attn_shared_workspace_bytes(...) bytes.
 */
PAGED_ATTN_API int paged_attn_decode_shared(
    const void* q, const void* k_cache, const void* v_cache, void* out,
    const int32_t* group_indptr, const int32_t* prefix_tables, const int32_t* prefix_lens,
    int num_groups, int prefix_max_blocks, const int32_t* block_tables, const int32_t* seq_lens,
    int num_seqs, int H_q, int H_kv, int head_dim, int max_blocks_per_seq, int block_size,
    float scale, float softcap, const float* alibi_slopes, void* workspace,
    size_t workspace_bytes, void* stream);

PAGED_ATTN_API size_t paged_attn_shared_workspace_bytes(int num_seqs, int num_groups, int H_q,
                                                        int H_kv, int head_dim,
                                                        int max_blocks_per_seq, int block_size);

/*
 * Block tables, query offsets and the slot map of a serving step, built on the
 * GPU from request lengths.  Sequence s holds seq_lens[s] tokens and new_lens[s]
 * arrive, as the rows qo_indptr[s] .. qo_indptr[s+1] - 1 of the step's packed
 * batch (qo_indptr: the running sum of new_lens, row 0 first).  The pages its
 * new tokens begin take blocks from the top of the free stack, in the order of
 * the sequences and of their pages:
 *
 *   need[s]  = ceil((seq_lens[s] + new_lens[s]) / block_size) - ceil(seq_lens[s] / block_size)
 *   block k of the call = free_blocks[free_count - 1 - k]
 *   slot_map[qo_indptr[s] + i] = block * block_size + t % block_size,  t = seq_lens[s] + i
 *
 *   seq_lens, new_lens  [num_seqs]  int32  (read)
 *   block_tables   [num_seqs, max_blocks_per_seq]  int32: the entries of the fresh
 *                  pages are written, the others are left (and the last page's
 *                  read, when tokens join it)
 *   free_blocks    [free_capacity]  int32  (read), free_count [1] int32 (read;
 *                  clamped to [0, free_capacity])
 *   seq_lens_out   [num_seqs]  int32: seq_lens + new_lens; may be seq_lens itself
 *   qo_indptr      [num_seqs + 1]  int32 (written)
 *   slot_map       [max_new]  int64 (written whole: -1 past the last row)
 *   free_count_out [1] int32: what is left; may be free_count itself
 *   refused        [1] int32, or null: how many sequences were refused
 *
 * A sequence is refused when its blocks and those of the sequences before it do
 * not all fit in the free stack, when its tokens do not fit its table row or
 * its rows do not fit in max_new, or when a length is negative (its rows count
 * as 0 then).  It takes no block, keeps its length (seq_lens_out) and its table
 * row, and its rows get slots of -1; sequences that need no block are served
 * whatever is free.  Other outputs must not overlap inputs.
 *
 * max_new bounds the sum of new_lens, so that a captured step serves any batch
 * of up to that many rows.  Any number of sequences (of none, the padding slots,
 * qo_indptr[0] and the counts are written); max_blocks_per_seq and
 * block_size as paged_attn_decode.  The tensors are 16-byte aligned, the
 * one-element ones 4-byte.  With paged_attn_set_checks on, a block id outside the
 * pool sets bit 0 and an invalid length bit 1 of the status word (such an id is
 * still assigned).  One launch; no workspace; asynchronous on `stream`.
 */
PAGED_ATTN_API int paged_kv_assign(const int32_t* seq_lens, const int32_t* new_lens,
                                   int32_t* block_tables, const int32_t* free_blocks,
                                   const int32_t* free_count, int32_t* seq_lens_out,
                                   int32_t* qo_indptr, int64_t* slot_map,
                                   int32_t* free_count_out, int32_t* refused, int num_seqs,
                                   int max_blocks_per_seq, int block_size, int free_capacity,
                                   int max_new, void* stream);

/*
 * Cache append by slot: row r of the new tokens goes to slot_map[r] = block *
 * block_size + place, for every KV head g
 *
 *   k_cache[block, g, place, :] = k_new[r, g, :]      (v alike)
 *
 * so that it needs neither tables nor lengths (paged_kv_assign makes the map).
 *
 *   k_new, v_new  row r begins k_stride (v_stride) elements after row r - 1 and
 *                 holds [H_kv, head_dim] bf16: slices of one fused projection
 *                 need no copy; strides are multiples of 8, at least H_kv * head_dim
 *   slot_map      [rows]  int64 (read).  A slot outside [0, num_blocks * block_size)
 *                 writes nothing (-1: a padding row); with paged_attn_set_checks on, one
 *                 past the pool sets bit 0 of the status word.
 *
 * The slots of a call must be distinct: of two rows with the same slot either
 * may remain, in pieces of 16 bytes.  num_blocks is the pool's size, in [1, 2^31).
 * Sizes and errors as paged_kv_append.  Asynchronous; allocates nothing.
 */
PAGED_ATTN_API int paged_kv_append_slots(const void* k_new, const void* v_new,
                                         long long k_stride, long long v_stride, void* k_cache,
                                         void* v_cache, const int64_t* slot_map, int rows,
                                         int H_kv, int head_dim, int block_size,
                                         long long num_blocks, void* stream);

/*
 * What comes between a layer's projection and its attention, in one pass: the norm of
 * each query and key head, their rotation by position, and the append of the K and V rows
 * by slot.  For row r and every head, in float32 up to the one rounding at the end:
 *
 *   y = x / sqrt(mean_d(x[d]^2) + eps) * norm[d]      (norm null: y = x)
 *   for the pairs i < rotary_dim / 2, (a, b) = (i, i + rotary_dim / 2), or (2i, 2i + 1)
 *   with interleaved != 0, p = positions[axis(i), r]:
 *     z[a] = y[a] cos_sin[p, i] - y[b] cos_sin[p, rotary_dim / 2 + i]
 *     z[b] = y[b] cos_sin[p, i] + y[a] cos_sin[p, rotary_dim / 2 + i]
 *   z[d] = y[d]  for d >= rotary_dim
 *
 *   q_out[r, h, :] = bf16(z of q[r, h, :])
 *   the cache rows at slot_map[r], as paged_kv_append_slots: bf16(z of k_new[r, g, :]) and
 *   v_new[r, g, :]; with k_scale and v_scale the caches are FP8 and z and v_new are
 *   quantized as paged_kv_append_fp8 does (z from its float32 values)
 *
 *   q, k_new, v_new  rows at their strides as paged_kv_append_slots (slices of one fused
 *                 projection need no copy); device memory
 *   q_out         [rows, H_q, head_dim]  bf16 (written); may be q where q_stride = H_q *
 *                 head_dim, else apart from all inputs (PAGED_ATTN_ERR_POINTER where it
 *                 meets a row of q, k_new or v_new)
 *   k_scale, v_scale  [num_blocks, H_kv, block_size]  float32 (written), or both null; with
 *                 them head_dim is 128 or 256
 *   slot_map      [rows]  int64.  A slot outside [0, num_blocks * block_size) writes no K
 *                 and V (-1: a padding row); q_out is written all the same
 *   positions     [num_axes, rows]  int32, clamped to [0, max_positions).  One axis for
 *                 text; time, height and width for images and video
 *   freq_axis     [rotary_dim / 2]  int32, 16-byte aligned: the axis of each pair, clamped
 *                 to [0, num_axes), or null (axis 0)
 *   cos_sin       [max_positions, rotary_dim]  float32: cosines, then sines, of each
 *                 position's angles (any frequencies, any scaling of them)
 *   q_norm, k_norm  [head_dim]  float32, or null
 *
 * rotary_dim is a multiple of 16 up to head_dim, or 0 (no rotation; positions and
 * cos_sin may be null then).  PAGED_ATTN_ERR_ROPE for other values, for num_axes or
 * max_positions below 1 and for an eps that is negative or not finite.  The slots of a
 * call must be distinct.  With paged_attn_set_checks on, a slot past the pool sets bit 0 of
 * the status word, a position outside the table bit 1 (and bit 2 reports a copy that did not
 * come, a library fault, never expected).  Strides, other sizes and
 * errors as paged_kv_append_slots.  One launch; asynchronous; allocates nothing.
 */
PAGED_ATTN_API int paged_kv_rope_append_slots(
    const void* q, const void* k_new, const void* v_new, long long q_stride, long long k_stride,
    long long v_stride, void* q_out, void* k_cache, void* v_cache, float* k_scale,
    float* v_scale, const int64_t* slot_map, const int32_t* positions, int num_axes,
    const int32_t* freq_axis, const float* cos_sin, int max_positions, int rotary_dim,
    int interleaved, const float* q_norm, const float* k_norm, float eps, int rows, int H_q,
    int H_kv, int head_dim, int block_size, long long num_blocks, void* stream);

/*
 * After the verification of drafted tokens: the rows of the accepted ones move together.
 * The tree of sequence s are its last q_len tokens, ctx = seq_lens[s] - q_len stand before
 * it (as paged_attn_decode_tree), and for every KV head, K and V (and the row floats of
 * FP8 caches, with k_scale and v_scale not null):
 *
 *   row of token ctx + i  =  old row of token ctx + accepted[s, i]     i < n
 *   seq_lens_out[s] = ctx + n
 *
 *   accepted      [num_seqs, max_accept]  int32 (read): drafted tokens in rising order,
 *                 padded with -1.  n is the place of the first entry that is not past
 *                 the one before it or not below q_len (max_accept where there is none)
 *   seq_lens_out  [num_seqs]  int32 (written), not seq_lens: paged_kv_release takes both to
 *                 give back the pages behind
 *
 * The cache rows behind the new length keep what they hold.  No block with tokens of a tree
 * may be in two sequences.  Block ids outside [0, num_blocks) move nothing (bit 0 of the
 * status word with checks on).  Sizes and errors as paged_kv_append_slots (PAGED_ATTN_ERR_SIZES
 * for max_accept outside [0, 2^30]).  One launch; asynchronous; allocates nothing.
 */
PAGED_ATTN_API int paged_kv_compact(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                    const int32_t* qo_indptr, const int32_t* accepted,
                                    const int32_t* block_tables, const int32_t* seq_lens,
                                    int32_t* seq_lens_out, int num_seqs, int max_accept, int H_kv,
                                    int head_dim, int max_blocks_per_seq, int block_size,
                                    long long num_blocks, void* stream);

/*
 * Sequences that continue another one (parallel samples, beams): table row children[i]
 * takes over the tokens of table row parents[i].  Whole pages are shared, a partly filled
 * last page is copied to a fresh block, so that both may append:
 *
 *   L = seq_lens[parents[i]], full = L / block_size
 *   block_tables[children[i], j] = block_tables[parents[i], j]  and its block_refs + 1,  j < full
 *   L % block_size > 0:  block_tables[children[i], full] = free_blocks[free_count - 1 - k], to
 *       which the rows of the L % block_size tokens are copied (K, V and FP8 row floats),
 *       k counting the forks before i with such a page
 *   seq_lens[children[i]] = L
 *
 *   block_tables  [num_rows, max_blocks_per_seq]  int32: the children's entries are written
 *   seq_lens      [num_rows]  int32: the children's are written
 *   parents, children  [num_forks]  int32.  The children of a call are distinct and none is
 *                 a parent of it; a parent may have any number of them.  A child's old pages
 *                 are not given back: it has ended before (paged_kv_release)
 *   block_refs    [num_blocks]  int32: the table rows that hold a block, less one (zero for
 *                 blocks fresh from paged_kv_assign and for free ones); paged_kv_release
 *                 counts it down.  Device memory
 *   free_blocks, free_count, free_count_out  as paged_kv_assign (free_count_out may be free_count,
 *                 at the cost of a second launch)
 *   refused       [1]  int32, or null: forks refused
 *
 * A fork is refused, its child left empty, when its block is not in the free stack or
 * a row is outside [0, num_rows).  With checks on, a block id outside [0, num_blocks) sets
 * bit 0 of the status word (it is handed on, not copied), an invalid row or length bit 1, as
 * does, in a call of up to 65536 forks, a child that is a parent or twice a child; a copy
 * that did not come sets bit 2.  PAGED_ATTN_ERR_SIZES for 2 num_forks H_kv past 2^30.
 * k_scale, v_scale, sizes and errors as paged_kv_compact.  Asynchronous; allocates nothing.
 */
PAGED_ATTN_API int paged_kv_fork(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                 int32_t* block_tables, int32_t* seq_lens,
                                 const int32_t* parents, const int32_t* children,
                                 int32_t* block_refs, const int32_t* free_blocks,
                                 const int32_t* free_count, int32_t* free_count_out,
                                 int32_t* refused, int num_forks, int num_rows, int H_kv,
                                 int head_dim, int max_blocks_per_seq, int block_size,
                                 int free_capacity, long long num_blocks, void* stream);

/*
 * Pages given back: sequence s keeps its first keep_lens[s] tokens (0: it has ended).  The
 * table entries past the page of the last kept token, up to the page of token seq_lens[s] -
 * 1, lose a holder, in the order of the sequences and of their pages:
 *
 *   block_refs[b] > 0 still counts other holders: it falls by one
 *   else the block is free: free_blocks[free_count + k] = b, k counting the blocks freed
 *   before it; a block that several entries of the call hold is freed once, in the place of
 *   the first of them, when all its holders are among them
 *   seq_lens_out[s] = min(keep_lens[s], seq_lens[s])
 *
 *   keep_lens     [num_seqs]  int32 (read), clamped to [0, seq_lens[s]]
 *   block_refs    [num_blocks]  int32 as paged_kv_fork, or null: no block is shared (num_blocks is
 *                 not used then)
 *   free_blocks   [free_capacity]  int32: written past the old count.  Room for the whole
 *                 pool is enough; a block that finds none is lost (bit 1 of the status word)
 *   free_count    [1] int32; free_count_out [1] int32 may be free_count
 *   seq_lens_out  [num_seqs]  may be seq_lens or keep_lens
 *
 * A kept last page that is only partly kept and that other rows hold too stays shared: tokens
 * appended to it would be theirs as well.  (Cut back into such a page, a sequence goes on
 * in a spare row: paged_kv_fork of it copies the page.)
 *
 * The table entries keep their values.  Entries outside [0, num_blocks) (without
 * block_refs: below 0) are passed over (bit 0 with checks on).  The result does not depend
 * on the order in which the GPU works.  num_seqs * max_blocks_per_seq below 2^31
 * (PAGED_ATTN_ERR_SIZES); other sizes, pointers and errors as paged_kv_assign.  One launch; no
 * workspace; asynchronous on `stream`.
 */
PAGED_ATTN_API int paged_kv_release(const int32_t* block_tables, const int32_t* seq_lens,
                                    const int32_t* keep_lens, int32_t* block_refs,
                                    long long num_blocks, int32_t* free_blocks,
                                    const int32_t* free_count, int32_t* seq_lens_out,
                                    int32_t* free_count_out, int num_seqs,
                                    int max_blocks_per_seq, int block_size, int free_capacity,
                                    void* stream);

/* Human-readable text for a PAGED_ATTN_* code (static storage). */
PAGED_ATTN_API const char* paged_attn_status_string(int status);

/*
 * Launch flags for the decode calls made afterwards from the calling host
 * thread (all entry points; 0, the default, restores the plain behaviour).
 * Returns PAGED_ATTN_ERR_FLAGS, and changes nothing, for unknown bits.
 *
 * PAGED_ATTN_FLAG_EARLY_PROLOGUE: every decode launch waits for the work
 * ahead of it in the stream (programmatic dependent launch) before touching
 * global memory.  With this flag the caller guarantees that this earlier work,
 * which may still be running, writes none of k_cache, v_cache (and their row
 * floats), block_tables, seq_lens or qo_indptr.  Only q, the new K/V rows of
 * the fused append and the output may be written by it.  The kernel then
 * scans the lengths, translates the first pages and starts their tensor
 * copies while that work finishes.  It waits for it only before reading q or
 * the new rows, and before writing the output, the workspace or a status
 * word.  In a layer-by-layer decode loop the kernel just before attention
 * typically writes q, and with paged_attn_append_decode the new K/V rows too,
 * but not the caches, tables or lengths.  With the caller's own
 * paged_kv_append or paged_kv_append_slots (or any other write of the caches)
 * just before, the flag must stay off.  Further back such a write is safe: every
 * launch of this library lets the next one begin only when the work ahead of its
 * call is complete, so a decode with the flag finds the call just ahead running
 * at most.  (A caller's kernel that begins its own dependents before its wait does
 * not keep to that: behind it any launch still running counts.)  The append-and-decode entry points never let their own
 * append break the guarantee: where the append is a launch of its own, the
 * decode after it is a plain launch whatever the flag says.  Results are
 * those of the plain launch.
 */
PAGED_ATTN_API int paged_attn_set_launch_flags(int flags);

/*
 * Zero-fills the library-owned workspaces of the current device, those of other
 * streams too, on `stream` (nothing to do when none exists yet); no call that uses
 * one may overlap it.  Needed only after a call reported a
 * combine wait that ran out (status bit 2), which can leave split counters set.
 */
PAGED_ATTN_API int paged_attn_reset_workspace(void* stream);

/* The last cudaError_t / CUresult value behind a PAGED_ATTN_ERR_CUDA on this thread. */
PAGED_ATTN_API int paged_attn_last_cuda_error(void);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
PAGED_ATTN_API int paged_attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_ATTN_H_ */
