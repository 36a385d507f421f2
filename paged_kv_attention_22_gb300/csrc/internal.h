// Host-side interface between the C ABI (api.cu) and the kernel translation
// units. Not installed; not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pkv.h"

namespace pkv {

// Record a failed CUDA call as this thread's last error (pkv_last_cuda_error)
// and return PKV_ERR_CUDA.
pkv_status cuda_fail(cudaError_t e, const char *where);

// SM count of the current device (cached per device); PKV_ERR_CUDA, with the
// error recorded, without a usable device or on a GPU older than sm_100.
pkv_status current_sm_count(int *sms);

// Launch with programmatic stream serialization (programmatic dependent
// launch), so a kernel's launch and prologue overlap the previous kernel's
// tail. Process-wide switch, on by default.
bool pdl_enabled();

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// ---------------------------------------------------------------- KV store
struct KvStoreArgs {
  const void *k, *v;
  void *k_cache, *v_cache;
  const int32_t *slot_mapping;
  int32_t num_tokens;
  int32_t row_vec16;      // 16-byte vectors per token row (H_kv * D * 2 / 16)
  int64_t num_slots;      // num_blocks * block_size
};
cudaError_t launch_kv_store(const KvStoreArgs &a, cudaStream_t stream);
cudaError_t take_kv_store_errors(cudaStream_t stream, uint32_t *flags);
// Device address of the kernel file's error word on the current device.
cudaError_t kv_store_error_word(uint32_t **word);

// ---------------------------------------------------------------- decode
constexpr int kDecodeChunk = 16;          // keys per unit (one TMA box of all heads of a group)
constexpr int kDecodeMaxSeqs = 1024;      // sequences per call (chunk prefix lives in smem)
constexpr int kDecodeMaxGroupHeads = 8;   // KV heads per CTA head group

// Launch shapes of the decode kernel (process-wide knob):
//   0  head groups of up to 8 KV heads, 3 TMA stages where they fit, 1 CTA/SM
//   1  head groups of up to 8 KV heads, 2 stages, 1 CTA/SM
//   2  head groups of up to 4 KV heads, 2 stages, 2 CTAs/SM
constexpr int kDecodeNumVariants = 3;
inline int decode_variant_group_max(int variant) { return variant == 2 ? 4 : 8; }
inline int decode_variant_ctas_per_sm(int variant) { return variant == 2 ? 2 : 1; }

// KV heads per CTA head group: the largest divisor of H_kv that is <= group_max.
inline int decode_group_heads(int num_kv_heads, int group_max = kDecodeMaxGroupHeads) {
  for (int d = group_max; d > 1; --d)
    if (num_kv_heads % d == 0) return d;
  return 1;
}

struct DecodeArgs {
  const void *k_new, *v_new;     // fused store: new rows [S, H_kv, D], or null
  void *k_cache_w, *v_cache_w;   // fused store: caches to write
  const int32_t *slot_mapping;   // fused store: slot of each sequence's new token
  const void *q;
  const int32_t *block_tables;
  const int32_t *context_lens;
  void *out;
  float *lse;
  float *ws_o;            // [2 grid, HG, G, D] partial outputs of pieces cut by CTA ranges
  float *ws_ml;           // [2 grid, HG, G, 2] their (max, sum), base 2
  int32_t max_blocks;
  int32_t max_context_len;
  int32_t num_seqs, num_q_heads, num_kv_heads, head_dim, block_size;
  int32_t num_blocks;
  int32_t grid;             // CTAs (persistent; one per SM by default)
  int32_t variant;          // launch shape (see kDecodeNumVariants)
  int32_t window;           // sliding window in keys (0: none)
  int32_t sinks;            // first keys that stay visible under a window, or -1: a call without sinks
  bool stable_inputs;       // caches, tables and lengths may be read before the wait
  float *logits;            // [S, H_q, logits_ld] (base 2, scaled) for key_scores, or null
  float *key_scores;        // [S, score_stride] or null; then lse is not null
  int64_t logits_ld, score_stride;
  float scale_log2;         // scale * log2(e)
};
cudaError_t launch_decode(const DecodeArgs &a, const CUtensorMap &k_map,
                          const CUtensorMap &v_map, const CUtensorMap &q_map,
                          const CUtensorMap &kn_map, const CUtensorMap &vn_map,
                          cudaStream_t stream);
cudaError_t take_decode_errors(cudaStream_t stream, uint32_t *flags);
cudaError_t decode_error_word(uint32_t **word);

// ---------------------------------------------------------------- prefill
struct PrefillArgs {
  const int32_t *cu_seqlens_q, *cu_seqlens_k;
  const int32_t *context_lens = nullptr;  // without a window: in place of cu_seqlens_k
  const int32_t *block_tables;
  void *out;
  float *lse;
  int32_t max_blocks;
  int32_t num_seqs, total_q, max_seqlen_q, max_seqlen_k;
  int32_t num_q_heads, num_kv_heads, head_dim, block_size;
  int32_t num_blocks;
  int32_t window;  // sliding window in keys (0: none)
  int32_t box_rows;  // rows per K/V TMA box: prefill_box_rows(block_size)
  int32_t num_sms;   // SMs of the device (persistent grid)
  int32_t total_k;   // segments end there at the latest, or -1: no such bound
  float scale_log2;
};
// Work items of one prefill call (row tiles x head pairs x sequences) are
// indexed with 32-bit integers, with headroom for the per-CTA walk.
constexpr int64_t kMaxPrefillItems = (int64_t{1} << 31) - (int64_t{1} << 20);
// Rows per K/V box of the prefill kernel: the largest of 128, 64, 32, 16 that
// divides the block size, so that a box never crosses a cache block and a
// 128-key tile takes as few copies as the block size allows.
inline int32_t prefill_box_rows(int32_t block_size) {
  int32_t r = 128;
  while (block_size % r != 0) r >>= 1;
  return r;
}
cudaError_t launch_prefill(const PrefillArgs &a, const CUtensorMap &q_map,
                           const CUtensorMap &k_map, const CUtensorMap &v_map,
                           cudaStream_t stream);
// pkv_paged_prefill_attn that also refuses segments of more than max_keys keys and, with
// total_k >= 0, those that lie outside [0, total_k) (and have queries).
pkv_status prefill_bounded(const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                           const int32_t *block_tables, int32_t max_blocks_per_seq, int32_t num_seqs,
                           int32_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k,
                           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                           int32_t block_size, int64_t num_blocks, float scale,
                           int32_t sliding_window, void *out, float *lse, int32_t max_keys,
                           int32_t total_k, void *stream);
cudaError_t take_prefill_errors(cudaStream_t stream, uint32_t *flags);
cudaError_t prefill_error_word(uint32_t **word);

// Division of a non-negative n < 2^31 by a fixed d >= 1 as a multiply and a
// shift: with l = ceil(log2 d) and mul = ceil(2^(31 + l) / d), n * mul / 2^(31 + l)
// exceeds n / d by less than n 2^l / (2^(31 + l) d) < 1 / d, so its floor is the
// quotient's.
struct FastDiv {
  uint32_t mul, shift, d;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((uint64_t{1} << l) < d) ++l;
  const uint64_t mul = ((uint64_t{1} << (31 + l)) + d - 1) / d;  // < 2^32, since d > 2^(l - 1)
  return {static_cast<uint32_t>(mul), 31 + l, d};
}
#ifdef __CUDACC__
__device__ __forceinline__ uint32_t fast_quotient(uint32_t n, const FastDiv &f) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * f.mul) >> f.shift);
}
#endif

// ---------------------------------------------------------------- 4-bit cache
struct Q4CacheArgs {
  void *k_codes, *k_params, *v_codes, *v_params;
  int32_t num_kv_heads, group_size, block_size;
  int64_t num_blocks;
};
struct Q4RowsArgs {
  Q4CacheArgs cache;
  const void *k, *v;      // store: the rows
  void *k_out, *v_out;    // load: where they go
  const int32_t *slots;
  int32_t num_tokens;
};
cudaError_t launch_q4_store(const Q4RowsArgs &a, cudaStream_t stream);
cudaError_t launch_q4_load(const Q4RowsArgs &a, cudaStream_t stream);

constexpr int32_t kQ4PrefillBlock = 128;  // rows of a workspace block: one K/V tile of the prefill kernel
struct Q4GatherArgs {
  Q4CacheArgs cache;
  const int32_t *cu_seqlens_q, *cu_seqlens_k, *block_tables;
  void *ws_k, *ws_v;
  int32_t *ws_tables;
  int32_t max_blocks, ws_max_blocks, num_seqs, max_seqlen_q, max_seqlen_k, total_k;
  int32_t window, num_sms;
};
cudaError_t launch_q4_gather(const Q4GatherArgs &a, cudaStream_t stream);
cudaError_t q4_cache_error_word(uint32_t **word);

// How a decode call over the 4-bit cache shares its work out: a CTA of `warps`
// (4, 8 or 16) warps for each (sequence, KV head), or, with range_ctas > 0, equal
// ranges for the 16 warps of each of that many CTAs.
constexpr int kQ4MaxRangeSeqs = 1024;  // sequences whose lengths fit beside the rings
struct Q4DecodePlan {
  int32_t warps, range_ctas;
};
struct Q4DecodeArgs {
  Q4CacheArgs cache;
  const void *q;
  const int32_t *block_tables, *context_lens;
  const int32_t *table_rows;  // table row of each sequence, or null; with it, length 0 raises nothing
  void *out;
  float *lse;             // required when key_scores is given
  float *ws_o, *ws_ml;    // split partials
  float *logits;          // [S, H_q, logits_ld], with key_scores
  float *key_scores;      // [S, score_stride] or null
  int64_t logits_ld, score_stride;
  int32_t max_blocks, max_context_len, num_seqs, num_q_heads;
  int32_t window;
  Q4DecodePlan plan;
  float scale_log2;
};
// Prefill by rows: fills context_lens and table_rows [total_q] for a decode launch.
struct Q4PrefillRowsArgs {
  const int32_t *cu_seqlens_q, *cu_seqlens_k;
  int32_t *context_lens, *table_rows;
  int32_t num_seqs, total_q, total_k, max_seqlen_q, max_seqlen_k, max_blocks, block_size;
};
cudaError_t launch_q4_prefill_rows(const Q4PrefillRowsArgs &a, cudaStream_t stream);
cudaError_t launch_q4_decode(const Q4DecodeArgs &a, cudaStream_t stream);
cudaError_t q4_decode_error_word(uint32_t **word);

// ---------------------------------------------------------------- eviction
struct EvictSelectArgs {
  const float *key_scores;
  int64_t score_stride;
  const int32_t *context_lens;
  int32_t *keep, *new_lens;
  int32_t max_context_len, num_seqs, budget, recent;
  bool mark_invalid;  // a sequence of invalid length gets -1 everywhere
};
cudaError_t launch_evict_select(const EvictSelectArgs &a, cudaStream_t stream);

// An array of cache rows: [num_blocks, planes, block_size] rows of row_bytes.
struct RowArray {
  void *base;
  int32_t planes, row_bytes;
  int64_t block_bytes;  // of all planes; set by the launch
};
constexpr int kMaxRowArrays = 4;
constexpr int kSliceBytes = 64;  // bytes of a row that one CTA of an in-place compaction moves, at most
struct EvictCompactArgs {
  RowArray arrays[kMaxRowArrays];
  int32_t num_arrays;
  const int32_t *src_tables, *dst_tables, *keep, *new_lens;
  const float *key_scores;
  float *dst_key_scores;
  int64_t score_stride, dst_score_stride;
  int32_t src_max_blocks, dst_max_blocks, budget, num_seqs, block_size, num_blocks, num_sms;
};
cudaError_t launch_evict_compact(const EvictCompactArgs &a, cudaStream_t stream);
cudaError_t evict_error_word(uint32_t **word);

// ---------------------------------------------------------------- queries and keys
struct HeadsArgs {
  const void *q, *k, *v, *q_weight, *k_weight;
  void *q_out, *k_out, *v_out;   // with slots: q's rows and the two caches
  const int32_t *positions, *slots;
  const pkv_rope *rope;          // host, or null
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int64_t num_slots;
  int32_t num_tokens, num_q_heads, num_kv_heads;
  int num_sms;
  float eps;
};
cudaError_t launch_heads(const HeadsArgs &a, cudaStream_t stream);
cudaError_t heads_error_word(uint32_t **word);

// ---------------------------------------------------------------- chunks
constexpr int kChunkMaxSeqs = 1024;  // sequences per call (their list fits in shared memory)
constexpr int kChunkMaxCtas = 384;    // one per SM, as many as share out the work in one block's threads
// A tile of 128 query rows whose keys are cut between CTAs, as the joining kernel reads it.
struct ChunkCut {
  int32_t pieces;  // 0: none
  int32_t slot0;   // of the first piece; piece x is in slot 2 (slot0 / 2 + x)
  int32_t head, row, n_tok;
};
struct ChunkArgs {
  const int32_t *cu_seqlens_q, *context_lens, *block_tables;
  void *out;
  float *lse;
  float *ws_o, *ws_ml;  // [2 num_ctas, 128, 128], [2 num_ctas, 128, 4]
  ChunkCut *cuts;       // [num_ctas]
  int32_t max_blocks, num_seqs, total_q, max_seqlen_q, max_context_len;
  int32_t num_q_heads, num_kv_heads, block_size, num_blocks;
  int32_t window, sinks;  // sinks: 0 without a window
  int32_t num_ctas;
  float scale_log2;
};
cudaError_t launch_chunk(const ChunkArgs &a, const CUtensorMap &q_map, const CUtensorMap &k_map,
                         const CUtensorMap &v_map, cudaStream_t stream);
cudaError_t chunk_error_word(uint32_t **word);

// ---------------------------------------------------------------- shared by the C entries
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
constexpr float kLog2e = 1.4426950408889634f;
// Longest context of the calls on 4-bit caches and of eviction: their kernels
// step through positions in 32 bits.
constexpr int32_t kMaxContext = 1 << 30;
// Whether the logits of a call with accumulated weights have a size that a
// workspace can have at all (2^40 values), before sizes are multiplied out.
inline bool logits_fit(int64_t num_seqs, int64_t num_q_heads, int64_t max_context_len) {
  return num_seqs * num_q_heads <= (int64_t{1} << 40) / (max_context_len + 15);
}

}  // namespace pkv
