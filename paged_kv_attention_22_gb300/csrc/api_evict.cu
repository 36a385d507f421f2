// The C entries of eviction by accumulated attention weight (declared in
// include/pkv.h): argument checks and launches.
#include "pkv.h"
#include "internal.h"

namespace {

using pkv::aligned16;
using pkv::cuda_fail;
using pkv::current_sm_count;

constexpr int32_t kMaxBudget = 1 << 29;  // the kernels count kept positions, four arrays of them, in 32 bits

constexpr int32_t kMaxSeqs = 1 << 27;    // of a selection: eight CTAs each

// The two selections; mark_invalid: the second's -1 for sequences of invalid length.
pkv_status select(const float *key_scores, int64_t score_stride, const int32_t *context_lens, int32_t max_context_len,
                  int32_t num_seqs, int32_t budget, int32_t recent, int32_t *keep, int32_t *new_lens, bool mark_invalid,
                  void *stream) {
  if (num_seqs < 0 || budget <= 0 || recent < 0 || recent > budget || max_context_len <= 0 ||
      score_stride < max_context_len)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs > 0 && (key_scores == nullptr || context_lens == nullptr || keep == nullptr || new_lens == nullptr))
    return PKV_ERR_INVALID_ARG;
  if (max_context_len > pkv::kMaxContext || budget > kMaxBudget || num_seqs > kMaxSeqs) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  int sms = 0;
  pkv_status st = current_sm_count(&sms);
  if (st != PKV_OK) return st;
  pkv::EvictSelectArgs a;
  a.key_scores = key_scores;
  a.score_stride = score_stride;
  a.context_lens = context_lens;
  a.keep = keep;
  a.new_lens = new_lens;
  a.max_context_len = max_context_len;
  a.num_seqs = num_seqs;
  a.budget = budget;
  a.recent = recent;
  a.mark_invalid = mark_invalid;
  cudaError_t e = pkv::launch_evict_select(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "evict_select launch");
  return PKV_OK;
}

// Checks shared by the two compactions; the arrays are already in `a`.
pkv_status compact(pkv::EvictCompactArgs &a, const int32_t *src_tables, int32_t src_max_blocks,
                   const int32_t *dst_tables, int32_t dst_max_blocks, const int32_t *keep, int32_t budget,
                   const int32_t *new_lens, int32_t num_seqs, int32_t block_size, int64_t num_blocks,
                   const float *key_scores, int64_t score_stride, float *dst_key_scores, int64_t dst_score_stride,
                   void *stream) {
  for (int k = 0; k < a.num_arrays; ++k) {
    if (a.arrays[k].base == nullptr || !aligned16(a.arrays[k].base)) return PKV_ERR_INVALID_ARG;
  }
  if (num_seqs < 0 || budget <= 0 || src_max_blocks <= 0 || dst_max_blocks <= 0 || block_size <= 0 || num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs > 0 && (src_tables == nullptr || dst_tables == nullptr || keep == nullptr || new_lens == nullptr))
    return PKV_ERR_INVALID_ARG;
  if ((key_scores == nullptr) != (dst_key_scores == nullptr)) return PKV_ERR_INVALID_ARG;
  if (key_scores != nullptr && (score_stride <= 0 || dst_score_stride <= 0)) return PKV_ERR_INVALID_ARG;
  // one score array under two row strides would be overwritten while it is read
  if (key_scores != nullptr && key_scores == dst_key_scores && score_stride != dst_score_stride)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs > 65535 || budget > kMaxBudget) return PKV_ERR_UNSUPPORTED;
  if (num_blocks > INT32_MAX || num_blocks * block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  int sms = 0;
  pkv_status st = current_sm_count(&sms);
  if (st != PKV_OK) return st;
  a.src_tables = src_tables;
  a.dst_tables = dst_tables;
  a.keep = keep;
  a.new_lens = new_lens;
  a.key_scores = key_scores;
  a.dst_key_scores = dst_key_scores;
  a.score_stride = score_stride;
  a.dst_score_stride = dst_score_stride;
  a.src_max_blocks = src_max_blocks;
  a.dst_max_blocks = dst_max_blocks;
  a.budget = budget;
  a.num_seqs = num_seqs;
  a.block_size = block_size;
  a.num_blocks = static_cast<int32_t>(num_blocks);
  a.num_sms = sms;
  cudaError_t e = pkv::launch_evict_compact(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "evict_compact launch");
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_evict_select(const float *key_scores, int64_t score_stride, const int32_t *context_lens,
                            int32_t max_context_len, int32_t num_seqs, int32_t budget, int32_t recent, int32_t *keep,
                            int32_t *new_lens, void *stream) {
  return select(key_scores, score_stride, context_lens, max_context_len, num_seqs, budget, recent, keep, new_lens, false,
                stream);
}

pkv_status pkv_evict_select_new(const float *key_scores, int64_t score_stride, const int32_t *context_lens,
                                int32_t max_context_len, int32_t num_seqs, int32_t budget, int32_t recent, int32_t *keep,
                                int32_t *new_lens, void *stream) {
  return select(key_scores, score_stride, context_lens, max_context_len, num_seqs, budget, recent, keep, new_lens, true,
                stream);
}

pkv_status pkv_evict_compact(void *k_cache, void *v_cache, const int32_t *src_tables, int32_t src_max_blocks,
                             const int32_t *dst_tables, int32_t dst_max_blocks, const int32_t *keep, int32_t budget,
                             const int32_t *new_lens, int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim,
                             int32_t block_size, int64_t num_blocks, const float *key_scores, int64_t score_stride,
                             float *dst_key_scores, int64_t dst_score_stride, void *stream) {
  if (num_kv_heads <= 0 || head_dim <= 0) return PKV_ERR_INVALID_ARG;
  if (head_dim != 128 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  pkv::EvictCompactArgs a;
  a.num_arrays = 2;
  a.arrays[0] = {k_cache, 1, num_kv_heads * head_dim * 2};
  a.arrays[1] = {v_cache, 1, num_kv_heads * head_dim * 2};
  return compact(a, src_tables, src_max_blocks, dst_tables, dst_max_blocks, keep, budget, new_lens, num_seqs,
                 block_size, num_blocks, key_scores, score_stride, dst_key_scores, dst_score_stride, stream);
}

pkv_status pkv_evict_compact_q4(void *k_codes, void *k_params, void *v_codes, void *v_params,
                                const int32_t *src_tables, int32_t src_max_blocks, const int32_t *dst_tables,
                                int32_t dst_max_blocks, const int32_t *keep, int32_t budget, const int32_t *new_lens,
                                int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t group_size,
                                int32_t block_size, int64_t num_blocks, const float *key_scores,
                                int64_t score_stride, float *dst_key_scores, int64_t dst_score_stride, void *stream) {
  if (num_kv_heads <= 0 || head_dim <= 0 || group_size <= 0) return PKV_ERR_INVALID_ARG;
  if (head_dim != 128 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  if (group_size != 32 && group_size != 64 && group_size != 128) return PKV_ERR_UNSUPPORTED;
  pkv::EvictCompactArgs a;
  a.num_arrays = 4;
  a.arrays[0] = {k_codes, num_kv_heads, 64};
  a.arrays[1] = {v_codes, num_kv_heads, 64};
  a.arrays[2] = {k_params, num_kv_heads, 512 / group_size};
  a.arrays[3] = {v_params, num_kv_heads, 512 / group_size};
  return compact(a, src_tables, src_max_blocks, dst_tables, dst_max_blocks, keep, budget, new_lens, num_seqs,
                 block_size, num_blocks, key_scores, score_stride, dst_key_scores, dst_score_stride, stream);
}

}  // extern "C"
