// The C entries of the 4-bit cache (declared in include/pkv.h): argument checks,
// workspace layout and launch planning. Allocates nothing; every call only
// enqueues work on the caller's stream.
#include <algorithm>
#include <cmath>

#include "pkv.h"
#include "internal.h"

namespace {

using pkv::align_up;
using pkv::aligned16;
using pkv::cuda_fail;
using pkv::current_sm_count;

constexpr int32_t kD = 128;

// Sizes and pointers of a 4-bit cache.
pkv_status check_cache(const pkv::Q4CacheArgs &c, int32_t head_dim) {
  if (c.k_codes == nullptr || c.k_params == nullptr || c.v_codes == nullptr || c.v_params == nullptr)
    return PKV_ERR_INVALID_ARG;
  if (c.num_kv_heads <= 0 || c.block_size <= 0 || c.num_blocks <= 0 || head_dim <= 0 || c.group_size <= 0)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kD) return PKV_ERR_UNSUPPORTED;
  if (c.group_size != 32 && c.group_size != 64 && c.group_size != 128) return PKV_ERR_UNSUPPORTED;
  if (c.num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  // slots are int32; num_blocks first, so that the product cannot overflow
  if (c.num_blocks > INT32_MAX || c.num_blocks * c.block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (!aligned16(c.k_codes) || !aligned16(c.k_params) || !aligned16(c.v_codes) || !aligned16(c.v_params))
    return PKV_ERR_INVALID_ARG;
  return PKV_OK;
}

// What the attention calls need beyond check_cache. max_gqa: the largest number
// of query heads a KV head.
pkv_status check_attention(const pkv::Q4CacheArgs &c, int32_t num_q_heads, int32_t max_blocks, int32_t max_gqa) {
  if (num_q_heads <= 0 || max_blocks <= 0) return PKV_ERR_INVALID_ARG;
  if (num_q_heads % c.num_kv_heads != 0 || num_q_heads > 65535) return PKV_ERR_UNSUPPORTED;
  const int32_t G = num_q_heads / c.num_kv_heads;
  if (G > max_gqa || (G & (G - 1)) != 0) return PKV_ERR_UNSUPPORTED;
  if (c.block_size % 16 != 0) return PKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_blocks) * c.block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  // the decode kernel holds a row's index / 16 in 32 bits
  if (c.num_blocks * c.block_size / 16 * c.num_kv_heads >= 0xffffffffll) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

// The plan of a decode call, by the least estimated time. With a step of 32 keys
// as the unit, an SM with 4, 8, 12 or 16 resident warps gets through 4.7, 6.4, 7.4
// or 8 steps a microsecond (measured with 16 x 8 pairs of 16,384 keys; 16 warps
// are the most its registers hold). A CTA for each pair costs some 2 us to start
// and finish, which its neighbours on the SM cover in part; ranges cost the scan
// of the lengths and the merge kernel.
// The estimate takes every sequence at the longest. Where they are not, ranges
// stay even, and one CTA a pair may be left with most of the work: pairs of more
// than kWarpKeys keys a warp always go by ranges.
constexpr int32_t kStepKeys = 32, kWarpKeys = 1024;

pkv::Q4DecodePlan decode_plan(int64_t num_seqs, int64_t heads, int64_t keys, int sms) {
  const int64_t steps = (keys + kStepKeys - 1) / kStepKeys, pairs = num_seqs * heads;
  pkv::Q4DecodePlan best = {16, 0};
  double best_us = 0;
  for (int warps = 4; warps <= 16; warps *= 2) {
    const int64_t per_sm = (pairs + sms - 1) / sms, per_warp = (steps + warps - 1) / warps;
    const int64_t resident = std::min<int64_t>(16, per_sm * warps);
    const double rate = resident <= 4 ? 4.7 : resident <= 8 ? 6.4 : resident <= 12 ? 7.4 : 8.0;
    const double rounds = std::max(1.0, static_cast<double>(per_sm * warps) / 16);
    const double us = per_sm * per_warp * warps / rate + 2 * rounds + (warps == 16 ? 0.8 : 0.0);
    if (warps == 4 || us < best_us) {
      best.warps = warps;
      best_us = us;
    }
  }
  if (num_seqs <= pkv::kQ4MaxRangeSeqs) {
    const double per_warp = static_cast<double>(pairs * steps) / (16 * sms);
    const double us = std::max(1.0, per_warp) * 2.0 + 7;
    if (us < best_us || keys > kWarpKeys * best.warps) best.range_ctas = sms;
  }
  return best;
}

struct DecodeWorkspace {
  size_t o, ml, lse, logits, total;
  int64_t logits_ld;
};

DecodeWorkspace decode_workspace(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t max_context_len,
                                 bool with_scores, int sms) {
  DecodeWorkspace w;
  // two pieces of a range a warp, 16 warps an SM, whatever the sequences
  const int64_t pieces = static_cast<int64_t>(sms) * 16 * 2 * (num_q_heads / num_kv_heads);
  const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads;
  w.logits_ld = static_cast<int64_t>(align_up(static_cast<size_t>(max_context_len), 16));
  w.o = 0;
  w.ml = w.o + static_cast<size_t>(pieces) * kD * sizeof(float);
  w.lse = w.ml + static_cast<size_t>(pieces) * 4 * sizeof(float);
  w.logits = w.lse + (with_scores ? align_up(rows * sizeof(float), 256) : 0);
  w.total = w.logits + (with_scores ? rows * static_cast<size_t>(w.logits_ld) * sizeof(float) : 0);
  return w;
}

struct PrefillWorkspace {
  size_t tables, k, v, total;
  int32_t max_blocks;
  int64_t num_blocks;
};

PrefillWorkspace prefill_workspace(int32_t num_seqs, int32_t total_k, int32_t max_seqlen_k, int32_t num_kv_heads) {
  constexpr int64_t B = pkv::kQ4PrefillBlock;
  PrefillWorkspace w;
  w.max_blocks = static_cast<int32_t>((static_cast<int64_t>(max_seqlen_k) + B - 1) / B);
  w.num_blocks = (static_cast<int64_t>(total_k) + B - 1) / B + num_seqs;
  const size_t cache = static_cast<size_t>(w.num_blocks) * B * num_kv_heads * kD * 2;
  w.tables = 0;
  w.k = align_up(static_cast<size_t>(num_seqs) * w.max_blocks * sizeof(int32_t), 256);
  w.v = w.k + cache;
  w.total = w.v + cache;
  return w;
}

pkv::Q4CacheArgs cache_args(const void *k_codes, const void *k_params, const void *v_codes, const void *v_params,
                            int32_t num_kv_heads, int32_t group_size, int32_t block_size, int64_t num_blocks) {
  return {const_cast<void *>(k_codes), const_cast<void *>(k_params), const_cast<void *>(v_codes),
          const_cast<void *>(v_params), num_kv_heads, group_size, block_size, num_blocks};
}

}  // namespace

extern "C" {

pkv_status pkv_kv_store_q4(const void *k, const void *v, void *k_codes, void *k_params, void *v_codes, void *v_params,
                           const int32_t *slot_mapping, int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                           int32_t group_size, int32_t block_size, int64_t num_blocks, void *stream) {
  pkv::Q4RowsArgs a = {};
  a.cache = cache_args(k_codes, k_params, v_codes, v_params, num_kv_heads, group_size, block_size, num_blocks);
  pkv_status st = check_cache(a.cache, head_dim);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || !aligned16(k) || !aligned16(v)) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (k == nullptr || v == nullptr || slot_mapping == nullptr) return PKV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_tokens) * num_kv_heads > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  a.k = k;
  a.v = v;
  a.slots = slot_mapping;
  a.num_tokens = num_tokens;
  cudaError_t e = pkv::launch_q4_store(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_store_q4 launch");
  return PKV_OK;
}

pkv_status pkv_kv_load_q4(const void *k_codes, const void *k_params, const void *v_codes, const void *v_params,
                          const int32_t *slots, void *k, void *v, int32_t num_tokens, int32_t num_kv_heads,
                          int32_t head_dim, int32_t group_size, int32_t block_size, int64_t num_blocks,
                          void *stream) {
  pkv::Q4RowsArgs a = {};
  a.cache = cache_args(k_codes, k_params, v_codes, v_params, num_kv_heads, group_size, block_size, num_blocks);
  pkv_status st = check_cache(a.cache, head_dim);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || !aligned16(k) || !aligned16(v)) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (k == nullptr || v == nullptr || slots == nullptr) return PKV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_tokens) * num_kv_heads > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  a.k_out = k;
  a.v_out = v;
  a.slots = slots;
  a.num_tokens = num_tokens;
  cudaError_t e = pkv::launch_q4_load(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_load_q4 launch");
  return PKV_OK;
}

size_t pkv_decode_q4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                    int32_t max_context_len, int32_t with_scores) {
  if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim != kD || max_context_len <= 0 ||
      num_q_heads % num_kv_heads != 0 || max_context_len > pkv::kMaxContext ||
      (with_scores != 0 && !pkv::logits_fit(num_seqs, num_q_heads, max_context_len)))
    return 0;
  int sms = 0;
  if (current_sm_count(&sms) != PKV_OK) return 0;
  return decode_workspace(num_seqs, num_q_heads, num_kv_heads, max_context_len, with_scores != 0, sms).total;
}

pkv_status pkv_paged_decode_attn_q4(const void *q, const void *k_codes, const void *k_params, const void *v_codes,
                                    const void *v_params, const int32_t *block_tables, int32_t max_blocks_per_seq,
                                    const int32_t *context_lens, int32_t max_context_len, int32_t num_seqs,
                                    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t group_size,
                                    int32_t block_size, int64_t num_blocks, float scale, int32_t sliding_window,
                                    void *out, float *lse, float *key_scores, int64_t score_stride, void *workspace,
                                    size_t workspace_bytes, void *stream) {
  if (q == nullptr || block_tables == nullptr || context_lens == nullptr || out == nullptr)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs <= 0 || max_context_len <= 0 || !std::isfinite(scale) || sliding_window < 0)
    return PKV_ERR_INVALID_ARG;
  if (key_scores != nullptr && score_stride < max_context_len) return PKV_ERR_INVALID_ARG;
  pkv::Q4DecodeArgs a = {};
  a.cache = cache_args(k_codes, k_params, v_codes, v_params, num_kv_heads, group_size, block_size, num_blocks);
  pkv_status st = check_cache(a.cache, head_dim);
  if (st != PKV_OK) return st;
  if ((st = check_attention(a.cache, num_q_heads, max_blocks_per_seq, 8)) != PKV_OK) return st;
  if (num_seqs > 65535 || max_context_len > pkv::kMaxContext) return PKV_ERR_UNSUPPORTED;
  if (key_scores != nullptr && !pkv::logits_fit(num_seqs, num_q_heads, max_context_len)) return PKV_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(out)) return PKV_ERR_INVALID_ARG;
  if (workspace == nullptr) return PKV_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_sm_count(&sms)) != PKV_OK) return st;
  const DecodeWorkspace w =
      decode_workspace(num_seqs, num_q_heads, num_kv_heads, max_context_len, key_scores != nullptr, sms);
  if (workspace_bytes < w.total) return PKV_ERR_WORKSPACE_TOO_SMALL;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  // with a window, each sequence's keys start at the 16-key boundary at or
  // before its first one
  const int64_t keys = sliding_window > 0 ? std::min<int64_t>(max_context_len, static_cast<int64_t>(sliding_window) + 15)
                                          : max_context_len;
  a.q = q;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.out = out;
  a.lse = lse != nullptr || key_scores == nullptr ? lse : reinterpret_cast<float *>(ws + w.lse);
  a.ws_o = reinterpret_cast<float *>(ws + w.o);
  a.ws_ml = reinterpret_cast<float *>(ws + w.ml);
  a.logits = key_scores != nullptr ? reinterpret_cast<float *>(ws + w.logits) : nullptr;
  a.key_scores = key_scores;
  a.logits_ld = w.logits_ld;
  a.score_stride = score_stride;
  a.max_blocks = max_blocks_per_seq;
  a.max_context_len = max_context_len;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.window = sliding_window;
  a.plan = decode_plan(num_seqs, num_kv_heads, keys, sms);
  a.scale_log2 = scale * pkv::kLog2e;
  cudaError_t e = pkv::launch_q4_decode(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "decode_q4 launch");
  return PKV_OK;
}

size_t pkv_prefill_q4_workspace_size(int32_t num_seqs, int32_t total_k, int32_t max_seqlen_k, int32_t num_kv_heads,
                                     int32_t head_dim) {
  if (num_seqs <= 0 || total_k < 0 || max_seqlen_k < 0 || num_kv_heads <= 0 || head_dim != kD) return 0;
  return prefill_workspace(num_seqs, total_k, max_seqlen_k, num_kv_heads).total;
}

pkv_status pkv_paged_prefill_attn_q4(const void *q, const void *k_codes, const void *k_params, const void *v_codes,
                                     const void *v_params, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                     const int32_t *block_tables, int32_t max_blocks_per_seq, int32_t num_seqs,
                                     int32_t total_q, int32_t total_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t group_size,
                                     int32_t block_size, int64_t num_blocks, float scale, int32_t sliding_window,
                                     void *out, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  if (cu_seqlens_q == nullptr || cu_seqlens_k == nullptr || block_tables == nullptr) return PKV_ERR_INVALID_ARG;
  if (num_seqs < 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || !std::isfinite(scale) ||
      sliding_window < 0 || max_seqlen_q > max_seqlen_k)
    return PKV_ERR_INVALID_ARG;
  pkv::Q4GatherArgs g = {};
  g.cache = cache_args(k_codes, k_params, v_codes, v_params, num_kv_heads, group_size, block_size, num_blocks);
  pkv_status st = check_cache(g.cache, head_dim);
  if (st != PKV_OK) return st;
  if ((st = check_attention(g.cache, num_q_heads, max_blocks_per_seq, 4)) != PKV_OK) return st;
  if (num_seqs > 65535) return PKV_ERR_UNSUPPORTED;
  if (total_q > 0 && (q == nullptr || out == nullptr)) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return PKV_OK;
  if (!aligned16(q) || !aligned16(out)) return PKV_ERR_INVALID_ARG;
  const PrefillWorkspace w = prefill_workspace(num_seqs, total_k, max_seqlen_k, num_kv_heads);
  // workspace rows are 32-bit TMA coordinates; units of 16 keys x heads are counted in 31 bits
  if (w.num_blocks * pkv::kQ4PrefillBlock > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if ((static_cast<int64_t>(max_seqlen_k) / 16 + 1) * num_kv_heads > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < w.total) return PKV_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_sm_count(&sms)) != PKV_OK) return st;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  g.cu_seqlens_q = cu_seqlens_q;
  g.cu_seqlens_k = cu_seqlens_k;
  g.block_tables = block_tables;
  g.ws_k = ws + w.k;
  g.ws_v = ws + w.v;
  g.ws_tables = reinterpret_cast<int32_t *>(ws + w.tables);
  g.max_blocks = max_blocks_per_seq;
  g.ws_max_blocks = w.max_blocks;
  g.num_seqs = num_seqs;
  g.max_seqlen_q = max_seqlen_q;
  g.max_seqlen_k = max_seqlen_k;
  g.total_k = total_k;
  g.window = sliding_window;
  g.num_sms = sms;
  cudaError_t e = pkv::launch_q4_gather(g, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "prefill_q4 widening launch");
  return pkv_paged_prefill_attn(q, g.ws_k, g.ws_v, cu_seqlens_q, cu_seqlens_k, g.ws_tables, w.max_blocks, num_seqs,
                                total_q, max_seqlen_q, max_seqlen_k, num_q_heads, num_kv_heads, head_dim,
                                pkv::kQ4PrefillBlock, w.num_blocks, scale, sliding_window, out, lse, nullptr, 0,
                                stream);
}

}  // extern "C"
