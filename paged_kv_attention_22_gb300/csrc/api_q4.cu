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
// are the most its registers hold). The first CTAs of an SM cost 5 us to start
// and finish; later ones, which start while others run, 2.5 for each round. Ranges
// take 2.1 us a step and warp, 9 for the scan of the lengths and the merge kernel,
// and 11 for every pair that a warp finishes. Estimated and measured, in us, with 4
// warps a pair, 8, 16 and by ranges:
//     512 pairs of   640 keys   15/16    18/19    23/-     22/22
//     128 pairs of 16,384       114/-    85/-     70/68    66/66
//     184 pairs of 1,015        15/13    15/13    16/16    16/16
//   4,096 pairs of   128        33/32    50/52    84/102   42/44
//   2,400 pairs of 2,048       141/138  151/150  171/188  154/154
// The estimate takes every sequence at the longest. Where they are not, ranges
// stay even, and one CTA a pair may be left with most of the work: pairs of more
// than kWarpKeys keys a warp go by ranges, in calls of at most kQ4MaxRangeSeqs
// sequences. Above that there is no list of steps to cut, and one long sequence among
// short ones runs on one CTA a KV head to its end.
constexpr int32_t kStepKeys = 32, kWarpKeys = 1024;

struct PlannedDecode {
  pkv::Q4DecodePlan plan;
  double us;
};

PlannedDecode decode_plan(int64_t num_seqs, int64_t heads, int64_t keys, int sms) {
  const int64_t steps = (keys + kStepKeys - 1) / kStepKeys, pairs = num_seqs * heads;
  PlannedDecode best = {{16, 0}, 0};
  for (int warps = 4; warps <= 16; warps *= 2) {
    const int64_t per_sm = (pairs + sms - 1) / sms, per_warp = (steps + warps - 1) / warps;
    const int64_t resident = std::min<int64_t>(16, per_sm * warps);
    const double rate = resident <= 4 ? 4.7 : resident <= 8 ? 6.4 : resident <= 12 ? 7.4 : 8.0;
    const double rounds = std::max(1.0, static_cast<double>(per_sm * warps) / 16);
    const double work = static_cast<double>(std::max(per_warp * resident, per_sm * steps)) / rate;
    const double us = work + 2.5 + 2.5 * rounds + (warps == 16 ? 0.8 : 0.0);
    if (warps == 4 || us < best.us) {
      best.plan.warps = warps;
      best.us = us;
    }
  }
  if (num_seqs <= pkv::kQ4MaxRangeSeqs) {
    const int64_t warps = 16 * static_cast<int64_t>(sms), per_warp = (pairs * steps + warps - 1) / warps;
    const double us = 2.1 * per_warp + 9 + 11.0 * pairs / warps;
    if (us < best.us || keys > kWarpKeys * best.plan.warps) {
      best.plan.range_ctas = sms;
      best.us = us;
    }
  }
  return best;
}

// Keys of the longest sequence that are read: with a window they start at the
// 16-key boundary at or before its first one.
int64_t window_keys(int64_t keys, int32_t window) {
  return window > 0 ? std::min<int64_t>(keys, static_cast<int64_t>(window) + 15) : keys;
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

// Prefill goes one of two ways. By rows, each query row is a decode of its own
// over the codes: for few new tokens over many keys. Widened, the keys are made
// bf16 once and the tensor-core prefill kernel reads them; there a (segment, two
// query heads) is one CTA that passes all its keys, 128 in 1.4 us. Measured, in us,
// by rows and widened: 8 segments of 8,192 keys with 1 query token each 28 and 150,
// with 8 127 and 150, with 16 239 and 150; one of 32,768 keys with 16 tokens 124
// and 390; 64 of 128 keys with 4 tokens 18 and 34, with 8 30 and 34; prompts alone, 4
// of 9 tokens 6.3 and 10.8, of 32 8.7 and 10.6, of 64 14.5 and 10.8.
constexpr int32_t kRowsMaxQ = 64;   // query tokens a segment by rows, at most (a workspace bound)

bool prefill_by_rows(int64_t num_seqs, int64_t total_q, int64_t max_q, int64_t total_k, int64_t keys, int64_t q_heads,
                     int64_t kv_heads, int sms) {
  if (max_q > kRowsMaxQ || total_q > std::min<int64_t>(65535, num_seqs * kRowsMaxQ)) return false;
  const double rows_us = 2 + decode_plan(total_q, kv_heads, keys, sms).us;
  const double widen_us = std::min<double>(total_k, static_cast<double>(num_seqs) * keys) * kv_heads * 672 / 6.2e6;
  const int64_t ctas = num_seqs * (q_heads > kv_heads ? q_heads / 2 : q_heads);
  const double attend_us = (ctas + sms - 1) / sms * (4 + keys / 128 * 1.4);
  return rows_us < 6.5 + widen_us + attend_us;
}

struct PrefillWorkspace {
  size_t tables, k, v;               // widened
  size_t lens, rows, o, ml;          // by rows
  size_t total;
  int32_t max_blocks;
  int64_t num_blocks;
};

PrefillWorkspace prefill_workspace(int32_t num_seqs, int32_t total_k, int32_t max_seqlen_k, int32_t num_kv_heads,
                                   int sms) {
  constexpr int64_t B = pkv::kQ4PrefillBlock;
  PrefillWorkspace w;
  w.max_blocks = static_cast<int32_t>((static_cast<int64_t>(max_seqlen_k) + B - 1) / B);
  w.num_blocks = (static_cast<int64_t>(total_k) + B - 1) / B + num_seqs;
  const size_t cache = static_cast<size_t>(w.num_blocks) * B * num_kv_heads * kD * 2;
  w.tables = 0;
  w.k = align_up(static_cast<size_t>(num_seqs) * w.max_blocks * sizeof(int32_t), 256);
  w.v = w.k + cache;
  const size_t most_rows = align_up(static_cast<size_t>(num_seqs) * kRowsMaxQ * sizeof(int32_t), 256);
  const size_t pieces = static_cast<size_t>(sms) * 16 * 2 * 4;  // of up to 4 query heads a KV head
  w.lens = 0;
  w.rows = most_rows;
  w.o = 2 * most_rows;
  w.ml = w.o + pieces * kD * sizeof(float);
  w.total = std::max(w.v + cache, w.ml + pieces * 4 * sizeof(float));
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
  a.plan = decode_plan(num_seqs, num_kv_heads, window_keys(max_context_len, sliding_window), sms).plan;
  a.scale_log2 = scale * pkv::kLog2e;
  cudaError_t e = pkv::launch_q4_decode(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "decode_q4 launch");
  return PKV_OK;
}

size_t pkv_prefill_q4_workspace_size(int32_t num_seqs, int32_t total_k, int32_t max_seqlen_k, int32_t num_kv_heads,
                                     int32_t head_dim) {
  if (num_seqs <= 0 || total_k < 0 || max_seqlen_k < 0 || num_kv_heads <= 0 || head_dim != kD) return 0;
  int sms = 0;
  if (current_sm_count(&sms) != PKV_OK) return 0;
  return prefill_workspace(num_seqs, total_k, max_seqlen_k, num_kv_heads, sms).total;
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
  if (workspace == nullptr) return PKV_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
  // workspace rows are 32-bit TMA coordinates; units of 16 keys x heads are counted in 31 bits
  if (((static_cast<int64_t>(total_k) + pkv::kQ4PrefillBlock - 1) / pkv::kQ4PrefillBlock + num_seqs) *
          pkv::kQ4PrefillBlock > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  if ((static_cast<int64_t>(max_seqlen_k) / 16 + 1) * num_kv_heads > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (workspace_bytes < prefill_workspace(num_seqs, total_k, max_seqlen_k, num_kv_heads, 0).total)
    return PKV_ERR_WORKSPACE_TOO_SMALL;  // for any device
  int sms = 0;
  if ((st = current_sm_count(&sms)) != PKV_OK) return st;
  const PrefillWorkspace w = prefill_workspace(num_seqs, total_k, max_seqlen_k, num_kv_heads, sms);
  if (workspace_bytes < w.total) return PKV_ERR_WORKSPACE_TOO_SMALL;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  if (max_seqlen_k <= pkv::kMaxContext &&
      prefill_by_rows(num_seqs, total_q, max_seqlen_q, total_k, window_keys(max_seqlen_k, sliding_window), num_q_heads,
                      num_kv_heads, sms)) {
    pkv::Q4PrefillRowsArgs r = {};
    r.cu_seqlens_q = cu_seqlens_q;
    r.cu_seqlens_k = cu_seqlens_k;
    r.context_lens = reinterpret_cast<int32_t *>(ws + w.lens);
    r.table_rows = reinterpret_cast<int32_t *>(ws + w.rows);
    r.num_seqs = num_seqs;
    r.total_q = total_q;
    r.total_k = total_k;
    r.max_seqlen_q = max_seqlen_q;
    r.max_seqlen_k = max_seqlen_k;
    r.max_blocks = max_blocks_per_seq;
    r.block_size = block_size;
    cudaError_t e = pkv::launch_q4_prefill_rows(r, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "prefill_q4 rows launch");
    pkv::Q4DecodeArgs d = {};
    d.cache = g.cache;
    d.q = q;
    d.block_tables = block_tables;
    d.context_lens = r.context_lens;
    d.table_rows = r.table_rows;
    d.out = out;
    d.lse = lse;
    d.ws_o = reinterpret_cast<float *>(ws + w.o);
    d.ws_ml = reinterpret_cast<float *>(ws + w.ml);
    d.max_blocks = max_blocks_per_seq;
    d.max_context_len = max_seqlen_k;
    d.num_seqs = total_q;
    d.num_q_heads = num_q_heads;
    d.window = sliding_window;
    d.plan = decode_plan(total_q, num_kv_heads, window_keys(max_seqlen_k, sliding_window), sms).plan;
    d.scale_log2 = scale * pkv::kLog2e;
    e = pkv::launch_q4_decode(d, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "prefill_q4 rows launch");
    return PKV_OK;
  }
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
  return pkv::prefill_bounded(q, g.ws_k, g.ws_v, cu_seqlens_q, cu_seqlens_k, g.ws_tables, w.max_blocks, num_seqs, total_q,
                              max_seqlen_q, max_seqlen_k, num_q_heads, num_kv_heads, head_dim, pkv::kQ4PrefillBlock,
                              w.num_blocks, scale, sliding_window, out, lse, max_blocks_per_seq * block_size, total_k,
                              stream);
}

}  // extern "C"
