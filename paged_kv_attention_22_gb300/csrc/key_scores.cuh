// Accumulated attention weights: after a decode call has left its logits
// z[s, h, p] (base 2, scaled) and lse[s, h] (natural log),
//   key_scores[s, p] += sum_h 2^(z[s, h, p] - lse[s, h] log2 e)
// for every key p that sequence s attended to; a logit of -inf has weight 0, also
// where the whole row is such (lse -inf). The sum runs over the heads in order,
// without atomics: the same call on the same device gives the same bits. Another
// launch shape (other sizes, bounds or SM count) may not: the logits' products and
// the pieces that the lse comes from are then summed in another order.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace pkv {

constexpr int kScoreThreads = 256;
template <int N> struct ScoreVecOf;    // N neighbouring positions a thread
template <> struct ScoreVecOf<2> { using T = float2; };
template <> struct ScoreVecOf<4> { using T = float4; };
constexpr int kMaxScoredHeads = 4096;  // query heads whose lse a scoring CTA holds in shared memory
constexpr float kScoreLog2e = 1.4426950408889634f;

struct KeyScoresParams {
  const float *logits;      // [S, H_q, logits_ld]
  const float *lse;         // [S, H_q]
  float *key_scores;        // [S, score_stride]
  const int32_t *context_lens;
  int64_t logits_ld, score_stride;
  int32_t max_context_len, num_q_heads, window;
  int64_t ctx_cap;          // max_blocks * block_size
};

// Chunk `chunk` of `chunks` of sequence s's positions, kScoreThreads * kVec at a
// time; all threads of the CTA. lse_of() gives the sequence's [H_q] values; it is
// called (by all threads, once) after the first loads, which do not need them.
template <int kVec, typename Lse>
__device__ __forceinline__ void add_key_scores(const KeyScoresParams &p, int s, int chunk, int chunks, Lse &&lse_of) {
  using Vec = typename ScoreVecOf<kVec>::T;
  constexpr int kHeads = 8;  // heads whose logits a thread has in flight
  int ctx = p.context_lens[s];
  if (ctx < 0 || ctx > p.max_context_len || ctx > p.ctx_cap) ctx = 0;
  const int first = p.window > 0 && ctx > p.window ? ctx - p.window : 0;
  // rows of logits are aligned and hold whole units of 16: positions that are not
  // attended to are loaded beside others, but not added
  const float *logits = p.logits + static_cast<int64_t>(s) * p.num_q_heads * p.logits_ld;
  float *scores = p.key_scores + s * p.score_stride;
  Vec z[kHeads];
  float old[kVec];
  auto load = [&](int64_t pos, int h0) {
#pragma unroll
    for (int u = 0; u < kHeads; ++u)
      if (h0 + u < p.num_q_heads) z[u] = *reinterpret_cast<const Vec *>(logits + (h0 + u) * p.logits_ld + pos);
  };
  auto load_first = [&](int64_t pos) {
    load(pos, 0);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (pos + i >= first && pos + i < ctx) old[i] = scores[pos + i];
  };
  int64_t pos = (static_cast<int64_t>(chunk) * kScoreThreads + threadIdx.x) * kVec;
  const int64_t step = static_cast<int64_t>(chunks) * kScoreThreads * kVec;
  while (pos + kVec <= first) pos += step;
  if (pos < ctx) load_first(pos);
  const float *lse = lse_of();
  while (pos < ctx) {
    float w[kVec] = {};
    for (int h0 = 0; h0 < p.num_q_heads; h0 += kHeads) {
      if (h0 > 0) load(pos, h0);
#pragma unroll
      for (int u = 0; u < kHeads; ++u) {
        if (h0 + u >= p.num_q_heads) break;
        const float l = lse[h0 + u];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float x = reinterpret_cast<const float *>(&z[u])[i];
          w[i] += x == -INFINITY ? 0.f : fast_exp2(fmaf(-kScoreLog2e, l, x));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (pos + i >= first && pos + i < ctx) scores[pos + i] = old[i] + w[i];
    pos += step;
    if (pos < ctx) load_first(pos);
  }
}

// Body of the per-file kernels; grid (position chunks, sequences).
template <int kVec>
__device__ __forceinline__ void key_scores_body(const KeyScoresParams &p) {
  add_key_scores<kVec>(p, blockIdx.y, blockIdx.x, gridDim.x,
                 [&] { return p.lse + static_cast<int64_t>(blockIdx.y) * p.num_q_heads; });
}

// Position chunks of a launch for these sizes.
inline unsigned key_scores_grid_x(int32_t max_context_len, int vec) {
  const int64_t n = (static_cast<int64_t>(max_context_len) + kScoreThreads * vec - 1) / (kScoreThreads * vec);
  return static_cast<unsigned>(n < 4096 ? n : 4096);
}

}  // namespace pkv
