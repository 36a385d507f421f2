// Accumulated attention weights: after a decode call has left its logits
// z[s, h, p] (base 2, scaled) and lse[s, h] (natural log),
//   key_scores[s, p] += sum_h 2^(z[s, h, p] - lse[s, h] log2 e)
// for every key p that sequence s attended to; a logit of -inf has weight 0, also
// where the whole row is such (lse -inf). The sum runs over the heads in
// order, so the result does not depend on the launch shape.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace pkv {

constexpr int kScoreThreads = 256;  // one position each
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

// Chunk `chunk` of `chunks` of sequence s's positions, kScoreThreads at a time;
// lse holds the sequence's [H_q] values.
__device__ __forceinline__ void add_key_scores(const KeyScoresParams &p, int s, int chunk, int chunks, const float *lse) {
  const int ctx = p.context_lens[s];
  if (ctx <= 0 || ctx > p.max_context_len || ctx > p.ctx_cap) return;
  const int first = p.window > 0 && ctx > p.window ? ctx - p.window : 0;
  for (int64_t pos = static_cast<int64_t>(chunk) * kScoreThreads + threadIdx.x; pos < ctx;
       pos += static_cast<int64_t>(chunks) * kScoreThreads) {
    if (pos < first) continue;
    const float *z = p.logits + static_cast<int64_t>(s) * p.num_q_heads * p.logits_ld + pos;
    float w = 0.f;
#pragma unroll 8
    for (int h = 0; h < p.num_q_heads; ++h) {
      const float x = z[h * p.logits_ld];
      w += x == -INFINITY ? 0.f : fast_exp2(fmaf(-kScoreLog2e, lse[h], x));
    }
    p.key_scores[s * p.score_stride + pos] += w;
  }
}

// Body of the per-file kernels; grid (position chunks, sequences).
__device__ __forceinline__ void key_scores_body(const KeyScoresParams &p) {
  add_key_scores(p, blockIdx.y, blockIdx.x, gridDim.x, p.lse + static_cast<int64_t>(blockIdx.y) * p.num_q_heads);
}

// Position chunks of a launch for these sizes.
inline unsigned key_scores_grid_x(int32_t max_context_len) {
  const int64_t n = (static_cast<int64_t>(max_context_len) + kScoreThreads - 1) / kScoreThreads;
  return static_cast<unsigned>(n < 4096 ? n : 4096);
}

}  // namespace pkv
