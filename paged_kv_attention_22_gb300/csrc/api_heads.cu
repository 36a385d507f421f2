// The C entries of the norms and rotation of queries and keys (declared in
// include/pkv.h): the frequencies of a rotation, argument checks and launches.
// Allocates nothing; every call only enqueues work on the caller's stream.
#include <algorithm>
#include <cmath>

#include "pkv.h"
#include "internal.h"

namespace {

using pkv::aligned16;
using pkv::cuda_fail;
using pkv::current_sm_count;

constexpr int32_t kD = 128;
constexpr double kPi = 3.14159265358979323846;

bool rotary_ok(int32_t rotary_dim) { return rotary_dim >= 0 && rotary_dim <= kD && rotary_dim % 8 == 0; }

// A stride in elements: whole 16-byte vectors, and `rows` heads side by side.
bool stride_ok(int64_t stride, int64_t least) {
  return stride % 8 == 0 && stride >= least && stride <= (int64_t{1} << 40);
}

// What both calls check. *nothing: there is nothing to do.
pkv_status check_heads(const pkv::HeadsArgs &a, int32_t head_dim, int32_t kv_rows, bool *nothing) {
  *nothing = false;
  if (a.num_tokens < 0 || a.num_q_heads < 0 || a.num_kv_heads < 0 || !std::isfinite(a.eps) || a.eps < 0.f)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kD) return head_dim <= 0 ? PKV_ERR_INVALID_ARG : PKV_ERR_UNSUPPORTED;
  if (a.rope != nullptr) {
    if (!rotary_ok(a.rope->rotary_dim)) return PKV_ERR_UNSUPPORTED;
    if (!std::isfinite(a.rope->magnitude)) return PKV_ERR_INVALID_ARG;
  }
  if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.q_weight) || !aligned16(a.k_weight) ||
      !aligned16(a.q_out) || !aligned16(a.k_out) || !aligned16(a.v_out))
    return PKV_ERR_INVALID_ARG;
  if (a.num_q_heads > 65535 || a.num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  const int64_t rows = static_cast<int64_t>(a.num_q_heads) + static_cast<int64_t>(kv_rows) * a.num_kv_heads;
  if (rows * a.num_tokens > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (a.num_tokens == 0 || rows == 0) {
    *nothing = true;
    return PKV_OK;
  }
  if (a.num_q_heads > 0 &&
      (a.q == nullptr || a.q_out == nullptr || !stride_ok(a.q_stride, 0) ||
       !stride_ok(a.q_out_stride, a.num_tokens > 1 ? static_cast<int64_t>(a.num_q_heads) * kD : 0)))
    return PKV_ERR_INVALID_ARG;
  if (a.num_kv_heads > 0 && (a.k == nullptr || a.k_out == nullptr || !stride_ok(a.k_stride, 0)))
    return PKV_ERR_INVALID_ARG;
  if (a.rope != nullptr && a.rope->rotary_dim > 0 && a.positions == nullptr) return PKV_ERR_INVALID_ARG;
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_rope_init_frequencies(pkv_rope *rope, int32_t rotary_dim, int32_t interleaved,
                                     const double *frequencies, float magnitude) {
  if (rope == nullptr || !std::isfinite(magnitude) || rotary_dim < 0 || (rotary_dim > 0 && frequencies == nullptr))
    return PKV_ERR_INVALID_ARG;
  if (!rotary_ok(rotary_dim)) return PKV_ERR_UNSUPPORTED;
  pkv_rope r = {};
  r.rotary_dim = rotary_dim;
  r.interleaved = interleaved != 0 ? 1 : 0;
  r.magnitude = magnitude;
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    if (!std::isfinite(frequencies[i])) return PKV_ERR_INVALID_ARG;
    // The fraction of the size is exact; that of a small negative number would be a number
    // near 1, rounded by 2^-54 of a turn. Negated as an integer, modulo 2^64.
    const double turns = std::fabs(frequencies[i]) / (2 * kPi);
    const uint64_t part = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
    r.turns[i] = std::signbit(frequencies[i]) ? 0 - part : part;
  }
  *rope = r;
  return PKV_OK;
}

pkv_status pkv_rope_init(pkv_rope *rope, int32_t rotary_dim, int32_t interleaved, double base, int32_t scaling,
                         double factor, int32_t original_positions, double beta_fast, double beta_slow) {
  if (rope == nullptr || rotary_dim < 0) return PKV_ERR_INVALID_ARG;
  if (!rotary_ok(rotary_dim)) return PKV_ERR_UNSUPPORTED;
  if (!std::isfinite(base) || base <= 1.0 || scaling < PKV_ROPE_PLAIN || scaling > PKV_ROPE_YARN)
    return PKV_ERR_INVALID_ARG;
  if (scaling == PKV_ROPE_PLAIN) factor = 1.0;
  if (!std::isfinite(factor) || factor <= 0.0) return PKV_ERR_INVALID_ARG;
  double low = 0, high = 0, magnitude = 1.0;
  if (scaling == PKV_ROPE_YARN) {
    if (factor < 1.0 || original_positions <= 0 || !std::isfinite(beta_fast) || !(beta_slow > 0.0) ||
        !(beta_fast >= beta_slow))
      return PKV_ERR_INVALID_ARG;
    const auto dim = [&](double beta) {
      return rotary_dim * std::log(original_positions / (beta * 2 * kPi)) / (2 * std::log(base));
    };
    low = std::max(std::floor(dim(beta_fast)), 0.0);
    high = std::min(std::ceil(dim(beta_slow)), static_cast<double>(rotary_dim) - 1);
    magnitude = 0.1 * std::log(factor) + 1.0;
  }
  if (scaling == PKV_ROPE_NTK && rotary_dim > 0) {
    base *= std::pow(factor, static_cast<double>(rotary_dim) / (rotary_dim - 2));
    if (!std::isfinite(base) || base <= 0.0) return PKV_ERR_INVALID_ARG;
  }
  double frequencies[kD / 2];
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == PKV_ROPE_LINEAR) f /= factor;
    if (scaling == PKV_ROPE_YARN) {
      const double ramp = std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
      f = f * (1 - ramp) + f / factor * ramp;
    }
    frequencies[i] = f;
  }
  return pkv_rope_init_frequencies(rope, rotary_dim, interleaved, frequencies, static_cast<float>(magnitude));
}

pkv_status pkv_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *q_weight,
                            const void *k_weight, float eps, const pkv_rope *rope, const int32_t *positions,
                            int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                            void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream) {
  pkv::HeadsArgs a = {};
  a.q = q, a.k = k, a.q_weight = q_weight, a.k_weight = k_weight;
  a.q_out = q_out, a.k_out = k_out;
  a.positions = positions, a.rope = rope;
  a.q_stride = q_stride, a.k_stride = k_stride, a.q_out_stride = q_out_stride, a.k_out_stride = k_out_stride;
  a.num_tokens = num_tokens, a.num_q_heads = num_q_heads, a.num_kv_heads = num_kv_heads;
  a.eps = eps;
  bool nothing;
  pkv_status st = check_heads(a, head_dim, 1, &nothing);
  if (st != PKV_OK || nothing) return st;
  if (num_kv_heads > 0 && !stride_ok(k_out_stride, num_tokens > 1 ? static_cast<int64_t>(num_kv_heads) * kD : 0))
    return PKV_ERR_INVALID_ARG;
  if ((st = current_sm_count(&a.num_sms)) != PKV_OK) return st;
  const cudaError_t e = pkv::launch_heads(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "qk_norm_rope launch");
  return PKV_OK;
}

pkv_status pkv_kv_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                         int64_t v_stride, const void *q_weight, const void *k_weight, float eps,
                         const pkv_rope *rope, const int32_t *positions, const int32_t *slot_mapping,
                         int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                         int32_t block_size, int64_t num_blocks, void *q_out, int64_t q_out_stride, void *k_cache,
                         void *v_cache, void *stream) {
  if (block_size <= 0 || num_blocks <= 0 || num_kv_heads <= 0 || k_cache == nullptr || v_cache == nullptr)
    return PKV_ERR_INVALID_ARG;
  // slots are int32; num_blocks first, so that the product cannot overflow
  if (num_blocks > INT32_MAX || num_blocks * block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  pkv::HeadsArgs a = {};
  a.q = q, a.k = k, a.v = v, a.q_weight = q_weight, a.k_weight = k_weight;
  a.q_out = q_out, a.k_out = k_cache, a.v_out = v_cache;
  a.positions = positions, a.slots = slot_mapping, a.rope = rope;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.q_out_stride = q_out_stride;
  a.num_tokens = num_tokens, a.num_q_heads = num_q_heads, a.num_kv_heads = num_kv_heads;
  a.num_slots = num_blocks * block_size;
  a.eps = eps;
  bool nothing;
  pkv_status st = check_heads(a, head_dim, 2, &nothing);
  if (st != PKV_OK || nothing) return st;
  if (v == nullptr || slot_mapping == nullptr || !stride_ok(v_stride, 0)) return PKV_ERR_INVALID_ARG;
  if ((st = current_sm_count(&a.num_sms)) != PKV_OK) return st;
  const cudaError_t e = pkv::launch_heads(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_append launch");
  return PKV_OK;
}

}  // extern "C"
