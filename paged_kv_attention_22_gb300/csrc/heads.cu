// Queries and keys between a layer's projections and its attention: the norm of
// each head's row and its rotation by the token's position, written back
// (pkv_qk_norm_rope) or, keys and values, into their slots of the paged cache
// (pkv_kv_append).
//
//   y = w x / sqrt(mean(x^2) + eps); pairs (y_a, y_b) of the first R dims rotate by
//   t = position * frequency.
//
// A copy with some arithmetic, bound by HBM bandwidth: every value is read once and
// written once. A warp takes rows of one token, two at a time, 16 lanes a row. Each
// lane holds 8 dims as two runs of 4, chosen so that it has both dims of its four
// pairs: in the half layout (pairs i, i + R / 2) lane l < R / 8 has dims 4 l .. and
// R / 2 + 4 l .., so that neither layout exchanges values between lanes. The cost
// is two 8-byte accesses a row in place of one of 16.
//
// The angle is taken in turns, modulo 1, in 64-bit integers: position times the
// pair's 64-bit fraction of a turn wraps to the fraction of the angle exactly (to
// 2^-64 of a turn a position), where fp32 angles of far positions have no digits
// left, and without the 64-bit floating point that this GPU hardly has. Its top 32
// bits go to sincospi. A lane needs four of them, computed once a token and
// shared by all of its rows; no table of cosines is read, whose rows would also be
// found only after the position has arrived.
#include "internal.h"
#include "ptx.cuh"

namespace pkv {

static __device__ uint32_t g_heads_errors;

namespace {

constexpr int kWarps = 8;
constexpr int kDepth = 4;  // pairs of rows whose loads a warp has in flight

struct HeadsParams {
  const __nv_bfloat16 *q, *k, *v;
  const __nv_bfloat16 *q_weight, *k_weight;
  __nv_bfloat16 *q_out, *k_out, *v_out;  // k_out, v_out: the caches, with slots
  const int32_t *positions, *slots;      // positions: null without a rotation; slots: null for k_out by token
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int64_t num_slots;
  int32_t num_tokens, num_q, num_kv, num_rows;  // heads; num_rows: rows of a token, q then k then v
  int32_t parts, part_rows;                     // warps a token and rows (an even number) of each
  int32_t rotary;
  float eps, magnitude;
  uint64_t turns[64];
};

// Four bf16 values as fp32.
__device__ __forceinline__ void widen(uint2 w, float (&x)[8], int at) {
  x[at] = bf16lo(w.x), x[at + 1] = bf16hi(w.x), x[at + 2] = bf16lo(w.y), x[at + 3] = bf16hi(w.y);
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32) heads_kernel(const __grid_constant__ HeadsParams p) {
  const int lane = threadIdx.x & 31, l = lane & 15;
  const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t token = unit / p.parts;
  const bool turned = 8 * l < p.rotary;  // this lane's dims are rotated
  // the lane's two runs of four dims
  const int run0 = !kInterleaved && turned ? 4 * l : 8 * l;
  const int run1 = !kInterleaved && turned ? p.rotary / 2 + 4 * l : 8 * l + 4;
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  griddep_launch_dependents();
  if (token >= static_cast<uint32_t>(p.num_tokens)) return;
  const int first = (unit - token * p.parts) * p.part_rows;
  const int last = min(first + p.part_rows, p.num_rows);
  int64_t slot = p.slots != nullptr ? p.slots[token] : 0;
  const int32_t position = p.positions != nullptr ? p.positions[token] : 0;

  // a row's source
  auto source = [&](int row) {
    const int kv = row - p.num_q;
    const __nv_bfloat16 *base = p.q + token * p.q_stride + row * 128;
    if (kv >= 0) base = p.k + token * p.k_stride + kv * 128;
    if (kv >= p.num_kv) base = p.v + token * p.v_stride + (kv - p.num_kv) * 128;
    return base;
  };
  uint2 in[kDepth][2];
  auto load = [&](int at) {  // rows at, at + 1 and so on: 2 kDepth of them
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      const int row = at + 2 * i + (lane >> 4);
      if (row < last) {
        const __nv_bfloat16 *src = source(row);
        in[i][0] = __ldcs(reinterpret_cast<const uint2 *>(src + run0));
        in[i][1] = __ldcs(reinterpret_cast<const uint2 *>(src + run1));
      }
    }
  };
  load(first);

  float c[4], s[4];
  uint2 wq[2] = {}, wk[2] = {};
  if (p.q_weight != nullptr) {
    wq[0] = __ldg(reinterpret_cast<const uint2 *>(p.q_weight + run0));
    wq[1] = __ldg(reinterpret_cast<const uint2 *>(p.q_weight + run1));
  }
  if (p.k_weight != nullptr) {
    wk[0] = __ldg(reinterpret_cast<const uint2 *>(p.k_weight + run0));
    wk[1] = __ldg(reinterpret_cast<const uint2 *>(p.k_weight + run1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(position)) * p.turns[(4 * l + i) & 63];
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &s[i], &c[i]);
    s[i] *= p.magnitude;
    c[i] *= p.magnitude;
  }
  if (slot < -1 || slot >= p.num_slots) {
    if (lane == 0 && first == 0) atomicOr(&g_heads_errors, kErrSlot);
    slot = -1;
  }

  for (int at = first; at < last; at += 2 * kDepth) {
    if (at > first) load(at);
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      if (at + 2 * i >= last) break;  // uniform over the warp
      const int row = at + 2 * i + (lane >> 4), kv = row - p.num_q;
      float x[8];
      widen(in[i][0], x, 0);
      widen(in[i][1], x, 4);
      const bool is_q = kv < 0, is_v = kv >= p.num_kv;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if ((is_q ? p.q_weight : p.k_weight) != nullptr && !is_v) {
        const float r = rsqrtf(fmaf(sum, 1.f / 128.f, p.eps));
        float w[8];
        widen(is_q ? wq[0] : wk[0], w, 0);
        widen(is_q ? wq[1] : wk[1], w, 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= r * w[j];
      }
      if (turned && !is_v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float &a = x[kInterleaved ? 2 * j : j], &b = x[kInterleaved ? 2 * j + 1 : j + 4];
          const float turned_a = a * c[j] - b * s[j];
          b = b * c[j] + a * s[j];
          a = turned_a;
        }
      }
      if (row >= last || (!is_q && slot < 0)) continue;
      __nv_bfloat16 *dst = p.q_out + token * p.q_out_stride + row * 128;
      if (!is_q) {
        const int64_t at_row = p.slots != nullptr ? slot * p.num_kv * 128 : token * p.k_out_stride;
        dst = (is_v ? p.v_out + at_row + (kv - p.num_kv) * 128 : p.k_out + at_row + kv * 128);
      }
      *reinterpret_cast<uint2 *>(dst + run0) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
      *reinterpret_cast<uint2 *>(dst + run1) = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
  }
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs &a, cudaStream_t stream) {
  HeadsParams p;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.k = static_cast<const __nv_bfloat16 *>(a.k);
  p.v = static_cast<const __nv_bfloat16 *>(a.v);
  p.q_weight = static_cast<const __nv_bfloat16 *>(a.q_weight);
  p.k_weight = static_cast<const __nv_bfloat16 *>(a.k_weight);
  p.q_out = static_cast<__nv_bfloat16 *>(a.q_out);
  p.k_out = static_cast<__nv_bfloat16 *>(a.k_out);
  p.v_out = static_cast<__nv_bfloat16 *>(a.v_out);
  p.rotary = a.rope != nullptr ? a.rope->rotary_dim : 0;
  p.positions = p.rotary > 0 ? a.positions : nullptr;
  p.slots = a.slots;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_out_stride = a.q_out_stride;
  p.k_out_stride = a.k_out_stride;
  p.num_slots = a.slots != nullptr ? a.num_slots : 1;
  p.num_tokens = a.num_tokens;
  p.num_q = a.num_q_heads;
  p.num_kv = a.num_kv_heads;
  p.num_rows = a.num_q_heads + (a.slots != nullptr ? 2 : 1) * a.num_kv_heads;
  p.eps = a.eps;
  p.magnitude = p.rotary > 0 ? a.rope->magnitude : 1.f;
  for (int i = 0; i < 64; ++i) p.turns[i] = p.rotary > 0 ? a.rope->turns[i] : 0;
  // warps a token: one where there are tokens enough, more for few tokens
  const int64_t want = 16 * static_cast<int64_t>(a.num_sms);
  int32_t parts = 1;
  while (parts * 2 <= (p.num_rows + 1) / 2 && static_cast<int64_t>(a.num_tokens) * parts < want) parts *= 2;
  p.part_rows = ((p.num_rows + parts - 1) / parts + 1) / 2 * 2;
  p.parts = (p.num_rows + p.part_rows - 1) / p.part_rows;
  const int64_t units = static_cast<int64_t>(a.num_tokens) * p.parts;
  const dim3 grid(static_cast<unsigned>((units + kWarps - 1) / kWarps));
  const bool interleaved = p.rotary > 0 && a.rope->interleaved != 0;
  return launch_pdl(interleaved ? heads_kernel<true> : heads_kernel<false>, grid, dim3(kWarps * 32), 0, stream, p);
}

cudaError_t heads_error_word(uint32_t **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_heads_errors);
}

}  // namespace pkv
