// Queries and keys between a layer's projections and its attention: the norm of
// each head's row and its rotation by the token's position, written back
// (pkv_qk_norm_rope) or, keys and values, into their slots of the paged cache
// (pkv_kv_append).
//
//   y = w x / sqrt(mean(x^2) + eps); pairs (y_a, y_b) of the first R dims rotate by
//   t = position * frequency.
//
// A copy with some arithmetic, bound by HBM bandwidth: every value is read once and
// written once. A warp takes groups of four rows of one token's queries, keys or values, 8
// lanes a row. Each lane holds 16 dims as two runs of 8, chosen so that it has both
// dims of its eight pairs: in the half layout (pairs i, i + R / 2) lane l < R / 16 has dims
// 8 l .. and R / 2 + 8 l .., so that neither layout exchanges values between lanes and
// all accesses are of 16 bytes. (Where R is no multiple of 16, runs of 4: accesses of 8 bytes.)
// Rows are copied to shared memory kStages groups ahead, across tokens, each lane its own,
// which keeps enough bytes in flight without registers for them.
//
// The angle is taken in turns, modulo 1, in 64-bit integers: position times the
// pair's 64-bit fraction of a turn wraps to the fraction of the angle without a
// rounding, where fp32 angles of far positions have no digits left, and without the
// 64-bit floating point that this GPU hardly has. Its top 32 bits go to sincospi as fp32,
// 2^-26 of a turn off at most; the fraction itself, from a 64-bit frequency, is off by
// 2^-54 of the frequency a position. A lane computes two of a token's 64 and fetches those of its
// pairs from the others; with the weights they make four factors a pair, the same for all
// of the token's queries (or keys), so that a dim costs two products. No table of cosines is
// read, whose rows would also be found only after the position has arrived.
//
// 32,768 tokens of 16 + 8 heads: 63 us, 6.35 TB/s, 95% of a plain copy's rate; with values,
// norms and into the cache 86 us, 6.25 TB/s. 64 tokens 2.9 us, four 2.6, of which an empty
// kernel takes about 2; 5,001 tokens of 12 rows 10.5 (floor 4.6): two tokens a warp, each some
// 2 us of dependent instructions behind its position. (Weights read again for each token, from
// the L1: 12.0.)
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {

static __device__ uint32_t g_heads_errors;

namespace {

constexpr int kWarps = 4;
// Blocks an SM, which the grid is limited to: 16 warps keep 64 KB of copies in flight. With 20
// and 24 the registers run short: 32,768 tokens into the cache 94 and 104 us where 16 took 89.
constexpr int kBlocks = 4;
constexpr int kRows = 4;    // rows a group
constexpr int kStages = 4;  // groups whose copies a warp has in flight
// How a lane's 16 dims lie in its row: pairs (i, i + R / 2) with R a multiple of 16, with R a
// multiple of 8, and pairs (2 i, 2 i + 1).
enum Layout { kHalf, kHalfNarrow, kInterleaved };

struct HeadsParams {
  const __nv_bfloat16 *q, *k, *v;
  const __nv_bfloat16 *q_weight, *k_weight;
  __nv_bfloat16 *q_out, *k_out, *v_out;  // k_out, v_out: the caches, with slots
  const int32_t *positions, *slots;      // positions: null without a rotation; slots: null for k_out by token
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int64_t num_slots;
  uint32_t num_units;              // tokens, then parts of tokens, taken by the warps in turn
  uint32_t whole;                  // the units that are tokens
  int32_t num_q, num_kv;           // heads
  int32_t k_group, v_group, num_groups;  // the first group of a token's keys, of its values; all
  int32_t parts, part_groups;      // units of each token behind those, groups of each
  int32_t rotary;
  float eps, magnitude;
  alignas(16) uint64_t turns[64];
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool wide) {
  if (wide)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// Two bf16 values as fp32.
__device__ __forceinline__ void widen(uint32_t w, float &a, float &b) { a = bf16lo(w), b = bf16hi(w); }

template <Layout kLayout>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) heads_kernel(const __grid_constant__ HeadsParams p) {
  // [warp][stage][run of 8][lane] x 16 bytes
  __shared__ uint4 staged[kWarps][kStages][2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7, sub = lane >> 3;
  // The lane's dims x[0 .. 15]: in the half layouts pair j is (x[j], x[j + 8]), else
  // (x[2 j], x[2 j + 1]); the first four of them turn if turned0, the others if turned1. run(i):
  // where x[4 i] .. x[4 i + 3] lie; i and i + 1 side by side for even i, but if kHalfNarrow.
  constexpr bool kWide = kLayout != kHalfNarrow;
  const bool turned0 = kLayout == kInterleaved ? 8 * l < p.rotary : 16 * l < p.rotary;
  const bool turned1 = kLayout == kInterleaved ? 64 + 8 * l < p.rotary : 16 * l + 8 < p.rotary;
  auto run = [&](int i) {
    if constexpr (kLayout == kInterleaved) return (i >> 1) * 64 + 8 * l + (i & 1) * 4;
    if constexpr (kLayout == kHalf)
      return turned0 ? (i >> 1) * (p.rotary / 2) + 8 * l + (i & 1) * 4
                     : p.rotary / 2 + (i >> 1) * (64 - p.rotary / 2) + 8 * l + (i & 1) * 4;
    return (i & 1 ? turned1 : turned0) ? (i >> 1) * (p.rotary / 2) + 8 * l + (i & 1) * 4
                                       : 16 * l + (i & 1) * 8 + (i >> 1) * 4;
  };
  const int run0 = run(0), run1 = run(1), run2 = run(2), run3 = run(3);
  // the pair of frequency x[]'s pair j has
  auto frequency = [&](int j) { return kLayout == kInterleaved ? (j >> 2) * 32 + 4 * l + (j & 3) : 8 * l + j; };
  // Read by its address: as an operand from the constant bank the lanes' 32 places would be
  // read one after the other (0.4 us of the 3 us of a small call).
  const uint64_t *turns_at = p.turns;
  asm volatile("" : "+l"(turns_at));
  const ulonglong2 turns = reinterpret_cast<const ulonglong2 *>(turns_at)[lane];
  const uint32_t stride = gridDim.x * kWarps;
  const uint32_t unit0 = blockIdx.x * kWarps + warp;
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  griddep_launch_dependents();
  if (unit0 >= p.num_units) return;

  // A place in the warp's work: a group of a unit, within its section (0, 1, 2: queries, keys,
  // values).
  struct At {
    uint32_t unit, token;
    int group, last;  // of the unit
    int what, end;    // the section, and where it or the unit ends
    int row, rows;    // the lane's row, and the section's
  };
  auto enter_section = [&](At &at) {
    const bool q = at.group < p.k_group, k = !q && at.group < p.v_group;
    at.what = q ? 0 : k ? 1 : 2;
    at.end = min(at.last, q ? p.k_group : k ? p.v_group : p.num_groups);
    at.row = (at.group - (q ? 0 : k ? p.k_group : p.v_group)) * kRows + sub;
    at.rows = q ? p.num_q : p.num_kv;
  };
  auto token_of = [&](uint32_t unit) {
    return unit < p.whole || p.parts == 1 ? unit : p.whole + (unit - p.whole) / p.parts;
  };
  auto enter = [&](At &at, uint32_t unit) {
    at.unit = unit;
    at.token = token_of(unit);
    at.group = unit < p.whole ? 0 : (unit - p.whole - (at.token - p.whole) * p.parts) * p.part_groups;
    at.last = unit < p.whole ? p.num_groups : min(at.group + p.part_groups, p.num_groups);
    enter_section(at);
  };
  At ahead = {};  // of the copies
  const __nv_bfloat16 *src = nullptr;
  auto locate = [&]() {
    src = (ahead.what == 0   ? p.q + ahead.token * p.q_stride
           : ahead.what == 1 ? p.k + ahead.token * p.k_stride
                             : p.v + ahead.token * p.v_stride) +
          ahead.row * 128;
  };
  enter(ahead, unit0);
  locate();
  const uint32_t stages = smem_u32(&staged[warp][0][0][lane]);
  uint32_t stage_ahead = 0;
  auto copy = [&]() {
    if (ahead.unit < p.num_units) {
      if (ahead.row < ahead.rows) {
        const uint32_t dst = stages + stage_ahead;
        copy_async(dst, src + run0, kWide);
        if (!kWide) copy_async(dst + 8, src + run1, false);
        copy_async(dst + 32 * 16, src + run2, kWide);
        if (!kWide) copy_async(dst + 32 * 16 + 8, src + run3, false);
      }
      ahead.row += kRows;
      src += kRows * 128;
      if (++ahead.group == ahead.end) {
        if (ahead.group == ahead.last)
          enter(ahead, ahead.unit + stride);
        else
          enter_section(ahead);
        locate();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    stage_ahead = stage_ahead + 1024 == kStages * 1024 ? 0 : stage_ahead + 1024;
  };

  At at;
  enter(at, unit0);
  int32_t next_slot = p.slots != nullptr ? p.slots[at.token] : 0;
  int32_t next_position = p.positions != nullptr ? p.positions[at.token] : 0;
  uint2 wq[4] = {}, wk[4] = {};  // of the lane's dims
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at_run = i == 0 ? run0 : i == 1 ? run1 : i == 2 ? run2 : run3;
    if (p.q_weight != nullptr) wq[i] = __ldg(reinterpret_cast<const uint2 *>(p.q_weight + at_run));
    if (p.k_weight != nullptr) wk[i] = __ldg(reinterpret_cast<const uint2 *>(p.k_weight + at_run));
  }
#pragma unroll 1
  for (int i = 0; i < kStages; ++i) copy();
  int64_t slot = 0;
  float cos0 = 1.f, cos1 = 1.f, sin0 = 0.f, sin1 = 0.f;  // of pairs 2 lane, 2 lane + 1
  // y_a = aa x_a + ba x_b, y_b = bb x_b + ab x_a, for pair j
  float aa[8], ba[8], ab[8], bb[8];
  bool normed = false;
  uint32_t stage = 0;
  bool new_unit = true, new_section = true;
  __nv_bfloat16 *dst = nullptr;
#pragma unroll 1
  while (at.unit < p.num_units) {
    if (new_unit) {
      slot = next_slot;
      const int32_t position = next_position;
      const uint32_t next = token_of(min(at.unit + stride, p.num_units - 1));
      if (p.slots != nullptr) next_slot = p.slots[next];
      if (p.positions != nullptr) next_position = p.positions[next];
      if (slot < -1 || slot >= p.num_slots) {
        if (lane == 0) atomicOr(&g_heads_errors, kErrSlot);
        slot = -1;
      }
      auto angle = [&](uint64_t fraction, float &c, float &s) {
        const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(position)) * fraction;
        sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &s, &c);
        s *= p.magnitude;
        c *= p.magnitude;
      };
      if (p.rotary > 0) {
        angle(turns.x, cos0, sin0);
        angle(turns.y, cos1, sin1);
      }
    }
    if (new_section) {
      dst = p.q_out + at.token * p.q_out_stride;
      if (at.what > 0)
        dst = (at.what == 1 ? p.k_out : p.v_out) + (p.slots != nullptr ? slot * p.num_kv * 128 : at.token * p.k_out_stride);
      dst += at.row * 128;
      if (at.what > 0 && slot < 0) at.rows = 0;  // nothing is written
    }
    if (new_section && at.what < 2) {
      normed = (at.what == 0 ? p.q_weight : p.k_weight) != nullptr;
      float w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = 1.f;
      if (normed) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2 u = at.what == 0 ? wq[i] : wk[i];
          widen(u.x, w[4 * i], w[4 * i + 1]);
          widen(u.y, w[4 * i + 2], w[4 * i + 3]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float wa = w[kLayout == kInterleaved ? 2 * j : j], wb = w[kLayout == kInterleaved ? 2 * j + 1 : j + 8];
        const int from = frequency(j) >> 1;
        float c = __shfl_sync(0xffffffffu, j & 1 ? cos1 : cos0, from);
        float s = __shfl_sync(0xffffffffu, j & 1 ? sin1 : sin0, from);
        if (!(j < 4 ? turned0 : turned1)) c = 1.f, s = 0.f;
        aa[j] = wa * c, ba[j] = -wb * s, ab[j] = wa * s, bb[j] = wb * c;
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    uint4 in[2] = {staged[warp][stage][0][lane], staged[warp][stage][1][lane]};
    stage = stage + 1 == kStages ? 0 : stage + 1;
    if (at.what < 2) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        widen(in[i].x, x[8 * i], x[8 * i + 1]);
        widen(in[i].y, x[8 * i + 2], x[8 * i + 3]);
        widen(in[i].z, x[8 * i + 4], x[8 * i + 5]);
        widen(in[i].w, x[8 * i + 6], x[8 * i + 7]);
      }
      if (normed) {
        float sums[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 16; ++j) sums[j & 1] = fmaf(x[j], x[j], sums[j & 1]);
        float sum = sums[0] + sums[1];
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const float r = rsqrtf(fmaf(sum, 1.f / 128.f, p.eps));
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= r;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float &a = x[kLayout == kInterleaved ? 2 * j : j], &b = x[kLayout == kInterleaved ? 2 * j + 1 : j + 8];
        float ya = a * aa[j], yb = b * bb[j];
        if (j < 4 ? turned0 : turned1) {  // else an infinity stays where it is
          ya = fmaf(b, ba[j], ya);
          yb = fmaf(a, ab[j], yb);
        }
        a = ya, b = yb;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        in[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                           pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
    }
    if (at.row < at.rows) {
      if constexpr (kWide) {
        *reinterpret_cast<uint4 *>(dst + run0) = in[0];
        *reinterpret_cast<uint4 *>(dst + run2) = in[1];
      } else {
        *reinterpret_cast<uint2 *>(dst + run0) = make_uint2(in[0].x, in[0].y);
        *reinterpret_cast<uint2 *>(dst + run1) = make_uint2(in[0].z, in[0].w);
        *reinterpret_cast<uint2 *>(dst + run2) = make_uint2(in[1].x, in[1].y);
        *reinterpret_cast<uint2 *>(dst + run3) = make_uint2(in[1].z, in[1].w);
      }
    }
    copy();  // into the stage just read
    dst += kRows * 128;
    at.row += kRows;
    new_section = ++at.group == at.end;
    new_unit = at.group == at.last;
    if (new_unit)
      enter(at, at.unit + stride);
    else if (new_section)
      enter_section(at);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
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
  p.num_q = a.num_q_heads;
  p.num_kv = a.num_kv_heads;
  const int q_groups = (a.num_q_heads + kRows - 1) / kRows, kv_groups = (a.num_kv_heads + kRows - 1) / kRows;
  p.k_group = q_groups;
  p.v_group = q_groups + kv_groups;
  p.num_groups = p.v_group + (a.slots != nullptr ? kv_groups : 0);
  p.eps = a.eps;
  p.magnitude = p.rotary > 0 ? a.rope->magnitude : 1.f;
  for (int i = 0; i < 64; ++i) p.turns[i] = p.rotary > 0 ? a.rope->turns[i] : 0;
  // As many tokens as give every warp the same number are units; each of the tokens behind is
  // split between as many warps as it has groups for and there are (of 5,001 tokens of 12 rows the
  // last 137, between four warps each).
  const int64_t warps = static_cast<int64_t>(kWarps * kBlocks) * a.num_sms;
  p.whole = static_cast<uint32_t>(a.num_tokens / warps * warps);
  const int64_t behind = a.num_tokens - p.whole;
  int32_t parts = 1;
  while (parts < p.num_groups && behind * parts * 2 <= warps) parts *= 2;
  p.part_groups = (p.num_groups + parts - 1) / parts;
  p.parts = (p.num_groups + p.part_groups - 1) / p.part_groups;
  p.num_units = static_cast<uint32_t>(p.whole + behind * p.parts);
  const int64_t blocks = std::min<int64_t>((static_cast<int64_t>(p.num_units) + kWarps - 1) / kWarps,
                                           kBlocks * static_cast<int64_t>(a.num_sms));
  const auto kernel = p.rotary > 0 && a.rope->interleaved != 0 ? heads_kernel<kInterleaved>
                      : p.rotary % 16 == 0                     ? heads_kernel<kHalf>
                                                               : heads_kernel<kHalfNarrow>;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0, stream, p);
}

cudaError_t heads_error_word(uint32_t **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_heads_errors);
}

}  // namespace pkv
