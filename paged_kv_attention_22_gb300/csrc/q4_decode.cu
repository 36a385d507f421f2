// Paged decode attention over a cache held in 4 bits, one query token per
// sequence.
//
// The keys of a (sequence, KV head) are cut into splits, one CTA each; the
// CTA's warps take the split's steps of 32 keys (two units of 16) in turn. A
// unit's codes are 1 KiB of K and 1 KiB of V, contiguous in the cache, and its
// parameters 64 to 256 bytes of each. Every warp streams its steps through a
// ring of its own with cp.async, so no warp waits for another before the end of
// the split.
//
// The products run on mma.sync m16n8k16 in bf16 with fp32 accumulators. A bf16
// of the cache's definition is what the codes are widened to, so the logits
// have exact products, as with a bf16 cache. With (g, t) = (lane / 4, lane % 4):
//   S^T = K Q^T      A = a unit's 16 keys, B = up to 8 query heads. A lane holds
//                    32 dims of two keys, 16 bytes of codes each.
//   O^T += V^T P^T   A = 16 dims a tile, eight tiles, B = P^T: S^T's accumulator
//                    fragment packed to bf16 and transposed in place (one
//                    movmatrix for 8 keys). A lane holds dims 16 g .. 16 g + 15
//                    of four keys, 8 bytes of codes each.
// Row r (and r + 8) of S^T is key 4 (r & 1) + (r >> 1) (and + 8): lane t then
// needs V rows t, 4 + t, 8 + t and 12 + t, so that four lanes of one load read
// neighbouring rows (free of bank conflicts with the row swizzle below).
//
// P is rounded to bf16 and the output divided by the sum of the rounded
// probabilities, the weights that the products used; the lse comes from the
// fp32 sum.
//
// Widening the codes is what the kernel spends its issue slots on: three
// instructions for two values, 400 of the some 600 that a step takes.
#include "internal.h"
#include "key_scores.cuh"
#include "q4.cuh"

namespace pkv {

static __device__ uint32_t g_q4_decode_errors;

namespace {

constexpr int kD = kQ4D;
constexpr int kUnit = 16;                    // keys a unit
constexpr int kStep = 2 * kUnit;             // keys a step
constexpr int kStages = 2;                   // steps in a warp's ring
constexpr int kMaxG = 8;                     // query heads a KV head (columns of a P^T tile)
constexpr int kUnitCodes = kUnit * kQ4RowBytes;  // 1 KiB of K or V codes
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kFloor = -1.7e38f;           // below every logit; differences stay finite
constexpr float kLazyMax = 8.0f;             // log2 units the running max may lag

struct Q4DecodeParams {
  const __nv_bfloat16 *q;
  const uint8_t *k_codes, *v_codes, *k_params, *v_params;
  const int32_t *block_tables, *context_lens;
  __nv_bfloat16 *out;
  float *lse;
  float *ws_o;     // [S, H_kv, n_splits, G, 128] partial outputs
  float4 *ws_ml;   // [S, H_kv, n_splits, G] (max, sum, sum of the rounded)
  float *logits;   // [S, H_q, logits_ld] or null
  int64_t logits_ld;
  FastDiv block;
  int32_t max_blocks, max_context_len, num_q_heads, num_kv_heads, num_blocks;
  int32_t gqa, window, n_splits, split_keys;
  float scale_log2;  // > 0: the sign of the scale is in q_signs, which flips q's
  uint32_t q_signs;
};

template <int NG, int kWarps>  // parameter groups a row: 4, 2 or 1; warps a CTA: 4, 8 or 16
struct Q4DecodeSmem {
  static constexpr int kParamBytes = kUnit * NG * 4;
  static constexpr int kUnitBytes = 2 * kUnitCodes + 2 * kParamBytes;  // K, V codes, K, V parameters
  static constexpr int kStageBytes = 2 * kUnitBytes;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kMergeBytes = kWarps * kMaxG * (kD + 4) * 4;  // O and (m, l, r) of each warp
  static constexpr int kTotal = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src) {
  if constexpr (N == 16)
    cp_async16(dst, src);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// d += a b, bf16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held by the warp, row g in the
// lanes 4 g .. 4 g + 3, two columns each.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The keys a sequence attends to: [first, ctx); its units start at the 16-key
// boundary at or before first. ctx <= 0 marks an invalid length.
struct KeyRange {
  int ctx, first, unit0;
};
__device__ __forceinline__ KeyRange key_range(const Q4DecodeParams &p, int s) {
  KeyRange r;
  r.ctx = p.context_lens[s];
  if (r.ctx > p.max_context_len || r.ctx > static_cast<int64_t>(p.max_blocks) * p.block.d) r.ctx = 0;
  r.first = p.window > 0 && r.ctx > p.window ? r.ctx - p.window : 0;
  r.unit0 = r.first / kUnit * kUnit;
  return r;
}

template <int NG, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 16 / kWarps) q4_decode_kernel(const Q4DecodeParams p) {
  using L = Q4DecodeSmem<NG, kWarps>;
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, head = blockIdx.y, s = blockIdx.z;
  const int G = p.gqa;
  const KeyRange range = key_range(p, s);
  if (range.ctx <= 0) {
    if (split == 0 && head == 0 && threadIdx.x == 0) atomicOr(&g_q4_decode_errors, kErrContext);
    return;
  }
  const int64_t key_begin64 = range.unit0 + static_cast<int64_t>(split) * p.split_keys;
  if (key_begin64 >= range.ctx) return;  // a split past this sequence's end
  const int key_begin = static_cast<int>(key_begin64);
  const int key_end = min(range.ctx - key_begin, p.split_keys) + key_begin;
  const int n_units = (key_end - key_begin + kUnit - 1) / kUnit;
  const int n_steps = (n_units + 1) / 2;
  const int n_mine = n_steps > warp ? (n_steps - warp + kWarps - 1) / kWarps : 0;

  // the query heads as B fragments: k-step 2w (2w + 1) pairs dims i and i + 4,
  // i = 0, 1 (2, 3), of the lane's w-th code word
  uint32_t qb[8][2];
  {
    const int64_t row = static_cast<int64_t>(s) * p.num_q_heads + head * G + g;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.q + row * kD + 32 * t);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint4 x = g < G ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
      x.x ^= p.q_signs;
      x.y ^= p.q_signs;
      x.z ^= p.q_signs;
      x.w ^= p.q_signs;
      qb[2 * w][0] = q4_low_halves(x.x, x.z);
      qb[2 * w][1] = q4_high_halves(x.x, x.z);
      qb[2 * w + 1][0] = q4_low_halves(x.y, x.w);
      qb[2 * w + 1][1] = q4_high_halves(x.y, x.w);
    }
  }

  // rows / 16 of this warp's unit i (two units a step) in the codes array, or
  // kNoUnit past the split's end and for an invalid table entry; a lane holds one
  // unit of a batch of 32
  constexpr uint32_t kNoUnit = 0xffffffffu;
  const int32_t *table = p.block_tables + static_cast<int64_t>(s) * p.max_blocks;
  auto unit_row = [&](int i) -> uint32_t {
    const int u = (warp + kWarps * (i >> 1)) * 2 + (i & 1);  // the split's unit
    if (u >= n_units) return kNoUnit;
    const int key = key_begin + u * kUnit;
    const uint32_t j = fast_quotient(key, p.block);
    const int blk = table[j];
    if (blk < 0 || blk >= p.num_blocks) {
      atomicOr(&g_q4_decode_errors, kErrBlock);
      return kNoUnit;
    }
    return static_cast<uint32_t>(
        ((static_cast<int64_t>(blk) * p.num_kv_heads + head) * p.block.d + (key - j * p.block.d)) / kUnit);
  };
  uint32_t batch = unit_row(lane), next_batch = n_mine > 16 ? unit_row(32 + lane) : kNoUnit;
  // one bit a unit that is there, of the batch being consumed and of the next
  uint32_t there = __ballot_sync(0xffffffffu, batch != kNoUnit);
  uint32_t there_next = __ballot_sync(0xffffffffu, next_batch != kNoUnit);

  const int kperm = 4 * (g & 1) + (g >> 1);  // key of row g
  const uint32_t ring = smem_u32(smem) + warp * kStages * L::kStageBytes;
  const uint8_t *ring_ptr = smem + warp * kStages * L::kStageBytes;
  // what this lane copies of a unit. K: the 16 bytes that it will read; V: rows
  // in order, chunk c of row r at c ^ 2 ((r >> 1) & 1); the parameter rows: lanes
  // 0..15 K's, 16..31 V's
  const uint8_t *k_src = p.k_codes + kperm * kQ4RowBytes + t * 16;
  const uint8_t *v_src = p.v_codes + lane * 16;
  const uint8_t *p_src = (lane < 16 ? p.k_params : p.v_params) + (lane & 15) * (4 * NG);
  const uint32_t v_dst = kUnitCodes + (lane >> 2) * kQ4RowBytes + ((lane & 3) ^ (((lane >> 3) & 1) << 1)) * 16;
  auto issue = [&](int i) {  // step i
    if (i < n_mine) {
      if (i > 0 && (i & 15) == 0) {
        batch = next_batch;
        next_batch = i + 16 < n_mine ? unit_row(2 * i + 32 + lane) : kNoUnit;
      }
      uint32_t st = ring + (i % kStages) * L::kStageBytes;
#pragma unroll
      for (int u = 0; u < 2; ++u, st += L::kUnitBytes) {
        const uint32_t row16 = __shfl_sync(0xffffffffu, batch, (2 * i + u) & 31);
        if (row16 == kNoUnit) continue;
        const uint8_t *k = k_src + static_cast<int64_t>(row16) * kUnitCodes;
        const uint8_t *v = v_src + static_cast<int64_t>(row16) * kUnitCodes;
        cp_async16(st + lane * 16, k);
        cp_async16(st + 512 + lane * 16, k + 512);
        cp_async16(st + v_dst, v);
        cp_async16(st + v_dst + 512, v + 512);
        cp_async_small<4 * NG>(st + 2 * kUnitCodes + lane * (4 * NG),
                               p_src + static_cast<int64_t>(row16) * L::kParamBytes);
      }
    }
    cp_async_commit();
  };

  float acc[8][4];  // O^T: dims 16 g + 2 m (and + 1), heads 2 t and 2 t + 1
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
  // of heads 2 t and 2 t + 1; lsum is over this lane's keys, rsum (a product's
  // fragment, its rows all alike) over the warp's. The maximum starts at a finite
  // floor, so that masked logits (-inf) have probability 0 even before the first
  // real one.
  float mx[2] = {kFloor, kFloor}, lsum[2] = {0.f, 0.f}, rsum[4] = {0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int i = 0; i < kStages; ++i) issue(i);

#pragma unroll 1
  for (int it = 0; it < n_mine; ++it) {
    cp_async_wait<kStages - 1>();
    __syncwarp();  // every lane's copies of this step have landed
    if (it > 0 && (it & 15) == 0) {
      there = there_next;
      there_next = __ballot_sync(0xffffffffu, next_batch != kNoUnit);
    }
    const uint8_t *st = ring_ptr + (it % kStages) * L::kStageBytes;
    const int key0 = key_begin + (warp + kWarps * it) * kStep;

    // ---- S^T = K Q^T
    float z[2][4];  // unscaled; keys kperm, 8 + kperm of each unit, heads 2 t, 2 t + 1: [u][2 * key + head]
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t *su = st + u * L::kUnitBytes;
      const uint32_t *kp = reinterpret_cast<const uint32_t *>(su + 2 * kUnitCodes) + kperm * NG + t * NG / 4;
      uint32_t words[2][4], s2[2], b2[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 kw = *reinterpret_cast<const uint4 *>(su + 512 * j + lane * 16);
        words[j][0] = kw.x;
        words[j][1] = kw.y;
        words[j][2] = kw.z;
        words[j][3] = kw.w;
        const uint32_t pw = kp[8 * j * NG];
        s2[j] = q4_dup_scale(pw);
        b2[j] = q4_dup_offset(pw);
      }
      float sc[2][4] = {};  // two chains of products
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t x[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          q4_pairs(words[j][w], x[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[j][i] = fma_bf16x2(x[j][i], s2[j], b2[j]);
        }
        mma_16816(sc[0], x[0][0], x[1][0], x[0][1], x[1][1], qb[2 * w][0], qb[2 * w][1]);
        mma_16816(sc[1], x[0][2], x[1][2], x[0][3], x[1][3], qb[2 * w + 1][0], qb[2 * w + 1][1]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) z[u][i] = sc[0][i] + sc[1][i];
    }

    // ---- masks, softmax
    uint32_t pv[2][4];  // V parameters of this lane's V rows
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pv[u][i] = reinterpret_cast<const uint32_t *>(st + u * L::kUnitBytes + 2 * kUnitCodes +
                                                      L::kParamBytes)[(4 * i + t) * NG + g * NG / 8];
    const uint32_t units = (there >> (2 * it & 31)) & 3u;
    if (p.logits != nullptr && 2 * t < G) {  // rows hold whole units: masked keys are written too
      float *dst = p.logits + (static_cast<int64_t>(s) * p.num_q_heads + head * G + 2 * t) * p.logits_ld + key0 + kperm;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!((units >> u) & 1u)) continue;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (2 * t + c >= G) continue;
          dst[c * p.logits_ld + u * kUnit] = z[u][c] * p.scale_log2;
          dst[c * p.logits_ld + u * kUnit + 8] = z[u][2 + c] * p.scale_log2;
        }
      }
    }
    if (key0 < range.first || key0 + kStep > key_end || units != 3u) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int lo = range.first - (key0 + u * kUnit);
        const int hi = ((units >> u) & 1u) ? key_end - (key0 + u * kUnit) : 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (8 * j + kperm < lo || 8 * j + kperm >= hi) z[u][2 * j] = z[u][2 * j + 1] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // the row reads as zeros, whatever its slot holds
          if (4 * i + t < lo || 4 * i + t >= hi) pv[u][i] = 0u;
      }
    }
    const float zm0 = fmaxf(fmax3(z[0][0], z[0][2], z[1][0]), z[1][2]) * p.scale_log2;
    const float zm1 = fmaxf(fmax3(z[0][1], z[0][3], z[1][1]), z[1][3]) * p.scale_log2;
    if (__any_sync(0xffffffffu, zm0 > mx[0] + kLazyMax || zm1 > mx[1] + kLazyMax)) {  // always on a first step
      float m_new[2] = {fmaxf(zm0, mx[0]), fmaxf(zm1, mx[1])}, alpha[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) m_new[c] = fmaxf(m_new[c], __shfl_xor_sync(0xffffffffu, m_new[c], off));
        alpha[c] = fast_exp2(mx[c] - m_new[c]);
        mx[c] = m_new[c];
        lsum[c] *= alpha[c];
      }
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] *= alpha[i & 1];
#pragma unroll
      for (int i = 0; i < 4; ++i) rsum[i] *= alpha[i & 1];
    }
    uint32_t pb[2][2];  // P^T fragments of each unit
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pr[i] = fast_exp2(fmaf(z[u][i], p.scale_log2, -mx[i & 1]));
        lsum[i & 1] += pr[i];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) pb[u][j] = transpose_8x8(pack_bf16x2(pr[2 * j], pr[2 * j + 1]));
      // the sums of the rounded probabilities are one more product, with ones
      constexpr uint32_t kOnes = 0x3F803F80u;
      mma_16816(rsum, kOnes, kOnes, kOnes, kOnes, pb[u][0], pb[u][1]);
    }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t sa = q4_low_halves(pv[u][0], pv[u][1]), ba = q4_high_halves(pv[u][0], pv[u][1]);
      const uint32_t sb = q4_low_halves(pv[u][2], pv[u][3]), bb = q4_high_halves(pv[u][2], pv[u][3]);
      uint2 vw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + t;
        vw[i] = *reinterpret_cast<const uint2 *>(st + u * L::kUnitBytes + kUnitCodes + row * kQ4RowBytes +
                                                 (((g >> 1) ^ (((row >> 1) & 1) << 1)) * 16) + (g & 1) * 8);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // dims 16 g + 4 j .. + 3
        const uint32_t w0 = (j & 2) ? vw[0].y : vw[0].x, w1 = (j & 2) ? vw[1].y : vw[1].x;
        const uint32_t w2 = (j & 2) ? vw[2].y : vw[2].x, w3 = (j & 2) ? vw[3].y : vw[3].x;
        uint32_t xa[4], xb[4];
        q4_pairs((j & 1) ? q4_high_halves(w0, w1) : q4_low_halves(w0, w1), xa);
        q4_pairs((j & 1) ? q4_high_halves(w2, w3) : q4_low_halves(w2, w3), xb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xa[i] = fma_bf16x2(xa[i], sa, ba);
          xb[i] = fma_bf16x2(xb[i], sb, bb);
        }
        mma_16816(acc[2 * j], xa[0], xa[1], xb[0], xb[1], pb[u][0], pb[u][1]);
        mma_16816(acc[2 * j + 1], xa[2], xa[3], xb[2], xb[3], pb[u][0], pb[u][1]);
      }
    }
    __syncwarp();  // every lane has read the stage: it may be filled again
    issue(it + kStages);
  }

  // ---- join the warps
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) lsum[c] += __shfl_xor_sync(0xffffffffu, lsum[c], off);
  cp_async_wait<0>();
  __syncthreads();  // no warp still reads or fills its ring
  float *so = reinterpret_cast<float *>(smem);                       // [warp][G][128]
  float4 *sml = reinterpret_cast<float4 *>(so + kWarps * kMaxG * kD);  // [warp][G]
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (2 * t + c < G)
        *reinterpret_cast<float2 *>(so + (warp * kMaxG + 2 * t + c) * kD + 16 * g + 2 * m) =
            make_float2(acc[m][c], acc[m][2 + c]);
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (g == 0 && 2 * t + c < G) sml[warp * kMaxG + 2 * t + c] = make_float4(mx[c], lsum[c], rsum[c], 0.f);
  __syncthreads();
  const bool whole = range.unit0 + static_cast<int64_t>(p.split_keys) >= range.ctx;
  const int d = threadIdx.x % kD;
  for (int h = threadIdx.x / kD; h < G; h += kWarps * 32 / kD) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w * kMaxG + h].x);
    float o = 0.f, l = 0.f, r = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 ml = sml[w * kMaxG + h];
      const float f = fast_exp2(ml.x - M);
      o = fmaf(so[(w * kMaxG + h) * kD + d], f, o);
      l = fmaf(ml.y, f, l);
      r = fmaf(ml.z, f, r);
    }
    const int64_t row = static_cast<int64_t>(s) * p.num_q_heads + head * G + h;
    if (whole) {
      p.out[row * kD + d] = __float2bfloat16_rn(o / r);
      if (d == 0 && p.lse != nullptr) p.lse[row] = (M + log2f(l)) * kLn2;
    } else {
      const int64_t at = ((static_cast<int64_t>(s) * p.num_kv_heads + head) * p.n_splits + split) * G + h;
      __stcg(p.ws_o + at * kD + d, o);
      if (d == 0) __stcg(p.ws_ml + at, make_float4(M, l, r, 0.f));
    }
  }
}

// Join the splits of the (sequence, query head)s that have more than one: a
// warp each, four dims a lane.
constexpr int kMergeWarps = 4;
constexpr int kMergeBatch = 8;  // splits whose loads are in flight

__global__ void __launch_bounds__(kMergeWarps * 32) q4_merge_kernel(const Q4DecodeParams p, int32_t num_seqs) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(num_seqs) * p.num_q_heads) return;
  const int s = static_cast<int>(row / p.num_q_heads), hq = static_cast<int>(row - static_cast<int64_t>(s) * p.num_q_heads);
  const KeyRange range = key_range(p, s);
  if (range.ctx <= 0) return;
  const int n = (range.ctx - range.unit0 + p.split_keys - 1) / p.split_keys;
  if (n <= 1) return;  // written whole
  const int G = p.gqa, head = hq / G, h = hq % G;
  const int64_t split0 = (static_cast<int64_t>(s) * p.num_kv_heads + head) * p.n_splits * G + h;
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, p.ws_ml[split0 + static_cast<int64_t>(i) * G].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float o[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f, r = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kMergeBatch) {
    float4 ml[kMergeBatch], ov[kMergeBatch];
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      ml[u] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      ov[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + u < n) {
        const int64_t at = split0 + static_cast<int64_t>(i0 + u) * G;
        ml[u] = p.ws_ml[at];
        ov[u] = reinterpret_cast<const float4 *>(p.ws_o + at * kD)[lane];
      }
    }
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const float f = fast_exp2(ml[u].x - M);
      o[0] = fmaf(ov[u].x, f, o[0]);
      o[1] = fmaf(ov[u].y, f, o[1]);
      o[2] = fmaf(ov[u].z, f, o[2]);
      o[3] = fmaf(ov[u].w, f, o[3]);
      l = fmaf(ml[u].y, f, l);
      r = fmaf(ml[u].z, f, r);
    }
  }
  uint2 v;
  v.x = pack_bf16x2(o[0] / r, o[1] / r);
  v.y = pack_bf16x2(o[2] / r, o[3] / r);
  reinterpret_cast<uint2 *>(p.out + row * kD)[lane] = v;
  if (lane == 0 && p.lse != nullptr) p.lse[row] = (M + log2f(l)) * kLn2;
}

__global__ void __launch_bounds__(kScoreThreads) q4_scores_kernel(const KeyScoresParams p) {
  griddep_wait();
  griddep_launch_dependents();
  key_scores_body(p);
}

template <int NG, int kWarps>
cudaError_t launch_splits(const Q4DecodeParams &p, int32_t num_seqs, cudaStream_t stream) {
  constexpr int kSmem = Q4DecodeSmem<NG, kWarps>::kTotal;
  if (kSmem > 48 * 1024) {
    cudaError_t e =
        cudaFuncSetAttribute(q4_decode_kernel<NG, kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(q4_decode_kernel<NG, kWarps>, dim3(p.n_splits, p.num_kv_heads, num_seqs), dim3(kWarps * 32),
                    kSmem, stream, p);
}

template <int NG>
cudaError_t launch_warps(const Q4DecodeParams &p, int32_t warps, int32_t num_seqs, cudaStream_t stream) {
  switch (warps) {
    case 4: return launch_splits<NG, 4>(p, num_seqs, stream);
    case 8: return launch_splits<NG, 8>(p, num_seqs, stream);
    case 16: return launch_splits<NG, 16>(p, num_seqs, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_q4_decode(const Q4DecodeArgs &a, cudaStream_t stream) {
  Q4DecodeParams p;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.k_codes = static_cast<const uint8_t *>(a.cache.k_codes);
  p.v_codes = static_cast<const uint8_t *>(a.cache.v_codes);
  p.k_params = static_cast<const uint8_t *>(a.cache.k_params);
  p.v_params = static_cast<const uint8_t *>(a.cache.v_params);
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.ws_o = a.ws_o;
  p.ws_ml = reinterpret_cast<float4 *>(a.ws_ml);
  p.logits = a.key_scores != nullptr ? a.logits : nullptr;
  p.logits_ld = a.logits_ld;
  p.max_blocks = a.max_blocks;
  p.max_context_len = a.max_context_len;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.cache.num_kv_heads;
  p.block = fast_div(a.cache.block_size);
  p.num_blocks = static_cast<int32_t>(a.cache.num_blocks);
  p.gqa = a.num_q_heads / a.cache.num_kv_heads;
  p.window = a.window;
  p.n_splits = a.plan.n_splits;
  p.split_keys = a.plan.split_keys;
  // a scale of 0 becomes the smallest positive one: its logits stay below 2^-100
  // unless a product passes 2^26, and masked logits stay -inf
  p.scale_log2 = fmaxf(fabsf(a.scale_log2), 0x1p-126f);
  p.q_signs = a.scale_log2 < 0.f ? 0x80008000u : 0u;
  cudaError_t e;
  switch (a.cache.group_size) {
    case 32: e = launch_warps<4>(p, a.plan.warps, a.num_seqs, stream); break;
    case 64: e = launch_warps<2>(p, a.plan.warps, a.num_seqs, stream); break;
    case 128: e = launch_warps<1>(p, a.plan.warps, a.num_seqs, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  if (p.n_splits > 1) {
    const int64_t rows = static_cast<int64_t>(a.num_seqs) * p.num_q_heads;
    e = launch_pdl(q4_merge_kernel, dim3(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps)),
                   dim3(kMergeWarps * 32), 0, stream, p, a.num_seqs);
    if (e != cudaSuccess) return e;
  }
  if (a.key_scores == nullptr) return cudaSuccess;
  KeyScoresParams k;
  k.logits = a.logits;
  k.lse = a.lse;
  k.key_scores = a.key_scores;
  k.context_lens = a.context_lens;
  k.logits_ld = a.logits_ld;
  k.score_stride = a.score_stride;
  k.max_context_len = a.max_context_len;
  k.num_q_heads = a.num_q_heads;
  k.window = a.window;
  k.ctx_cap = static_cast<int64_t>(a.max_blocks) * a.cache.block_size;
  return launch_pdl(q4_scores_kernel, dim3(key_scores_grid_x(a.max_context_len), a.num_seqs),
                    dim3(kScoreThreads), 0, stream, k);
}

cudaError_t q4_decode_error_word(uint32_t **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_q4_decode_errors);
}

}  // namespace pkv
