// Paged decode attention over a cache held in 4 bits, one query token per
// sequence.
//
// The work is (sequence, KV head) pairs of steps of 32 keys (two units of 16). A
// unit's codes are 1 KiB of K and 1 KiB of V, contiguous in the cache, and its
// parameters 64 to 256 bytes of each. Every warp streams its steps through a ring
// of its own with cp.async, so no warp waits for another within its work. Two
// ways of sharing the steps out (decode_plan in api_q4.cu chooses):
//   pairs    one CTA of 4, 8 or 16 warps a pair, which take its steps in turn
//            and join through shared memory. One kernel: the way for many pairs.
//   ranges   16 warps an SM; the steps of all pairs, listed in order, are cut into
//            equal ranges, one a warp, whatever the lengths. A pair cut between
//            warps leaves one partial result each in the workspace (a warp's
//            first piece in slot 2w, its last in slot 2w + 1), joined by a
//            second kernel: the way for few or unequal pairs. (Splits of fixed
//            length in CTAs of their own took 68 us where ranges take 65.7;
//            joined in clusters through distributed shared memory, 73.)
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
// What bounds it: widening the codes, a shift, a logic operation and a packed fma
// for two values, some 420 of the 680 instructions of a step. Shifts and logic
// share one half-rate pipe and packed fmas have another. 16 sequences of 16,384
// keys, 8 KV heads, 2 query heads each: 65.7 us, 336 MB at 5.1 TB/s; issue slots
// 62 % used, the shift and logic pipe 57 %. (Without the widening the same loop
// streams at 6.3 TB/s; a step of 16 keys, or 20 or 24 warps an SM with fewer
// registers, took 71 to 78 us.) 64 sequences of 640 keys: 15.4 us.
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
constexpr int kQueryBytes = 32 * 64;         // a warp's query fragments
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kFloor = -1.7e38f;           // below every logit; differences stay finite
constexpr float kLazyMax = 8.0f;             // log2 units the running max may lag

struct Q4DecodeParams {
  const __nv_bfloat16 *q;
  const uint8_t *k_codes, *v_codes, *k_params, *v_params;
  const int32_t *block_tables, *context_lens;
  const int32_t *table_rows;  // row of block_tables of each sequence, or null: its own index
  __nv_bfloat16 *out;
  float *lse;
  float *ws_o;     // ranges: [2 warps, G, 128] partial outputs
  float4 *ws_ml;   // ranges: [2 warps, G] (max, sum, sum of the rounded)
  float *logits;   // [S, H_q, logits_ld] or null
  int64_t logits_ld;
  FastDiv block;
  int32_t max_blocks, max_context_len, num_q_heads, num_kv_heads, num_blocks;
  int32_t num_seqs, gqa, window;
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
// boundary at or before first. ctx == 0 marks an invalid length.
struct KeyRange {
  int ctx, first, unit0;
};
__device__ __forceinline__ KeyRange key_range(const Q4DecodeParams &p, int ctx) {
  KeyRange r;
  r.ctx = ctx;
  if (ctx <= 0 || ctx > p.max_context_len || ctx > static_cast<int64_t>(p.max_blocks) * p.block.d) r.ctx = 0;
  r.first = p.window > 0 && r.ctx > p.window ? r.ctx - p.window : 0;
  r.unit0 = r.first / kUnit * kUnit;
  return r;
}
__device__ __forceinline__ const int32_t *table_of(const Q4DecodeParams &p, int s) {
  return p.block_tables + static_cast<int64_t>(p.table_rows != nullptr ? p.table_rows[s] : s) * p.max_blocks;
}
__device__ __forceinline__ int steps_of(const KeyRange &r) { return (r.ctx - r.unit0 + kStep - 1) / kStep; }

// ---- ranges: the list of steps, in (sequence, KV head, step) order

// prefix[s] = steps of one head of the sequences before s, for all s <= num_seqs,
// and the lengths (0: invalid); one warp.
__device__ __forceinline__ void build_prefix(const Q4DecodeParams &p, int64_t *prefix, int *ctx_of, bool raise,
                                             int lane) {
  constexpr int kLoads = 8;  // lengths a lane has in flight
  int64_t carry = 0;
  for (int base = 0; base < p.num_seqs; base += 32 * kLoads) {
    int len[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int s = base + 32 * u + lane;
      len[u] = s < p.num_seqs ? p.context_lens[s] : 0;
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int s = base + 32 * u + lane;
      if (base + 32 * u >= p.num_seqs) break;
      int64_t n = 0;
      if (s < p.num_seqs) {
        const KeyRange r = key_range(p, len[u]);
        if (r.ctx == 0 && raise && p.table_rows == nullptr) atomicOr(&g_q4_decode_errors, kErrContext);
        n = r.ctx > 0 ? steps_of(r) : 0;
        if (ctx_of != nullptr) ctx_of[s] = r.ctx;
      }
      int64_t incl = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      if (s < p.num_seqs) prefix[s] = carry + incl - n;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (lane == 0) prefix[p.num_seqs] = carry;
}

struct Step {
  int s, head, k;
};
// Step u of the list (u below its length).
__device__ __forceinline__ Step locate(const int64_t *prefix, int num_seqs, int heads, int64_t u) {
  int lo = 0, hi = num_seqs - 1;  // the last s with heads * prefix[s] <= u: it has steps
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (heads * prefix[mid] <= u) lo = mid; else hi = mid - 1;
  }
  const int64_t n = prefix[lo + 1] - prefix[lo], r = u - heads * prefix[lo];
  const int head = static_cast<int>(r / n);
  return {lo, head, static_cast<int>(r - head * n)};
}
// First step of warp w's range of U steps among W <= U warps, and the warp whose
// range holds step u.
__device__ __forceinline__ int64_t range_start(int64_t w, int64_t W, int64_t U) { return w * U / W; }
__device__ __forceinline__ int64_t owner_of(int64_t u, int64_t W, int64_t U) { return ((u + 1) * W + U - 1) / U - 1; }

template <int NG, int kWarps, bool kRanges>
__global__ void __launch_bounds__(kWarps * 32, 16 / kWarps) q4_decode_kernel(const Q4DecodeParams p) {
  using L = Q4DecodeSmem<NG, kWarps>;
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.gqa;
  // ranges: the list of steps, behind the rings and the warps' queries
  [[maybe_unused]] int64_t *prefix = reinterpret_cast<int64_t *>(smem + L::kTotal + kWarps * kQueryBytes);
  [[maybe_unused]] int *ctx_of = reinterpret_cast<int *>(prefix + p.num_seqs + 1);
  [[maybe_unused]] int64_t first_step = 0;  // this warp's range starts there
  Step cur = {static_cast<int>(blockIdx.y), static_cast<int>(blockIdx.x), 0};
  KeyRange range;
  int n_mine;  // this warp's steps
  [[maybe_unused]] int first_entry = 0;
  if constexpr (kRanges) {
    if (warp == 0) build_prefix(p, prefix, ctx_of, blockIdx.x == 0, lane);
    __syncthreads();
    const int64_t U = p.num_kv_heads * prefix[p.num_seqs];
    const int64_t W = min(static_cast<int64_t>(gridDim.x) * kWarps, U);
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (w >= W) return;
    first_step = range_start(w, W, U);
    n_mine = static_cast<int>(range_start(w + 1, W, U) - first_step);
    cur = locate(prefix, p.num_seqs, p.num_kv_heads, first_step);
    range = key_range(p, ctx_of[cur.s]);
  } else {
    // the table entry of the lane's first unit is loaded beside the length,
    // before the length says whether the unit exists (without a window the first
    // unit is at position 0)
    const uint32_t j = fast_quotient((warp + kWarps * (lane >> 1)) * kStep + (lane & 1) * kUnit, p.block);
    first_entry = table_of(p, cur.s)[min(j, static_cast<uint32_t>(p.max_blocks) - 1)];
    range = key_range(p, p.context_lens[cur.s]);
    if (range.ctx == 0) {
      if (cur.head == 0 && threadIdx.x == 0 && p.table_rows == nullptr) atomicOr(&g_q4_decode_errors, kErrContext);
      return;
    }
    const int n_steps = steps_of(range);
    n_mine = n_steps > warp ? (n_steps - warp + kWarps - 1) / kWarps : 0;
  }

  // the pair's query heads as B fragments: k-step 2w (2w + 1) pairs dims i and
  // i + 4, i = 0, 1 (2, 3), of the lane's w-th code word. They are kept in shared
  // memory (each lane its own, read back for every unit), not in 16 registers (16 x
  // 16,384 keys 67.8 us in registers, 65.7 so; 300 x 2,048 136.0 and 134.2)
  uint4 *sq = reinterpret_cast<uint4 *>(smem + L::kTotal) + warp * 4 * 32 + lane;
  auto load_q = [&]() {
    const int64_t row = static_cast<int64_t>(cur.s) * p.num_q_heads + cur.head * G + g;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.q + row * kD + 32 * t);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint4 x = g < G ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
      x.x ^= p.q_signs;
      x.y ^= p.q_signs;
      x.z ^= p.q_signs;
      x.w ^= p.q_signs;
      sq[w * 32] = make_uint4(q4_low_halves(x.x, x.z), q4_high_halves(x.x, x.z), q4_low_halves(x.y, x.w),
                              q4_high_halves(x.y, x.w));
    }
  };
  load_q();

  // rows / 16 of this warp's unit i (two units a step) in the codes array, or
  // kNoUnit past the last key and for an invalid table entry; a lane holds one
  // unit of a batch of 32
  constexpr uint32_t kNoUnit = 0xffffffffu;
  auto unit_row = [&](int i, bool loaded = false) -> uint32_t {
    int s, head, key, ctx;
    if constexpr (kRanges) {
      if ((i >> 1) >= n_mine) return kNoUnit;
      const Step at = locate(prefix, p.num_seqs, p.num_kv_heads, first_step + (i >> 1));
      const KeyRange r = key_range(p, ctx_of[at.s]);
      s = at.s, head = at.head, ctx = r.ctx;
      key = r.unit0 + at.k * kStep + (i & 1) * kUnit;
    } else {
      const int64_t k = range.unit0 + static_cast<int64_t>(warp + kWarps * (i >> 1)) * kStep + (i & 1) * kUnit;
      if (k >= range.ctx) return kNoUnit;
      s = cur.s, head = cur.head, ctx = range.ctx;
      key = static_cast<int>(k);
    }
    if (key >= ctx) return kNoUnit;
    const uint32_t j = fast_quotient(key, p.block);
    const int blk = loaded ? first_entry : table_of(p, s)[j];
    if (blk < 0 || blk >= p.num_blocks) {
      atomicOr(&g_q4_decode_errors, kErrBlock);
      return kNoUnit;
    }
    return static_cast<uint32_t>(
        ((static_cast<int64_t>(blk) * p.num_kv_heads + head) * p.block.d + (key - j * p.block.d)) / kUnit);
  };
  uint32_t batch = unit_row(lane, !kRanges && range.unit0 == 0), next_batch = n_mine > 16 ? unit_row(32 + lane) : kNoUnit;
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
        cp_async<4 * NG>(st + 2 * kUnitCodes + lane * (4 * NG),
                         p_src + static_cast<int64_t>(row16) * L::kParamBytes);
      }
    }
    cp_async_commit();
  };

  float acc[8][4];  // O^T: dims 16 g + 2 m (and + 1), heads 2 t and 2 t + 1
  // of heads 2 t and 2 t + 1; lsum is over this lane's keys, rsum (a product's
  // fragment, its rows all alike) over the warp's. The maximum starts at a finite
  // floor, so that masked logits (-inf) have probability 0 even before the first
  // real one.
  float mx[2], lsum[2], rsum[4];
  auto reset = [&]() {
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
    mx[0] = mx[1] = kFloor;
    lsum[0] = lsum[1] = 0.f;
    rsum[0] = rsum[1] = rsum[2] = rsum[3] = 0.f;
  };
  reset();
  // lsum over the warp's keys
  auto join_lanes = [&]() {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) lsum[c] += __shfl_xor_sync(0xffffffffu, lsum[c], off);
  };
  int key0 = range.unit0 + (kRanges ? cur.k : warp) * kStep;  // first key of the step
  // ranges: whether the pair's first step is this warp's, and its slot
  [[maybe_unused]] bool opened = cur.k == 0;
  [[maybe_unused]] int64_t slot = 2 * (static_cast<int64_t>(blockIdx.x) * kWarps + warp);

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
      // chains of products: one for pairs (64 x 640 keys 15.4 us, 15.6 with two), two
      // for ranges (16 x 16,384 keys 65.5 us, 66.8 with one)
      constexpr int kChains = kRanges ? 2 : 1;
      float sc[kChains][4] = {};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t x[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          q4_pairs(words[j][w], x[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[j][i] = fma_bf16x2(x[j][i], s2[j], b2[j]);
        }
        const uint4 y = sq[w * 32];
        mma_16816(sc[0], x[0][0], x[1][0], x[0][1], x[1][1], y.x, y.y);
        mma_16816(sc[kChains - 1], x[0][2], x[1][2], x[0][3], x[1][3], y.z, y.w);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) z[u][i] = kChains == 2 ? sc[0][i] + sc[kChains - 1][i] : sc[0][i];
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
      float *dst = p.logits + (static_cast<int64_t>(cur.s) * p.num_q_heads + cur.head * G + 2 * t) * p.logits_ld + key0 + kperm;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (key0 + u * kUnit >= range.ctx) continue;
        const bool is = (units >> u) & 1u;  // no such block: left out
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (2 * t + c >= G) continue;
          dst[c * p.logits_ld + u * kUnit] = is ? z[u][c] * p.scale_log2 : -INFINITY;
          dst[c * p.logits_ld + u * kUnit + 8] = is ? z[u][2 + c] * p.scale_log2 : -INFINITY;
        }
      }
    }
    if (key0 < range.first || key0 + kStep > range.ctx || units != 3u) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int lo = range.first - (key0 + u * kUnit);
        const int hi = ((units >> u) & 1u) ? range.ctx - (key0 + u * kUnit) : 0;
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
    if constexpr (!kRanges) {
      key0 += kWarps * kStep;
    } else {
      key0 += kStep;
      const bool closes = key0 >= range.ctx;
      if (closes || it == n_mine - 1) {
        join_lanes();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (2 * t + c >= G) continue;
          if (opened && closes) {  // the whole pair
            const int64_t row = static_cast<int64_t>(cur.s) * p.num_q_heads + cur.head * G + 2 * t + c;
            const float inv = 1.f / rsum[c];
            uint32_t o[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) o[m] = pack_bf16x2(acc[m][c] * inv, acc[m][2 + c] * inv);
            uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * kD + 16 * g);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
            if (g == 0 && p.lse != nullptr) p.lse[row] = (mx[c] + log2f(lsum[c])) * kLn2;
          } else {
            const int64_t at = slot * G + 2 * t + c;
            float4 *dst = reinterpret_cast<float4 *>(p.ws_o + at * kD + 16 * g);
#pragma unroll
            for (int m = 0; m < 8; m += 2)
              __stcg(dst + m / 2, make_float4(acc[m][c], acc[m][2 + c], acc[m + 1][c], acc[m + 1][2 + c]));
            if (g == 0) __stcg(p.ws_ml + at, make_float4(mx[c], lsum[c], rsum[c], 0.f));
          }
        }
        if (it + 1 < n_mine) {  // the next pair, past sequences without steps
          if (++cur.head == p.num_kv_heads) {
            cur.head = 0;
            do ++cur.s;
            while (prefix[cur.s + 1] == prefix[cur.s]);
            range = key_range(p, ctx_of[cur.s]);
          }
          key0 = range.unit0;
          opened = true;
          slot |= 1;
          load_q();
          reset();
        }
      }
    }
  }
  if constexpr (kRanges) {
    cp_async_wait<0>();
    return;
  }

  // ---- pairs: join the warps
  join_lanes();
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
    const int64_t row = static_cast<int64_t>(cur.s) * p.num_q_heads + cur.head * G + h;
    p.out[row * kD + d] = __float2bfloat16_rn(o / r);
    if (d == 0 && p.lse != nullptr) p.lse[row] = (M + log2f(l)) * kLn2;
  }
}

// Ranges: join the pieces of the (sequence, query head)s whose pairs were cut,
// kPerRow warps each (8 for pairs cut into many pieces), four dims a lane.
constexpr int kMergeWarps = 8;
constexpr int kMergeBatch = 8;  // pieces whose loads a warp has in flight
static_assert(kMergeWarps * 32 == kScoreThreads, "a CTA of the merge's launch may be one of the weights'");

// The pieces of a (sequence, query head): the first one's warp, how many, and the
// first one's slot (the others': twice their warp).
struct Pieces {
  int64_t first, n, slot;
};
__device__ __forceinline__ Pieces pieces_of(const Q4DecodeParams &p, const int64_t *prefix, int64_t W, int64_t U, int s,
                                            int head) {
  const int64_t steps = prefix[s + 1] - prefix[s], P0 = p.num_kv_heads * prefix[s] + head * steps;
  if (steps == 0) return {0, 0, 0};
  const int64_t wa = owner_of(P0, W, U);
  return {wa, owner_of(P0 + steps - 1, W, U) - wa + 1, 2 * wa + (range_start(wa, W, U) < P0 ? 1 : 0)};
}

// With accumulated weights the launch's first `score_ctas` CTAs (chunks of each
// sequence's positions) add them, beside the CTAs that merge: they take the
// lse from the pieces themselves, half a warp a head, and need not wait for the merge.
template <int kPerRow, int kVec>
__global__ void __launch_bounds__(kMergeWarps * 32)
    q4_merge_kernel(const Q4DecodeParams p, int32_t decode_warps, const KeyScoresParams k, int32_t score_ctas,
                    int32_t score_chunks) {
  extern __shared__ int64_t merge_prefix[];  // [S + 1], then the lse of a scoring CTA's sequence [H_q]
  __shared__ float4 s_o[kMergeWarps][32];
  __shared__ float s_ml[kMergeWarps][3];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kPerRow;
  if (warp == 0) build_prefix(p, merge_prefix, nullptr, false, lane);
  __syncthreads();
  const int64_t U = p.num_kv_heads * merge_prefix[p.num_seqs];
  const int64_t W = min(static_cast<int64_t>(decode_warps), U);
  if (static_cast<int>(blockIdx.x) < score_ctas) {
    float *lse = reinterpret_cast<float *>(merge_prefix + p.num_seqs + 1);
    const int s = blockIdx.x / score_chunks, chunk = blockIdx.x - s * score_chunks;
    add_key_scores<kVec>(k, s, chunk, score_chunks, [&]() -> const float * {
      const int half = lane & 15;
      for (int h0 = 2 * warp; h0 < p.num_q_heads; h0 += 2 * kMergeWarps) {
        const int hq = h0 + (lane >> 4);
        const Pieces c = hq < p.num_q_heads ? pieces_of(p, merge_prefix, W, U, s, hq / p.gqa) : Pieces{0, 0, 0};
        float M = kFloor, l = 0.f;
        for (int64_t i = half; i < (c.n > 1 ? c.n : 0); i += 16) {
          const float4 ml = p.ws_ml[(i == 0 ? c.slot : 2 * (c.first + i)) * p.gqa + hq % p.gqa];
          const float m_new = fmaxf(M, ml.x);
          l = fmaf(l, fast_exp2(M - m_new), ml.y * fast_exp2(ml.x - m_new));
          M = m_new;
        }
        float top = M;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        l *= fast_exp2(M - top);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        // one piece: written whole by the decode kernel (none: an invalid length)
        if (half == 0 && c.n > 0)
          lse[hq] = c.n == 1 ? p.lse[static_cast<int64_t>(s) * p.num_q_heads + hq] : (top + log2f(l)) * kLn2;
      }
      __syncthreads();
      return lse;
    });
    return;
  }
  const int64_t row = static_cast<int64_t>(blockIdx.x - score_ctas) * (kMergeWarps / kPerRow) + warp / kPerRow;
  Pieces c = {0, 0, 0};
  int h = 0;
  if (row < static_cast<int64_t>(p.num_seqs) * p.num_q_heads) {
    const int s = static_cast<int>(row / p.num_q_heads), hq = static_cast<int>(row % p.num_q_heads);
    h = hq % p.gqa;
    c = pieces_of(p, merge_prefix, W, U, s, hq / p.gqa);
  }
  const int64_t wa = c.first, slot_a = c.slot;
  const int64_t n = c.n == 1 ? 0 : c.n;  // one piece: written whole
  float M = kFloor, o[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f, r = 0.f;
#pragma unroll 1
  for (int64_t i0 = sub; i0 < n; i0 += kMergeBatch * kPerRow) {
    float4 ml[kMergeBatch], ov[kMergeBatch];
    float m_new = M;
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int64_t i = i0 + u * kPerRow;
      ml[u] = make_float4(kFloor, 0.f, 0.f, 0.f);
      ov[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const int64_t at = (i == 0 ? slot_a : 2 * (wa + i)) * p.gqa + h;
        ml[u] = p.ws_ml[at];
        ov[u] = reinterpret_cast<const float4 *>(p.ws_o + at * kD)[lane];
      }
    }
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) m_new = fmaxf(m_new, ml[u].x);
    const float alpha = fast_exp2(M - m_new);
    M = m_new;
    l *= alpha;
    r *= alpha;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] *= alpha;
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
  if constexpr (kPerRow > 1) {
    s_o[warp][lane] = make_float4(o[0], o[1], o[2], o[3]);
    if (lane == 0) s_ml[warp][0] = M, s_ml[warp][1] = l, s_ml[warp][2] = r;
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int w = 1; w < kPerRow; ++w) M = fmaxf(M, s_ml[warp + w][0]);
    o[0] = o[1] = o[2] = o[3] = l = r = 0.f;
#pragma unroll
    for (int w = 0; w < kPerRow; ++w) {
      const float f = fast_exp2(s_ml[warp + w][0] - M);
      const float4 v = s_o[warp + w][lane];
      o[0] = fmaf(v.x, f, o[0]);
      o[1] = fmaf(v.y, f, o[1]);
      o[2] = fmaf(v.z, f, o[2]);
      o[3] = fmaf(v.w, f, o[3]);
      l = fmaf(s_ml[warp + w][1], f, l);
      r = fmaf(s_ml[warp + w][2], f, r);
    }
  }
  if (n == 0) return;
  uint2 v;
  v.x = pack_bf16x2(o[0] / r, o[1] / r);
  v.y = pack_bf16x2(o[2] / r, o[3] / r);
  reinterpret_cast<uint2 *>(p.out + row * kD)[lane] = v;
  if (lane == 0 && p.lse != nullptr) p.lse[row] = (M + log2f(l)) * kLn2;
}

__global__ void __launch_bounds__(kScoreThreads) q4_scores_kernel(const KeyScoresParams p) {
  griddep_wait();
  griddep_launch_dependents();
  key_scores_body<2>(p);
}

// Prefill by rows: every query row of a varlen batch becomes a sequence of its own
// for the decode kernel, with the keys up to its position and its segment's
// table. A row of a segment that the call refuses, and a row behind the last
// segment, gets length 0: it is left out. The bit is raised by a thread a segment,
// also for one without rows, as the widened way's prefill kernel does.
struct Segment {
  int64_t q0, q1, k0, k1;
  bool refused;
};
__device__ __forceinline__ Segment load_segment(const Q4PrefillRowsArgs &a, int s) {
  // four loads in flight together
  Segment g = {a.cu_seqlens_q[s], a.cu_seqlens_q[s + 1], a.cu_seqlens_k[s], a.cu_seqlens_k[s + 1], false};
  const int64_t Lq = g.q1 - g.q0, Lk = g.k1 - g.k0;
  g.refused = g.q0 < 0 || Lq < 0 || Lk < Lq || Lq > a.max_seqlen_q || Lk > a.max_seqlen_k || g.q1 > a.total_q ||
              Lk > static_cast<int64_t>(a.max_blocks) * a.block_size || (Lq > 0 && (g.k0 < 0 || g.k1 > a.total_k));
  return g;
}
__global__ void __launch_bounds__(256) q4_rows_kernel(const Q4PrefillRowsArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x * blockDim.x + threadIdx.x;
  // segments from the last thread on: in a small batch, other warps than those with rows
  const int s = static_cast<int>(gridDim.x * blockDim.x) - 1 - row;
  if (s < a.num_seqs && load_segment(a, s).refused) atomicOr(&g_q4_decode_errors, kErrSeqlens);
  if (row >= a.total_q) return;
  int lo = 0, hi = a.num_seqs - 1;  // the last segment that starts at or before the row
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu_seqlens_q[mid] <= row) lo = mid; else hi = mid - 1;
  }
  const Segment g = load_segment(a, lo);
  const bool in = g.q0 <= row && row < g.q1 && !g.refused;
  a.context_lens[row] = in ? static_cast<int>(g.k1 - g.k0 - (g.q1 - row) + 1) : 0;
  a.table_rows[row] = lo;
}

template <int NG, int kWarps, bool kRanges>
cudaError_t launch_shape(const Q4DecodeParams &p, dim3 grid, cudaStream_t stream) {
  auto kernel = q4_decode_kernel<NG, kWarps, kRanges>;
  // beside the rings and queries, by ranges, what grows with the sequences. The limit
  // is the kernel's, not the call's: another host thread may be between its own two
  // lines here, so it is always set to the most that any call wants.
  constexpr int kFixed = Q4DecodeSmem<NG, kWarps>::kTotal + kWarps * kQueryBytes;
  constexpr auto of_seqs = [](int n) { return kRanges ? 8 * (n + 1) + 4 * n : 0; };
  constexpr int kMost = kFixed + of_seqs(kQ4MaxRangeSeqs);
  static_assert(kMost <= 227 * 1024, "shared memory");
  if (kMost > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, grid, dim3(kWarps * 32), kFixed + of_seqs(p.num_seqs), stream, p);
}

// k: the accumulated weights, or null; added here by ranges with at most
// kMaxScoredHeads query heads.
template <int NG>
cudaError_t launch_plan(const Q4DecodeParams &p, const Q4DecodePlan &plan, const KeyScoresParams *k,
                        cudaStream_t stream) {
  const dim3 pairs(p.num_kv_heads, p.num_seqs);
  if (plan.range_ctas > 0) {
    cudaError_t e = launch_shape<NG, 16, true>(p, dim3(plan.range_ctas), stream);
    if (e != cudaSuccess) return e;
    const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.num_q_heads;
    const int warps = plan.range_ctas * 16;
    // many pieces a pair: as many warps a row as a CTA has
    const bool many = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads * 16 < warps;
    const int64_t ctas = many ? rows : (rows + kMergeWarps - 1) / kMergeWarps;
    // scoring CTAs: two positions a thread if all the CTAs then run at once (two an
    // SM), else four. With 16 heads: 8 sequences of 8,193 keys 28.1 and 28.8 us, 16 of
    // them 46.0 and 44.1
    int64_t chunks = 0;
    bool pairs_of = true;
    if (k != nullptr && p.num_q_heads > kMaxScoredHeads) k = nullptr;  // behind the merge
    if (k != nullptr) {
      chunks = key_scores_grid_x(p.max_context_len, 2);
      pairs_of = ctas + chunks * p.num_seqs <= 2 * plan.range_ctas;
      if (!pairs_of) chunks = key_scores_grid_x(p.max_context_len, 4);
    }
    const size_t smem = sizeof(int64_t) * (p.num_seqs + 1) + (k != nullptr ? sizeof(float) * p.num_q_heads : 0);
    const auto kernel = many ? (pairs_of ? q4_merge_kernel<kMergeWarps, 2> : q4_merge_kernel<kMergeWarps, 4>)
                             : (pairs_of ? q4_merge_kernel<1, 2> : q4_merge_kernel<1, 4>);
    static_assert(8 * (kQ4MaxRangeSeqs + 1) + 4 * kMaxScoredHeads <= 40 * 1024, "no attribute needed, beside the static arrays");
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas + chunks * p.num_seqs)), dim3(kMergeWarps * 32), smem,
                      stream, p, warps, k != nullptr ? *k : KeyScoresParams{},
                      static_cast<int32_t>(chunks * p.num_seqs), static_cast<int32_t>(chunks));
  }
  switch (plan.warps) {
    case 4: return launch_shape<NG, 4, false>(p, pairs, stream);
    case 8: return launch_shape<NG, 8, false>(p, pairs, stream);
    case 16: return launch_shape<NG, 16, false>(p, pairs, stream);
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
  p.table_rows = a.table_rows;
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
  p.num_seqs = a.num_seqs;
  // a scale of 0 becomes the smallest positive one: its logits stay below 2^-100
  // unless a product passes 2^26, and masked logits stay -inf
  p.scale_log2 = fmaxf(fabsf(a.scale_log2), 0x1p-126f);
  p.q_signs = a.scale_log2 < 0.f ? 0x80008000u : 0u;
  KeyScoresParams k = {};
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
  const KeyScoresParams *scores = a.key_scores != nullptr ? &k : nullptr;
  cudaError_t e;
  switch (a.cache.group_size) {
    case 32: e = launch_plan<4>(p, a.plan, scores, stream); break;
    case 64: e = launch_plan<2>(p, a.plan, scores, stream); break;
    case 128: e = launch_plan<1>(p, a.plan, scores, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess || scores == nullptr || (a.plan.range_ctas > 0 && a.num_q_heads <= kMaxScoredHeads)) return e;
  return launch_pdl(q4_scores_kernel, dim3(key_scores_grid_x(a.max_context_len, 2), a.num_seqs),
                    dim3(kScoreThreads), 0, stream, k);
}

cudaError_t launch_q4_prefill_rows(const Q4PrefillRowsArgs &a, cudaStream_t stream) {
  const int threads = a.total_q > a.num_seqs ? a.total_q : a.num_seqs;
  return launch_pdl(q4_rows_kernel, dim3((threads + 255) / 256), dim3(256), 0, stream, a);
}

cudaError_t q4_decode_error_word(uint32_t **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_q4_decode_errors);
}

}  // namespace pkv
