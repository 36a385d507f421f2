// The 4-bit cache's rows: quantise new K/V rows into their slots
// (pkv_kv_store_q4), read rows back by slot (pkv_kv_load_q4), and widen the
// keys of a prefill batch into a bf16 workspace (first half of
// pkv_paged_prefill_attn_q4).
//
// A (token, head)'s K row and V row are handled together, by 8 lanes each in the
// store (16 values a lane) and by 16 in the others (8 values a lane, one 32-bit
// word of codes). A warp has several such pairs' loads in flight.
//
// All three are copies with some arithmetic: HBM bandwidth bounds them, once the
// arithmetic is short enough (the store spends some five packed operations on
// two values) and indices are found without 64-bit divisions. 32,768 tokens of 8
// heads: store 37 us (176 MB, 4.8 TB/s; its issue slots are 74 % used, so it is between
// the two bounds), load 30 us (176 MB, 5.9 TB/s), widening for prefill 28 us
// (6.3 TB/s). With 8 values a lane the store took 10 us more, its per-row work
// being shared by half as many values.
#include "internal.h"
#include "q4.cuh"

namespace pkv {

static __device__ uint32_t g_q4_cache_errors;

namespace {

constexpr int kWarps = 8;
// (token, head) pairs whose loads a warp has in flight (the store's two at a time).
// More leave large calls as they are and lengthen small ones: 64 tokens of 8 heads
// stored and read back 3.6 us in a graph, 5.0 with 4 and 8; 32,768 tokens 63.9 and
// 63.5 (with 2 and 2: 68.7).
constexpr int kStoreRows = 2;
constexpr int kLoadRows = 4;

// The smaller of each half; a NaN in either operand wins.
__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// (smallest, -largest) of the sixteen values of x, as a bf16 pair.
__device__ __forceinline__ uint32_t extremes(const uint32_t (&x)[8]) {
  uint32_t lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan_bf16x2(lo, x[i]);
    hi = max_nan_bf16x2(hi, x[i]);
  }
  hi ^= 0x80008000u;
  return min_nan_bf16x2(q4_low_halves(lo, hi), q4_high_halves(lo, hi));
}

// (scale, offset) of a group with these extremes, as a params word:
//   scale  = bf16(fp32(hi - lo) * fp32(1/15)), 0 if that product is below 2^-100
//   offset = bf16(lo - 16 scale), the value of a code -16
// A group whose spread or offset is not finite (a NaN or an infinity among its
// values, or too wide a range) gets scale 0 and offset NaN.
__device__ __forceinline__ uint32_t group_params(float lo, float hi) {
  const float range = hi - lo;
  float s = range * (1.0f / 15.0f);
  if (s < 0x1p-100f) s = 0.f;
  s = __bfloat162float(__float2bfloat16_rn(s));
  const float b = __bfloat162float(__float2bfloat16_rn(__fsub_rn(lo + 0.f, __fmul_rn(16.f, s))));
  if (!(fabsf(range) <= 3.4e38f) || !(fabsf(b) <= 3.4e38f)) return 0x7FC00000u;
  return pack_bf16x2(s, b);
}

// Codes of the eight values in four words, n = clamp(floor(t / s + 1/2) - 16, 0, 15)
// with t = fp32(x - b), one value at a time. The quotient is only estimated and
// rounded to the nearest integer c; the remainder t - c s, where it is near the
// thresholds -s / 2 and s / 2 exact in fp32 (s has 8 bits, c at most 7), settles it.
// t may be infinite: its code is the last one.
__device__ __noinline__ uint32_t codes_one_by_one(uint4 x, float s, float b) {
  const float r = 1.f / s, h = 0.5f * s;
  const uint32_t wx[4] = {x.x, x.y, x.z, x.w};
  uint32_t codes = 0;
  for (int i = 0; i < 8; ++i) {
    const float t = ((i & 1) ? bf16hi(wx[i >> 1]) : bf16lo(wx[i >> 1])) - b;
    float c = rintf(fminf(fmaxf(t * r, 0.f), 100.f));
    const float rest = fmaf(-c, s, t);
    if (rest >= h) c += 1.f;
    else if (rest < -h) c -= 1.f;
    const int n = min(max(static_cast<int>(c) - 16, 0), 15);
    codes |= static_cast<uint32_t>(n) << (4 * i);
  }
  return codes;
}

// The same for sixteen values, two at a time. y = t r' + M, with r' a little
// above 1 / s and M = 2^23 + 2^22 - 16, rounds the quotient to an integer c in its
// low mantissa bits, which then hold the code. r' exceeds the reciprocal by 2^-19,
// more than the estimate's own error, so that a half (common: the inputs have 8
// bits) rounds up and a quotient at most 2^-14 below one may do so wrongly: the
// remainder t - c s, exact in fp32, is then below -s / 2 and the code one less (the
// sign of remainder + s / 2, as an integer, is added).
// Only groups whose offset's rounding pushes an extreme past the code range, or
// whose differences overflow, need clamping; they take the other way.
__device__ __forceinline__ uint2 codes_of(const uint32_t (&x)[8], uint32_t pw, float lo, float hi) {
  constexpr float kM = 12582896.f;
  const float s = bf16lo(pw), b = bf16hi(pw);
  if (s == 0.f) return make_uint2(0u, 0u);
  if (lo - b < 15.75f * s || hi - b > fminf(31.25f * s, 3.4e38f))  // an infinite difference, too
    return make_uint2(codes_one_by_one(make_uint4(x[0], x[1], x[2], x[3]), s, b),
                      codes_one_by_one(make_uint4(x[4], x[5], x[6], x[7]), s, b));
  const float r = __fdividef(1.f + 0x1p-19f, s), h = 0.5f * s;
  const uint64_t nb2 = f32x2(-b, -b), r2 = f32x2(r, r), m2 = f32x2(kM, kM), s2 = f32x2(s, s);
  const uint64_t one2 = f32x2(1.f, 1.f), neg2 = f32x2(-1.f, -1.f), h2 = f32x2(h, h);
  uint32_t byte[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t t = fma2(f32x2(bf16lo(x[i]), bf16hi(x[i])), one2, nb2);
    const uint64_t y = fma2(t, r2, m2);
    const uint64_t rest = fma2(fma2(y, neg2, m2), s2, t);  // t - c s
    const uint64_t over = fma2(rest, one2, h2);            // its sign is exact
    const int n0 = static_cast<int>(y) + (static_cast<int>(over) >> 31);
    const int n1 = static_cast<int>(y >> 32) + (static_cast<int>(over >> 32) >> 31);
    byte[i] = n1 * 16 + n0;  // its low byte
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = __byte_perm(__byte_perm(byte[4 * i], byte[4 * i + 1], 0x0040),
                       __byte_perm(byte[4 * i + 2], byte[4 * i + 3], 0x0040), 0x5410);
  return make_uint2(w[0], w[1]);
}

struct Q4RowsParams {
  const uint4 *k, *v;             // store: rows [T, H_kv, 128] bf16
  uint4 *k_out, *v_out;           // load: the same, written
  uint32_t *k_codes, *v_codes;    // eight codes a word
  uint32_t *k_params, *v_params;  // (scale, offset) words
  const int32_t *slots;
  FastDiv heads, block;
  int32_t groups_log2;            // log2 of the groups a row
  uint32_t num_rows;              // T * H_kv
  int64_t num_slots;
};

// 32 bytes, 32-byte aligned or (two loads) 16-byte aligned.
__device__ __forceinline__ void ld_stream(const uint4 *p, uint32_t (&r)[8]) {
  const uint4 a = __ldcs(p), b = __ldcs(p + 1);
  r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w;
  r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
}

// Where (token, head) pair i lives: its row in the codes and params arrays, or
// -1 for none; an invalid slot raises its bit and counts as none.
__device__ __forceinline__ int64_t cache_row(const Q4RowsParams &p, uint32_t i, int lane) {
  if (i >= p.num_rows) return -1;
  const uint32_t token = fast_quotient(i, p.heads), head = i - token * p.heads.d;
  const int32_t slot = p.slots[token];
  if (slot < 0 || slot >= p.num_slots) {
    if (slot != -1 && lane == 0) atomicOr(&g_q4_cache_errors, kErrSlot);
    return -1;
  }
  const uint32_t blk = fast_quotient(slot, p.block), off = slot - blk * p.block.d;
  return (static_cast<int64_t>(blk) * p.heads.d + head) * p.block.d + off;
}

__global__ void __launch_bounds__(kWarps * 32) q4_store_kernel(const Q4RowsParams p) {
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane & 7;
  const bool is_v = (lane & 8) != 0;
  const uint32_t first = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kStoreRows + (lane >> 4);
  const uint4 *in = is_v ? p.v : p.k;
  uint32_t x[kStoreRows / 2][8];
  int64_t row[kStoreRows / 2];
#pragma unroll
  for (int u = 0; u < kStoreRows / 2; ++u) {
    const uint32_t i = first + 2 * u;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[u][j] = 0;
    if (i < p.num_rows) ld_stream(in + static_cast<int64_t>(i) * 16 + 2 * l, x[u]);
  }
#pragma unroll
  for (int u = 0; u < kStoreRows / 2; ++u) row[u] = cache_row(p, first + 2 * u, lane & 15);
  uint32_t *codes = is_v ? p.v_codes : p.k_codes, *params = is_v ? p.v_params : p.k_params;
  const int lanes_log2 = 3 - p.groups_log2;  // lanes sharing a group
#pragma unroll
  for (int u = 0; u < kStoreRows / 2; ++u) {
    if (first - (lane >> 4) + 2 * u >= p.num_rows) break;  // uniform over the warp
    uint32_t e = extremes(x[u]);
    e = min_nan_bf16x2(e, __shfl_xor_sync(0xffffffffu, e, 1));
    if (lanes_log2 >= 2) e = min_nan_bf16x2(e, __shfl_xor_sync(0xffffffffu, e, 2));
    if (lanes_log2 >= 3) e = min_nan_bf16x2(e, __shfl_xor_sync(0xffffffffu, e, 4));
    const float lo = bf16lo(e), hi = -bf16hi(e);
    const uint32_t pw = group_params(lo, hi);
    if (row[u] < 0) continue;
    reinterpret_cast<uint2 *>(codes)[row[u] * 8 + l] = codes_of(x[u], pw, lo, hi);
    if ((l & ((1 << lanes_log2) - 1)) == 0) params[(row[u] << p.groups_log2) + (l >> lanes_log2)] = pw;
  }
}

__global__ void __launch_bounds__(kWarps * 32) q4_load_kernel(const Q4RowsParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool is_v = lane >= 16;
  const uint32_t first = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kLoadRows;
  const uint32_t *codes = is_v ? p.v_codes : p.k_codes, *params = is_v ? p.v_params : p.k_params;
  const int lanes_log2 = 4 - p.groups_log2;
  uint32_t w[kLoadRows], pw[kLoadRows];
#pragma unroll
  for (int u = 0; u < kLoadRows; ++u) {
    const int64_t row = cache_row(p, first + u, lane);
    w[u] = pw[u] = 0;  // no slot: zeros
    if (row >= 0) {
      w[u] = codes[row * 16 + l];
      pw[u] = params[(row << p.groups_log2) + (l >> lanes_log2)];
    }
  }
  uint4 *out = is_v ? p.v_out : p.k_out;
#pragma unroll
  for (int u = 0; u < kLoadRows; ++u)
    if (first + u < p.num_rows) out[static_cast<int64_t>(first + u) * 16 + l] = q4_widen(w[u], pw[u]);
}

// Widen the keys of a prefill batch into bf16 blocks of kQ4PrefillBlock rows in
// the workspace, whose block tables it writes. Sequence s starts at workspace
// block ceil(cu_k[s] / block) + s, which leaves every sequence its
// ceil(Lk / block) blocks. Grid: (chunks, sequences); a warp takes 16 keys of one
// head, which lie in one cache block: one table entry, 1 KiB of K and of V codes.
struct Q4GatherParams {
  const int32_t *cu_q, *cu_k, *block_tables;
  const uint32_t *k_codes, *v_codes, *k_params, *v_params;
  uint4 *k_out, *v_out;         // workspace K and V [blocks, kQ4PrefillBlock, H_kv, 128]
  int32_t *ws_tables;           // [S, ws_max_blocks]
  FastDiv heads, block;
  int32_t max_blocks, ws_max_blocks, max_seqlen_q, max_seqlen_k, total_k;
  int32_t groups_log2, num_blocks, window;
};
constexpr int kGatherKeys = 16;

__global__ void __launch_bounds__(kWarps * 32) q4_gather_kernel(const Q4GatherParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.y;
  const int k_begin = p.cu_k[s], k_end = p.cu_k[s + 1];
  const int q_begin = p.cu_q[s], q_end = p.cu_q[s + 1];
  const int64_t Lk64 = static_cast<int64_t>(k_end) - k_begin, Lq64 = static_cast<int64_t>(q_end) - q_begin;
  // segments that the prefill kernel refuses (it raises the bit) are not widened
  const bool ok = Lk64 > 0 && Lq64 > 0 && Lq64 <= Lk64 && Lq64 <= p.max_seqlen_q && Lk64 <= p.max_seqlen_k &&
                  k_begin >= 0 && k_end <= p.total_k &&
                  Lk64 <= static_cast<int64_t>(p.max_blocks) * p.block.d;
  const int Lk = ok ? static_cast<int>(Lk64) : 0, Lq = ok ? static_cast<int>(Lq64) : 0;
  const int ws_block0 = ok ? (k_begin + kQ4PrefillBlock - 1) / kQ4PrefillBlock + s : 0;
  for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < p.ws_max_blocks; j += gridDim.x * blockDim.x)
    p.ws_tables[static_cast<int64_t>(s) * p.ws_max_blocks + j] =
        j < (Lk + kQ4PrefillBlock - 1) / kQ4PrefillBlock ? ws_block0 + j : -1;
  // keys before the first query's window are masked, but those in its tile (a
  // workspace block) are still multiplied, by zeros: they must hold numbers
  const int first_seen = p.window > 0 ? max(0, Lk - Lq - p.window + 1) : 0;
  const int first_key = first_seen / kQ4PrefillBlock * kQ4PrefillBlock;
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool is_v = lane >= 16;
  const uint32_t *codes = is_v ? p.v_codes : p.k_codes, *params = is_v ? p.v_params : p.k_params;
  uint4 *out = is_v ? p.v_out : p.k_out;
  const int lanes_log2 = 4 - p.groups_log2;
  const int64_t H = p.heads.d;
  // units of 16 keys, the heads of one key range after each other: what the
  // warps write together is contiguous
  const int64_t n_units = (static_cast<int64_t>(Lk - first_key) + kGatherKeys - 1) / kGatherKeys * H;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); unit < n_units;
       unit += n_warps) {
    const uint32_t chunk = fast_quotient(static_cast<uint32_t>(unit), p.heads);
    const uint32_t head = static_cast<uint32_t>(unit) - chunk * p.heads.d;
    const int pos0 = first_key + static_cast<int>(chunk) * kGatherKeys;
    const int n = min(kGatherKeys, Lk - pos0);
    const uint32_t j = fast_quotient(pos0, p.block);
    const int blk = p.block_tables[static_cast<int64_t>(s) * p.max_blocks + j];
    const bool there = blk >= 0 && blk < p.num_blocks;
    if (!there && lane == 0 && pos0 + n > first_seen) atomicOr(&g_q4_cache_errors, kErrBlock);
    const int64_t row0 = there ? (blk * H + head) * p.block.d + (pos0 - j * p.block.d) : 0;
    uint4 *dst = out + ((static_cast<int64_t>(ws_block0) * kQ4PrefillBlock + pos0) * H + head) * 16 + l;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t w[kGatherKeys / 2], pw[kGatherKeys / 2];
#pragma unroll
      for (int u = 0; u < kGatherKeys / 2; ++u) {
        const int i = half * (kGatherKeys / 2) + u;
        w[u] = pw[u] = 0;  // no such block: zeros
        if (there && i < n) {
          w[u] = codes[(row0 + i) * 16 + l];
          pw[u] = params[((row0 + i) << p.groups_log2) + (l >> lanes_log2)];
        }
      }
#pragma unroll
      for (int u = 0; u < kGatherKeys / 2; ++u) {
        const int i = half * (kGatherKeys / 2) + u;
        if (i < n) dst[i * H * 16] = q4_widen(w[u], pw[u]);
      }
    }
  }
}

int32_t groups_log2(int32_t group_size) { return group_size == 32 ? 2 : group_size == 64 ? 1 : 0; }

Q4RowsParams rows_params(const Q4RowsArgs &a) {
  Q4RowsParams p;
  p.k = static_cast<const uint4 *>(a.k);
  p.v = static_cast<const uint4 *>(a.v);
  p.k_out = static_cast<uint4 *>(a.k_out);
  p.v_out = static_cast<uint4 *>(a.v_out);
  p.k_codes = static_cast<uint32_t *>(a.cache.k_codes);
  p.v_codes = static_cast<uint32_t *>(a.cache.v_codes);
  p.k_params = static_cast<uint32_t *>(a.cache.k_params);
  p.v_params = static_cast<uint32_t *>(a.cache.v_params);
  p.slots = a.slots;
  p.heads = fast_div(a.cache.num_kv_heads);
  p.block = fast_div(a.cache.block_size);
  p.groups_log2 = groups_log2(a.cache.group_size);
  p.num_rows = static_cast<uint32_t>(a.num_tokens) * static_cast<uint32_t>(a.cache.num_kv_heads);
  p.num_slots = a.cache.num_blocks * a.cache.block_size;
  return p;
}

// The caller has checked that num_tokens * num_kv_heads is below 2^31.
cudaError_t launch_rows(void (*kernel)(Q4RowsParams), int rows, const Q4RowsArgs &a, cudaStream_t stream) {
  const Q4RowsParams p = rows_params(a);
  const uint32_t per_cta = kWarps * rows;
  return launch_pdl(kernel, dim3((p.num_rows + per_cta - 1) / per_cta), dim3(kWarps * 32), 0, stream, p);
}

}  // namespace

cudaError_t launch_q4_store(const Q4RowsArgs &a, cudaStream_t stream) {
  return launch_rows(q4_store_kernel, kStoreRows, a, stream);
}

cudaError_t launch_q4_load(const Q4RowsArgs &a, cudaStream_t stream) {
  return launch_rows(q4_load_kernel, kLoadRows, a, stream);
}

cudaError_t launch_q4_gather(const Q4GatherArgs &a, cudaStream_t stream) {
  Q4GatherParams p;
  p.cu_q = a.cu_seqlens_q;
  p.cu_k = a.cu_seqlens_k;
  p.block_tables = a.block_tables;
  p.k_codes = static_cast<const uint32_t *>(a.cache.k_codes);
  p.v_codes = static_cast<const uint32_t *>(a.cache.v_codes);
  p.k_params = static_cast<const uint32_t *>(a.cache.k_params);
  p.v_params = static_cast<const uint32_t *>(a.cache.v_params);
  p.k_out = static_cast<uint4 *>(a.ws_k);
  p.v_out = static_cast<uint4 *>(a.ws_v);
  p.ws_tables = a.ws_tables;
  p.max_blocks = a.max_blocks;
  p.ws_max_blocks = a.ws_max_blocks;
  p.max_seqlen_q = a.max_seqlen_q;
  p.max_seqlen_k = a.max_seqlen_k;
  p.total_k = a.total_k;
  p.heads = fast_div(a.cache.num_kv_heads);
  p.block = fast_div(a.cache.block_size);
  p.groups_log2 = groups_log2(a.cache.group_size);
  p.num_blocks = static_cast<int32_t>(a.cache.num_blocks);
  p.window = a.window;
  // CTAs a sequence for its longest possible key range, at most some 16 an SM in all
  const int64_t units = (static_cast<int64_t>(a.max_seqlen_k) + kGatherKeys - 1) / kGatherKeys * a.cache.num_kv_heads;
  int64_t gx = (units + kWarps - 1) / kWarps;
  const int64_t cap = (16 * static_cast<int64_t>(a.num_sms) + a.num_seqs - 1) / a.num_seqs;
  if (gx > cap) gx = cap;
  return launch_pdl(q4_gather_kernel, dim3(static_cast<unsigned>(gx), a.num_seqs), dim3(kWarps * 32),
                    0, stream, p);
}

cudaError_t q4_cache_error_word(uint32_t **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_q4_cache_errors);
}

}  // namespace pkv
