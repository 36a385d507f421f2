// The 4-bit cache's rows: quantise new K/V rows into their slots
// (pkv_kv_store_q4), read rows back by slot (pkv_kv_load_q4), and widen the
// keys of a prefill batch into a bf16 workspace (first half of
// pkv_paged_prefill_attn_q4).
//
// Half a warp handles one row of 128 values: eight values a lane, so that a
// lane's codes are one 32-bit word; lanes 0-15 take a (token, head)'s K row and
// lanes 16-31 its V row. Each warp has kRowsInFlight such pairs' loads in
// flight.
#include "internal.h"
#include "q4.cuh"

namespace pkv {

static __device__ uint32_t g_q4_cache_errors;

namespace {

constexpr int kWarps = 8;
constexpr int kRowsInFlight = 4;

// (scale, offset) of a group with these extremes, as a params word:
//   scale  = bf16(fp32(hi - lo) * fp32(1/15)), 0 if that product is below 2^-100
//   offset = bf16(lo - 16 scale), the value of a code -16
// A group whose spread or offset is not finite (a NaN or an infinity among its
// values, or too wide a range) gets scale 0 and offset NaN.
__device__ __forceinline__ uint32_t group_params(float lo, float hi, bool nan) {
  const float range = hi - lo;
  float s = range * (1.0f / 15.0f);
  if (s < 0x1p-100f) s = 0.f;
  s = __bfloat162float(__float2bfloat16_rn(s));
  const float b = __bfloat162float(__float2bfloat16_rn(__fsub_rn(lo + 0.f, __fmul_rn(16.f, s))));
  if (nan || !(fabsf(range) <= 3.4e38f) || !(fabsf(b) <= 3.4e38f)) return 0x7FC00000u;
  return pack_bf16x2(s, b);
}

// Codes of the eight values of x (four words of two bf16): with t = fp32(x - b),
// n = clamp(floor(t / s + 1/2) - 16, 0, 15). The quotient is only estimated
// (t * (1/s), rounded to the nearest integer c); the two comparisons with the
// thresholds (c - 1/2) s and (c + 1/2) s, which are exact in fp32 (s has 8
// bits, c at most 6), settle it.
__device__ __forceinline__ uint32_t codes_of(const uint4 x, uint32_t pw) {
  const float s = bf16lo(pw), b = bf16hi(pw);
  if (s == 0.f) return 0u;
  const float r = 1.f / s, h = 0.5f * s;
  const uint32_t wx[4] = {x.x, x.y, x.z, x.w};
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = ((i & 1) ? bf16hi(wx[i >> 1]) : bf16lo(wx[i >> 1])) - b;
    float c = rintf(t * r);
    const float at = c * s;
    if (t >= at + h) c += 1.f;
    else if (t < at - h) c -= 1.f;
    const int n = min(max(static_cast<int>(c) - 16, 0), 15);
    codes |= static_cast<uint32_t>(n) << (4 * i);
  }
  return codes;
}

struct Q4RowsParams {
  const uint4 *k, *v;           // store: rows [T, H_kv, 128] bf16
  uint4 *k_out, *v_out;         // load: the same, written
  uint32_t *k_codes, *v_codes;    // eight codes a word
  uint32_t *k_params, *v_params;  // (scale, offset) words
  const int32_t *slots;
  int32_t num_kv_heads, block_size, groups;
  int64_t num_rows;             // T * H_kv
  int64_t num_slots;
};

// Row index of a slot's row of head h in the codes and params arrays.
__device__ __forceinline__ int64_t q4_row(int64_t slot, int h, int num_kv_heads, int block_size) {
  const int64_t blk = slot / block_size;
  return (blk * num_kv_heads + h) * block_size + (slot - blk * block_size);
}

__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// The slot of row i (a (token, head) pair), or -1 for none; an invalid one
// raises its bit and counts as none.
__device__ __forceinline__ int64_t slot_of_row(const Q4RowsParams &p, int64_t i, int lane) {
  if (i >= p.num_rows) return -1;
  const int64_t slot = p.slots[i / p.num_kv_heads];
  if (slot < -1 || slot >= p.num_slots) {
    if (lane == 0) atomicOr(&g_q4_cache_errors, kErrSlot);
    return -1;
  }
  return slot;
}

__global__ void __launch_bounds__(kWarps * 32) q4_store_kernel(const Q4RowsParams p) {
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, kv = lane >> 4, l = lane & 15;
  const int64_t first =
      (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kRowsInFlight;
  int64_t slot[kRowsInFlight];
  uint4 x[kRowsInFlight];
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u) {
    slot[u] = slot_of_row(p, first + u, lane);
    if (slot[u] >= 0) x[u] = ld_stream((kv ? p.v : p.k) + (first + u) * 16 + l);
  }
  const int per_group = 16 / p.groups;  // lanes sharing a group
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u) {
    if (slot[u] < 0) continue;  // uniform over the warp
    const uint32_t wx[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
    float lo = bf16lo(wx[0]), hi = lo;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = (i & 1) ? bf16hi(wx[i >> 1]) : bf16lo(wx[i >> 1]);
      lo = fminf(lo, f);
      hi = fmaxf(hi, f);
      nan |= f != f;
    }
    for (int off = 1; off < per_group; off <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
      nan |= __shfl_xor_sync(0xffffffffu, static_cast<int>(nan), off) != 0;
    }
    const uint32_t pw = group_params(lo, hi, nan);
    const int64_t row = q4_row(slot[u], static_cast<int>((first + u) % p.num_kv_heads),
                               p.num_kv_heads, p.block_size);
    (kv ? p.v_codes : p.k_codes)[row * 16 + l] = codes_of(x[u], pw);
    if (l % per_group == 0) (kv ? p.v_params : p.k_params)[row * p.groups + l / per_group] = pw;
  }
}

__global__ void __launch_bounds__(kWarps * 32) q4_load_kernel(const Q4RowsParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, kv = lane >> 4, l = lane & 15;
  const int64_t first =
      (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kRowsInFlight;
  const int per_group = 16 / p.groups;
  uint32_t w[kRowsInFlight], pw[kRowsInFlight];
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u) {
    const int64_t slot = slot_of_row(p, first + u, lane);
    w[u] = pw[u] = 0;  // no slot: zeros
    if (slot >= 0) {
      const int64_t row = q4_row(slot, static_cast<int>((first + u) % p.num_kv_heads),
                                 p.num_kv_heads, p.block_size);
      w[u] = (kv ? p.v_codes : p.k_codes)[row * 16 + l];
      pw[u] = (kv ? p.v_params : p.k_params)[row * p.groups + l / per_group];
    }
  }
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u)
    if (first + u < p.num_rows) (kv ? p.v_out : p.k_out)[(first + u) * 16 + l] = q4_widen(w[u], pw[u]);
}

// Widen the keys of a prefill batch into bf16 blocks of kQ4PrefillBlock rows in
// the workspace, whose block tables it writes. Sequence s starts at workspace
// block ceil(cu_k[s] / block) + s, which leaves every sequence its
// ceil(Lk / block) blocks. Grid: (row chunks, sequences); a warp widens the
// kRowsInFlight (position, head) pairs that follow each other.
struct Q4GatherParams {
  const int32_t *cu_q, *cu_k, *block_tables;
  const uint32_t *k_codes, *v_codes, *k_params, *v_params;
  uint4 *k_out, *v_out;         // workspace K and V [blocks, kQ4PrefillBlock, H_kv, 128]
  int32_t *ws_tables;           // [S, ws_max_blocks]
  int32_t max_blocks, ws_max_blocks, num_seqs, max_seqlen_q, max_seqlen_k, total_k;
  int32_t num_kv_heads, block_size, groups, num_blocks, window;
};

__global__ void __launch_bounds__(kWarps * 32) q4_gather_kernel(const Q4GatherParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.y;
  const int k_begin = p.cu_k[s], k_end = p.cu_k[s + 1];
  const int Lk = k_end - k_begin, Lq = p.cu_q[s + 1] - p.cu_q[s];
  // segments the prefill kernel refuses are not widened (it raises the bit):
  // here they also must not pass the workspace's end
  if (Lk <= 0 || Lq <= 0 || Lq > Lk || Lq > p.max_seqlen_q || Lk > p.max_seqlen_k || k_begin < 0 ||
      k_end > p.total_k || static_cast<int64_t>(Lk) > static_cast<int64_t>(p.max_blocks) * p.block_size) {
    // empty or refused: no workspace block for it. A segment that only passes
    // total_k is refused here, since the prefill kernel does not know it.
    if (k_end > p.total_k && Lq > 0 && blockIdx.x == 0 && threadIdx.x == 0)
      atomicOr(&g_q4_cache_errors, kErrSeqlens);
    for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < p.ws_max_blocks; j += gridDim.x * blockDim.x)
      p.ws_tables[static_cast<int64_t>(s) * p.ws_max_blocks + j] = -1;
    return;
  }
  const int ws_block0 = (k_begin + kQ4PrefillBlock - 1) / kQ4PrefillBlock + s;
  for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < p.ws_max_blocks; j += gridDim.x * blockDim.x)
    p.ws_tables[static_cast<int64_t>(s) * p.ws_max_blocks + j] =
        j < (Lk + kQ4PrefillBlock - 1) / kQ4PrefillBlock ? ws_block0 + j : -1;
  // keys before the first query's window are masked, but those in its tile (a
  // workspace block) are still multiplied, by zeros: they must hold numbers
  const int first_seen = p.window > 0 ? max(0, Lk - Lq - p.window + 1) : 0;
  const int first_key = first_seen / kQ4PrefillBlock * kQ4PrefillBlock;
  const int lane = threadIdx.x & 31, kv = lane >> 4, l = lane & 15;
  const int per_group = 16 / p.groups;
  const int64_t H = p.num_kv_heads, n_rows = (Lk - first_key) * H;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kRowsInFlight;
       i0 < n_rows; i0 += n_warps * kRowsInFlight) {
    uint32_t w[kRowsInFlight], pw[kRowsInFlight];
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      w[u] = pw[u] = 0;
      const int64_t i = i0 + u;
      if (i >= n_rows) continue;
      const int pos = first_key + static_cast<int>(i / H);
      const int blk = p.block_tables[static_cast<int64_t>(s) * p.max_blocks + pos / p.block_size];
      if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0 && pos >= first_seen) atomicOr(&g_q4_cache_errors, kErrBlock);
        continue;  // zeros
      }
      const int64_t row = (blk * H + i % H) * p.block_size + pos % p.block_size;
      w[u] = (kv ? p.v_codes : p.k_codes)[row * 16 + l];
      pw[u] = (kv ? p.v_params : p.k_params)[row * p.groups + l / per_group];
    }
    const int64_t out0 = (static_cast<int64_t>(ws_block0) * kQ4PrefillBlock + first_key) * H + i0;
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u)
      if (i0 + u < n_rows) (kv ? p.v_out : p.k_out)[(out0 + u) * 16 + l] = q4_widen(w[u], pw[u]);
  }
}

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
  p.num_kv_heads = a.cache.num_kv_heads;
  p.block_size = a.cache.block_size;
  p.groups = kQ4D / a.cache.group_size;
  p.num_rows = static_cast<int64_t>(a.num_tokens) * a.cache.num_kv_heads;
  p.num_slots = a.cache.num_blocks * a.cache.block_size;
  return p;
}

cudaError_t launch_rows(void (*kernel)(Q4RowsParams), const Q4RowsArgs &a, cudaStream_t stream) {
  const Q4RowsParams p = rows_params(a);
  const int64_t per_cta = kWarps * kRowsInFlight;
  const int64_t grid = (p.num_rows + per_cta - 1) / per_cta;
  if (grid == 0) return cudaSuccess;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kWarps * 32), 0, stream, p);
}

}  // namespace

cudaError_t launch_q4_store(const Q4RowsArgs &a, cudaStream_t stream) {
  return launch_rows(q4_store_kernel, a, stream);
}

cudaError_t launch_q4_load(const Q4RowsArgs &a, cudaStream_t stream) {
  return launch_rows(q4_load_kernel, a, stream);
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
  p.num_seqs = a.num_seqs;
  p.max_seqlen_q = a.max_seqlen_q;
  p.max_seqlen_k = a.max_seqlen_k;
  p.total_k = a.total_k;
  p.num_kv_heads = a.cache.num_kv_heads;
  p.block_size = a.cache.block_size;
  p.groups = kQ4D / a.cache.group_size;
  p.num_blocks = static_cast<int32_t>(a.cache.num_blocks);
  p.window = a.window;
  // enough CTAs a sequence for its longest possible key range, a few rounds each
  const int64_t per_cta = kWarps * kRowsInFlight;
  int64_t gx = (static_cast<int64_t>(a.max_seqlen_k) * a.cache.num_kv_heads + per_cta - 1) / per_cta;
  const int64_t cap = (16 * static_cast<int64_t>(a.num_sms) + a.num_seqs - 1) / a.num_seqs;
  if (gx > cap) gx = cap;
  return launch_pdl(q4_gather_kernel, dim3(static_cast<unsigned>(gx), a.num_seqs), dim3(kWarps * 32),
                    0, stream, p);
}

cudaError_t q4_cache_error_word(uint32_t **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_q4_cache_errors);
}

}  // namespace pkv
