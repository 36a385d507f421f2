// Eviction from the paged cache by accumulated attention weight: which tokens
// of each sequence stay (evict_select) and moving their rows together
// (evict_compact).
//
// Selection. One CTA a sequence finds the want-th largest score with a radix
// select over the scores' order-preserving 32-bit keys, eight bits a pass, then
// writes the kept positions in ascending order: each warp owns a contiguous
// range of positions, counts the keys above and at the threshold, and after one
// scan over the warps writes its own with ballots. Equal scores are taken from
// the lowest position on.
//
// Compaction. Row i of the destination is row keep[i] >= i of the source, so
// that in place nothing is overwritten before it has been read when the rows go
// in order: a CTA owns a slice (up to 64 bytes) of every row of one sequence
// and moves its rows in chunks, loading a whole chunk before it stores any of
// it. Slices are independent, which is what spreads one sequence over the SMs.
#include "internal.h"
#include "ptx.cuh"

namespace pkv {

static __device__ uint32_t g_evict_errors;

namespace {

// ---------------------------------------------------------------- selection

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;
constexpr int kHistCopies = 8;  // histograms a warp group of four shares, against contention

struct SelectParams {
  const float *key_scores;
  int64_t score_stride;
  const int32_t *context_lens;
  int32_t *keep, *new_lens;
  int32_t max_context_len, budget, recent;
};

// Larger scores have larger keys; NaN sorts below every number; -0 equals 0.
__device__ __forceinline__ uint32_t score_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectParams p) {
  __shared__ uint32_t hist[kHistCopies][kBins];
  __shared__ uint32_t s_prefix, s_want;
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  griddep_launch_dependents();
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctx = p.context_lens[s];
  if (ctx < 0 || ctx > p.max_context_len) {
    if (tid == 0) atomicOr(&g_evict_errors, kErrContext);
    return;
  }
  const float *score = p.key_scores + s * p.score_stride;
  int32_t *keep = p.keep + static_cast<int64_t>(s) * p.budget;
  const int new_len = min(ctx, p.budget), recent = min(ctx, p.recent);
  const int old = ctx - recent;         // positions that compete
  const int want = new_len - recent;    // how many of them stay
  if (tid == 0) p.new_lens[s] = new_len;
  for (int i = new_len + tid; i < p.budget; i += kSelThreads) keep[i] = -1;
  for (int i = tid; i < recent; i += kSelThreads) keep[want + i] = old + i;
  if (want == old) {  // nothing to evict
    for (int i = tid; i < old; i += kSelThreads) keep[i] = i;
    return;
  }
  if (want == 0) return;

  // ---- the want-th largest key, most significant digit first
  uint32_t prefix = 0, left = want;  // keys above the prefix are in; left more come from below it
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < kHistCopies * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    uint32_t *h = hist[warp % kHistCopies];
    for (int i = tid; i < old; i += kSelThreads) {
      const uint32_t k = score_key(score[i]);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&h[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l sums bins 255 - 8 l .. 248 - 8 l, highest first
      uint32_t n[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[j] = 0;
        for (int c = 0; c < kHistCopies; ++c) n[j] += hist[c][255 - 8 * lane - j];
        sum += n[j];
      }
      uint32_t above = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, above, off);
        if (lane >= off) above += v;
      }
      above -= sum;  // keys in higher lanes' bins
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (above < left && left <= above + n[j]) {
          s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - j) << shift);
          s_want = left - above;
        }
        above += n[j];
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_want;
  }

  // ---- kept positions in order: keys above the threshold, and the first
  // `left` of those equal to it
  const int per_warp = ((old + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int begin = min(old, warp * per_warp), end = min(old, begin + per_warp);
  int gt = 0, eq = 0;
  for (int i = begin + lane; i - lane < end; i += 32) {
    const uint32_t k = i < end ? score_key(score[i]) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i < end && k > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, i < end && k == prefix));
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  int gt0 = 0, eq0 = 0;  // in the warps before
  for (int w = 0; w < warp; ++w) {
    gt0 += s_gt[w];
    eq0 += s_eq[w];
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i = begin + lane; i - lane < end; i += 32) {
    const uint32_t k = i < end ? score_key(score[i]) : 0u;
    const uint32_t bg = __ballot_sync(0xffffffffu, i < end && k > prefix);
    const uint32_t be = __ballot_sync(0xffffffffu, i < end && k == prefix);
    const int my_gt = gt0 + __popc(bg & below), my_eq = eq0 + __popc(be & below);
    const bool in = ((bg >> lane) & 1u) || (((be >> lane) & 1u) && my_eq < static_cast<int>(left));
    if (in) keep[my_gt + min(my_eq, static_cast<int>(left))] = i;
    gt0 += __popc(bg);
    eq0 += __popc(be);
  }
}

// ---------------------------------------------------------------- compaction

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;       // rows a thread has in flight

struct CompactParams {
  RowArray arrays[kMaxRowArrays];
  int32_t num_arrays;
  const int32_t *src_tables, *dst_tables, *keep, *new_lens;
  const float *key_scores;           // [S, score_stride] or null
  float *dst_key_scores;             // [S, dst_score_stride]
  int64_t score_stride, dst_score_stride;
  int32_t src_max_blocks, dst_max_blocks, budget, block_size, num_blocks;
};

template <int N> struct Piece;
template <> struct Piece<16> { using T = uint4; };
template <> struct Piece<8> { using T = uint2; };
template <> struct Piece<4> { using T = uint32_t; };

// Byte offset of position pos's row of one plane, or -1 (with its bit raised)
// for a position or block that does not exist.
__device__ __forceinline__ int64_t row_offset(const CompactParams &p, const int32_t *table, int max_blocks,
                                              const RowArray &a, int plane, int pos) {
  const int j = pos / p.block_size;
  if (pos < 0 || j >= max_blocks) {
    atomicOr(&g_evict_errors, kErrContext);
    return -1;
  }
  const int blk = table[j];
  if (blk < 0 || blk >= p.num_blocks) {
    atomicOr(&g_evict_errors, kErrBlock);
    return -1;
  }
  return ((static_cast<int64_t>(blk) * a.planes + plane) * p.block_size + (pos - j * p.block_size)) * a.row_bytes;
}

// Move `bytes` bytes at `at` of every kept row of one plane, N bytes a thread.
template <int N>
__device__ void move_slice(const CompactParams &p, const RowArray &a, int plane, int at, int bytes, int s, int n) {
  using T = typename Piece<N>::T;
  const int per_row = bytes / N;
  const int rows = kMoveThreads / per_row;  // rows a step
  const int r = threadIdx.x / per_row, c = at + threadIdx.x % per_row * N;
  const int32_t *keep = p.keep + static_cast<int64_t>(s) * p.budget;
  const int32_t *src = p.src_tables + static_cast<int64_t>(s) * p.src_max_blocks;
  const int32_t *dst = p.dst_tables + static_cast<int64_t>(s) * p.dst_max_blocks;
  uint8_t *base = static_cast<uint8_t *>(a.base);
  for (int i0 = 0; i0 < n; i0 += rows * kMoveUnroll) {
    T x[kMoveUnroll];
    int64_t to[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = i0 + u * rows + r;
      to[u] = -1;
      if (r < rows && i < n) {
        const int64_t from = row_offset(p, src, p.src_max_blocks, a, plane, keep[i]);
        to[u] = row_offset(p, dst, p.dst_max_blocks, a, plane, i);
        if (from < 0 || from == to[u]) to[u] = -1;
        if (to[u] >= 0) x[u] = *reinterpret_cast<const T *>(base + from + c);
      }
    }
    __syncthreads();  // the whole chunk is loaded: its places may be overwritten
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (to[u] >= 0) *reinterpret_cast<T *>(base + to[u] + c) = x[u];
  }
}

__device__ void move_scores(const CompactParams &p, int s, int n) {
  const int32_t *keep = p.keep + static_cast<int64_t>(s) * p.budget;
  const float *src = p.key_scores + s * p.score_stride;
  float *dst = p.dst_key_scores + s * p.dst_score_stride;
  for (int i0 = 0; i0 < n; i0 += kMoveThreads * kMoveUnroll) {
    float x[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = i0 + u * kMoveThreads + threadIdx.x;
      const int k = i < n ? keep[i] : -1;
      x[u] = 0.f;
      if (k >= 0 && k < p.score_stride) x[u] = src[k];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = i0 + u * kMoveThreads + threadIdx.x;
      if (i < n) dst[i] = x[u];
    }
  }
  __syncthreads();
  for (int64_t i = n + static_cast<int64_t>(threadIdx.x); i < p.dst_score_stride; i += kMoveThreads) dst[i] = 0.f;
}

// Grid (slices of all arrays, then one for the scores; sequences).
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const CompactParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.y;
  const int n = p.new_lens[s];
  if (n < 0 || n > p.budget || n > static_cast<int64_t>(p.dst_max_blocks) * p.block_size ||
      (p.key_scores != nullptr && n > p.dst_score_stride)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_evict_errors, kErrContext);
    return;
  }
  int slice = blockIdx.x;
#pragma unroll 1
  for (int k = 0; k < p.num_arrays; ++k) {
    const RowArray &a = p.arrays[k];
    const int per_plane = a.row_bytes > kSliceBytes ? a.row_bytes / kSliceBytes : 1;
    if (slice < a.planes * per_plane) {
      const int bytes = a.row_bytes / per_plane, plane = slice / per_plane, at = slice % per_plane * bytes;
      if (bytes % 16 == 0) move_slice<16>(p, a, plane, at, bytes, s, n);
      else if (bytes % 8 == 0) move_slice<8>(p, a, plane, at, bytes, s, n);
      else move_slice<4>(p, a, plane, at, bytes, s, n);
      return;
    }
    slice -= a.planes * per_plane;
  }
  move_scores(p, s, n);
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectArgs &a, cudaStream_t stream) {
  SelectParams p;
  p.key_scores = a.key_scores;
  p.score_stride = a.score_stride;
  p.context_lens = a.context_lens;
  p.keep = a.keep;
  p.new_lens = a.new_lens;
  p.max_context_len = a.max_context_len;
  p.budget = a.budget;
  p.recent = a.recent;
  return launch_pdl(evict_select_kernel, dim3(a.num_seqs), dim3(kSelThreads), 0, stream, p);
}

cudaError_t launch_evict_compact(const EvictCompactArgs &a, cudaStream_t stream) {
  CompactParams p;
  int64_t slices = a.key_scores != nullptr ? 1 : 0;
  p.num_arrays = a.num_arrays;
  for (int k = 0; k < a.num_arrays; ++k) {
    p.arrays[k] = a.arrays[k];
    slices += static_cast<int64_t>(a.arrays[k].planes) *
              (a.arrays[k].row_bytes > kSliceBytes ? a.arrays[k].row_bytes / kSliceBytes : 1);
  }
  p.src_tables = a.src_tables;
  p.dst_tables = a.dst_tables;
  p.keep = a.keep;
  p.new_lens = a.new_lens;
  p.key_scores = a.key_scores;
  p.dst_key_scores = a.dst_key_scores;
  p.score_stride = a.score_stride;
  p.dst_score_stride = a.dst_score_stride;
  p.src_max_blocks = a.src_max_blocks;
  p.dst_max_blocks = a.dst_max_blocks;
  p.budget = a.budget;
  p.block_size = a.block_size;
  p.num_blocks = a.num_blocks;
  return launch_pdl(evict_compact_kernel, dim3(static_cast<unsigned>(slices), a.num_seqs), dim3(kMoveThreads), 0,
                    stream, p);
}

cudaError_t evict_error_word(uint32_t **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_evict_errors);
}

}  // namespace pkv
