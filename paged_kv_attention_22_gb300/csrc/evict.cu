// Eviction from the paged cache by accumulated attention weight: which tokens
// of each sequence stay (evict_select) and moving their rows together
// (evict_compact).
//
// Selection. One CTA, or a cluster of eight for long sequences, finds the
// want-th largest score with a radix select over the scores' order-preserving
// 32-bit keys, eight bits a pass (the keys stay in shared memory while they fit),
// until the bin that holds it is taken whole. It then writes the kept positions
// in ascending order: each warp owns a contiguous range of positions, counts the
// keys above and at the threshold, and after one scan over the warps writes its
// own with ballots. Equal scores are taken from the lowest position on.
//
// Compaction, bound by HBM bandwidth: every kept row is read and written once.
// Row i of the destination is row keep[i] >= i of the source. A sequence whose
// destination blocks are all fresh has no hazard: warps move whole rows, in any
// order. With a block in both tables (in place), nothing is overwritten before
// it has been read as long as the rows go in order: a CTA then owns a slice (up
// to kSliceBytes) of every row and moves its rows in chunks, a whole chunk loaded
// before any of it is stored, the next one on its way meanwhile; slices are
// independent. Which of the two holds is found on the device, from the tables.
// 8 x 4,096 rows of 4 KiB: 48 us fresh (268 MB, 5.6 TB/s; it waits for memory with
// 24 warps an SM, the lookup of the next rows running ahead), 73 us in place
// (issue slots: every slice looks all the rows up). The same rows of a 4-bit cache (8
// heads, groups of 32: 84 MB, 12 us at the memory's rate): 33 us fresh (its lanes take
// the pieces of one array's row, 8 of 32 of them those of its parameters), 29 in place.
// One kernel for both ways at three CTAs an SM: 80 registers, 112 bytes of stack, 228
// bytes of spill stores and 212 of loads.
// Selection: 10.3 us for 8 x 16,384 scores (back to back in a graph; 12.8 as a single
// cold launch), mostly barriers between its passes.
#include "internal.h"
#include "ptx.cuh"

namespace pkv {

static __device__ uint32_t g_evict_errors;

namespace {

// ---------------------------------------------------------------- selection

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelLoads = 16;
constexpr int kBins = 256;
constexpr int kHistCopies = 8;  // histograms, each shared by four warps, against contention
constexpr size_t kSelMaxKeyBytes = 200 * 1024;  // beside the histograms
constexpr int kSelSmall = 256;                  // positions that are ranked by comparison instead
constexpr unsigned kSelCluster = 8;             // CTAs a long sequence
constexpr int32_t kSelAlone = 4096;             // longest sequences that one CTA takes

struct SelectParams {
  const float *key_scores;
  int64_t score_stride;
  const int32_t *context_lens;
  int32_t *keep, *new_lens;
  int32_t max_context_len, budget, recent;
  bool mark_invalid;
};

// Larger scores have larger keys; NaN sorts below every number; -0 equals 0.
__device__ __forceinline__ uint32_t score_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One cluster of CTAs a sequence (grid: sequences x cluster), each with a part of
// the competing positions: their histograms are summed through distributed
// shared memory, and every CTA finds the threshold for itself. kCached: the
// part's keys fit in dynamic shared memory.
template <bool kCached>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectParams p) {
  extern __shared__ uint32_t s_keys[];
  __shared__ uint32_t hist[kHistCopies][kBins];
  __shared__ uint32_t part[2][kBins];   // this CTA's histogram, of odd and even passes
  __shared__ uint32_t total[kBins];     // the cluster's
  __shared__ uint32_t s_prefix, s_left, s_whole, s_counts[2];
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  griddep_launch_dependents();
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int s = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the CTAs of a cluster leave before its first barrier together, or not at all
  const int ctx = p.context_lens[s];
  const int me = rank * kSelThreads + tid, all = C * kSelThreads;
  int32_t *keep = p.keep + static_cast<int64_t>(s) * p.budget;
  if (ctx < 0 || ctx > p.max_context_len) {
    if (me == 0) atomicOr(&g_evict_errors, kErrContext);
    if (p.mark_invalid) {
      if (me == 0) p.new_lens[s] = -1;
      for (int i = me; i < p.budget; i += all) keep[i] = -1;
    }
    return;
  }
  const float *score = p.key_scores + s * p.score_stride;
  const int new_len = min(ctx, p.budget), recent = min(ctx, p.recent);
  const int old = ctx - recent;         // positions that compete
  const int want = new_len - recent;    // how many of them stay
  if (me == 0) p.new_lens[s] = new_len;
  for (int i = new_len + me; i < p.budget; i += all) keep[i] = -1;
  for (int i = me; i < recent; i += all) keep[want + i] = old + i;
  if (want == old) {  // nothing to evict
    for (int i = me; i < old; i += all) keep[i] = i;
    return;
  }
  if (want == 0) return;
  if (kCached && C == 1 && old <= kSelSmall) {
    // a thread a position: its rank is the number of keys before its own (by key,
    // then by position), found by comparing with all of them
    if (tid < kSelSmall) s_keys[tid] = tid < old ? score_key(score[tid]) : 0u;
    __syncthreads();
    if (tid >= kSelSmall) return;
    const uint32_t k = s_keys[tid];
    int rank_of = 0;
#pragma unroll 8
    for (int i = 0; i < old; ++i) {
      const uint32_t other = s_keys[i];
      rank_of += other > k || (other == k && i < tid);
    }
    const bool in = tid < old && rank_of < want;
    const uint32_t kept = __ballot_sync(0xffffffffu, in);
    if (lane == 0) s_gt[warp] = __popc(kept);
    asm volatile("bar.sync 1, %0;" ::"n"(kSelSmall) : "memory");  // the threads still here
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? s_gt[lane] : 0);
    if (in) keep[before + __popc(kept & ((1u << lane) - 1u))] = tid;
    return;
  }
  // this CTA's positions
  const int per_cta = ((old + C - 1) / C + 31) / 32 * 32;
  const int cta0 = min(old, rank * per_cta), mine = min(old, cta0 + per_cta) - cta0;
  score += cta0;
  auto key_of = [&](int i) { return kCached ? s_keys[i] : score_key(score[i]); };

  // ---- the want-th largest key, most significant digit first
  uint32_t prefix = 0, left = want;  // keys above the prefix are in; left more come from below it
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < kHistCopies * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    uint32_t *h = hist[warp % kHistCopies];
    if (shift == 24) {
      // the one pass over global memory: kSelLoads loads a thread in flight
      for (int i0 = tid; i0 < mine; i0 += kSelThreads * kSelLoads) {
        float f[kSelLoads];
#pragma unroll
        for (int u = 0; u < kSelLoads; ++u) f[u] = i0 + u * kSelThreads < mine ? score[i0 + u * kSelThreads] : 0.f;
#pragma unroll
        for (int u = 0; u < kSelLoads; ++u) {
          const int i = i0 + u * kSelThreads;
          if (i >= mine) break;
          const uint32_t k = score_key(f[u]);
          if (kCached) s_keys[i] = k;
          atomicAdd(&h[k >> 24], 1u);
        }
      }
    } else {
#pragma unroll 8
      for (int i = tid; i < mine; i += kSelThreads) {
        const uint32_t k = key_of(i);
        if ((k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&h[(k >> shift) & 255u], 1u);
      }
    }
    __syncthreads();
    if (tid < kBins) {
      uint32_t n = 0;
#pragma unroll
      for (int c = 0; c < kHistCopies; ++c) n += hist[c][tid];
      if (C == 1) total[tid] = n;
      else part[(shift >> 3) & 1][tid] = n;
    }
    if (C > 1) {
      // a part is read until its CTA's next barrier but one writes it again
      cluster_sync();
      if (tid < kBins) {
        const uint32_t at = smem_u32(&part[(shift >> 3) & 1][tid]);
        uint32_t n = 0;
#pragma unroll 8
        for (int c = 0; c < C; ++c) n += ld_cluster_u32(at, c);
        total[tid] = n;
      }
    }
    __syncthreads();
    if (warp == 0) {
      // lane l sums bins 255 - 8 l .. 248 - 8 l, highest first
      uint32_t n[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[j] = total[255 - 8 * lane - j];
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
          s_left = left - above;
          s_whole = left == above + n[j];
        }
        above += n[j];
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
    if (s_whole) {
      // every key with this prefix stays: those above prefix - 1 (the prefix is
      // not 0, or all positions would stay, with want < old)
      prefix -= 1;
      left = 0;
      break;
    }
  }

  // ---- kept positions in order: keys above the threshold, and the first
  // `left` of those equal to it
  const int per_warp = ((mine + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int begin = min(mine, warp * per_warp), end = min(mine, begin + per_warp);
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = begin + lane; i - lane < end; i += 32) {
    const uint32_t k = i < end ? key_of(i) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i < end && k > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, i < end && k == prefix));
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  // in the warps before this one, and in the CTAs before this one
  int gt0 = __reduce_add_sync(0xffffffffu, lane < warp ? s_gt[lane] : 0);
  int eq0 = __reduce_add_sync(0xffffffffu, lane < warp ? s_eq[lane] : 0);
  if (C > 1) {
    if (warp == 0) {
      const int a = __reduce_add_sync(0xffffffffu, s_gt[lane]), b = __reduce_add_sync(0xffffffffu, s_eq[lane]);
      if (lane == 0) {
        s_counts[0] = a;
        s_counts[1] = b;
      }
    }
    cluster_sync();
    gt0 += __reduce_add_sync(0xffffffffu, lane < rank ? ld_cluster_u32(smem_u32(&s_counts[0]), lane) : 0u);
    eq0 += __reduce_add_sync(0xffffffffu, lane < rank ? ld_cluster_u32(smem_u32(&s_counts[1]), lane) : 0u);
  }
  const uint32_t below = (1u << lane) - 1u;
  const int quota = static_cast<int>(left);
#pragma unroll 2
  for (int i = begin + lane; i - lane < end; i += 32) {
    const uint32_t k = i < end ? key_of(i) : 0u;
    const uint32_t bg = __ballot_sync(0xffffffffu, i < end && k > prefix);
    const uint32_t be = __ballot_sync(0xffffffffu, i < end && k == prefix);
    const int my_gt = gt0 + __popc(bg & below), my_eq = eq0 + __popc(be & below);
    const bool in = ((bg >> lane) & 1u) || (((be >> lane) & 1u) && my_eq < quota);
    if (in) keep[my_gt + min(my_eq, quota)] = cta0 + i;
    gt0 += __popc(bg);
    eq0 += __popc(be);
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another reads its counts
}

// ---------------------------------------------------------------- compaction

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;       // scores a thread has in flight
constexpr int kRingStages = 2, kRingUnroll = 4;  // chunks in the ring; pieces of a chunk a thread
constexpr size_t kRingBytes = static_cast<size_t>(kRingStages) * kRingUnroll * kMoveThreads * 16;
static_assert(kRingStages * kRingUnroll <= 32, "bits of `moved`");
static_assert(kRingBytes <= 48 * 1024, "no attribute needed");
constexpr int kRowsPerWarp = 4;      // rows a warp moves together, without hazards

struct CompactParams {
  RowArray arrays[kMaxRowArrays];
  int32_t num_arrays;
  const int32_t *src_tables, *dst_tables, *keep, *new_lens;
  const float *key_scores;           // [S, score_stride] or null
  float *dst_key_scores;             // [S, dst_score_stride]
  int64_t score_stride, dst_score_stride;
  int32_t src_max_blocks, dst_max_blocks, budget, num_blocks;
  int32_t slice_bytes;               // in place: bytes of a row a CTA moves at a time, at most
  FastDiv block;
};

template <int N> struct Piece;
template <> struct Piece<16> { using T = uint4; };
template <> struct Piece<8> { using T = uint2; };
template <> struct Piece<4> { using T = uint32_t; };

// Byte offset of position pos's row of plane 0 in an array, or -1 (with its bit
// raised) for a position or block that does not exist. Plane k's row lies k
// times block_size * row_bytes further.
__device__ __forceinline__ int64_t row_at(const CompactParams &p, const RowArray &a, const int32_t *table, int max_blocks,
                                          int pos) {
  const int j = pos < 0 ? max_blocks : static_cast<int>(fast_quotient(pos, p.block));
  if (j >= max_blocks) {
    atomicOr(&g_evict_errors, kErrContext);
    return -1;
  }
  const int blk = table[j];
  if (blk < 0 || blk >= p.num_blocks) {
    atomicOr(&g_evict_errors, kErrBlock);
    return -1;
  }
  return blk * a.block_bytes + static_cast<int64_t>(pos - j * static_cast<int>(p.block.d)) * a.row_bytes;
}

// Move `bytes` bytes at `at` of every kept row of one plane, N bytes a piece. The
// rows go in chunks through a ring in shared memory, kRingStages - 1 chunks ahead
// of the stores; a piece is loaded and stored by the same thread. (Three or four
// stages take as long as two.) A row of chunk c
// comes from position keep[i] >= i, behind all that earlier chunks overwrite: its
// load may run ahead of their stores. What chunk c overwrites was loaded by chunks
// up to c, which the barrier makes sure of.
template <int N>
__device__ void move_slice(const CompactParams &p, const RowArray &a, int plane, int at, int bytes, int s, int n,
                           uint4 *ring) {
  using T = typename Piece<N>::T;
  const int per_row = bytes / N;
  const int rows = kMoveThreads / per_row;  // rows a step
  const int chunk = rows * kRingUnroll;
  const int r = threadIdx.x / per_row;
  const int32_t *keep = p.keep + static_cast<int64_t>(s) * p.budget;
  const int32_t *src = p.src_tables + static_cast<int64_t>(s) * p.src_max_blocks;
  const int32_t *dst = p.dst_tables + static_cast<int64_t>(s) * p.dst_max_blocks;
  uint8_t *base = static_cast<uint8_t *>(a.base) + static_cast<int64_t>(plane) * p.block.d * a.row_bytes + at +
                  threadIdx.x % per_row * N;
  const int end = r < rows ? n : 0;
  uint32_t moved = 0;  // which pieces are on their way, kRingUnroll bits a chunk, the newest lowest
  int next[kRingUnroll];
  auto look_up = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kRingUnroll; ++u) {
      const int i = i0 + u * rows + r;
      next[u] = i < end ? keep[i] : 0;
    }
  };
  auto load = [&](int i0, int stage) {
#pragma unroll
    for (int u = 0; u < kRingUnroll; ++u) {
      const int i = i0 + u * rows + r;
      moved <<= 1;
      if (i < end) {
        const int64_t from = row_at(p, a, src, p.src_max_blocks, next[u]);
        bool stays = false;  // at its place already, in a block that others may share
        if (next[u] == i) {
          const uint32_t j = fast_quotient(i, p.block);
          stays = from >= 0 && src[j] == dst[j];
        }
        if (from >= 0 && !stays) {
          moved |= 1;
          cp_async<N>(smem_u32(ring + (stage * kRingUnroll + u) * kMoveThreads + threadIdx.x), base + from);
        }
      }
    }
    cp_async_commit();
    look_up(i0 + chunk);
  };
  look_up(0);
#pragma unroll
  for (int c = 0; c < kRingStages - 1; ++c) load(c * chunk, c);
  int stage = 0;
  for (int i0 = 0; i0 < n; i0 += chunk) {
    cp_async_wait<kRingStages - 2>();
    __syncthreads();  // the whole chunk is loaded: its places may be overwritten
    const uint32_t now = moved >> (kRingUnroll * (kRingStages - 2));
    load(i0 + (kRingStages - 1) * chunk, stage == 0 ? kRingStages - 1 : stage - 1);
#pragma unroll
    for (int u = 0; u < kRingUnroll; ++u) {
      if (now >> (kRingUnroll - 1 - u) & 1) {
        const int64_t into = row_at(p, a, dst, p.dst_max_blocks, i0 + u * rows + r);
        if (into >= 0) *reinterpret_cast<T *>(base + into) =
            *reinterpret_cast<const T *>(ring + (stage * kRingUnroll + u) * kMoveThreads + threadIdx.x);
      }
    }
    stage = stage == kRingStages - 1 ? 0 : stage + 1;
  }
}

// The pieces of N bytes of kRowsPerWarp rows of one array, all planes of a row
// together, kPieces a lane in flight. from / to hold the rows' offsets (to -1: not
// moved).
constexpr int kPieces = 2;
template <int N>
__device__ __forceinline__ void move_rows(const CompactParams &p, const RowArray &a, const int64_t (&from)[kRowsPerWarp],
                                          const int64_t (&to)[kRowsPerWarp], int lane) {
  using T = typename Piece<N>::T;
  const int per_plane = a.row_bytes / N, pieces = a.planes * per_plane;
  const int64_t plane_bytes = static_cast<int64_t>(p.block.d) * a.row_bytes;
  uint8_t *base = static_cast<uint8_t *>(a.base);
#pragma unroll 1
  for (int i0 = lane; i0 < pieces; i0 += 32 * kPieces) {
    T x[kPieces][kRowsPerWarp];
    int64_t at[kPieces];
#pragma unroll
    for (int v = 0; v < kPieces; ++v) {
      const int i = i0 + 32 * v;
      const int plane = a.planes == 1 ? 0 : i / per_plane;
      at[v] = plane * plane_bytes + (i - plane * per_plane) * N;
#pragma unroll
      for (int u = 0; u < kRowsPerWarp; ++u)
        if (i < pieces && to[u] >= 0) x[v][u] = __ldcs(reinterpret_cast<const T *>(base + from[u] + at[v]));
    }
#pragma unroll
    for (int v = 0; v < kPieces; ++v)
#pragma unroll
      for (int u = 0; u < kRowsPerWarp; ++u)
        if (i0 + 32 * v < pieces && to[u] >= 0) *reinterpret_cast<T *>(base + to[u] + at[v]) = x[v][u];
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

// Grid (CTAs a sequence, the last one for the scores if there are any; sequences).
__global__ void __launch_bounds__(kMoveThreads, 3) evict_compact_kernel(const CompactParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.y;
  const int n = p.new_lens[s];
  if (n < 0 || n > p.budget || n > static_cast<int64_t>(p.dst_max_blocks) * p.block.d ||
      (p.key_scores != nullptr && n > p.dst_score_stride)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_evict_errors, kErrContext);
    return;
  }
  const int movers = static_cast<int>(gridDim.x) - (p.key_scores != nullptr ? 1 : 0);
  if (static_cast<int>(blockIdx.x) >= movers) {
    move_scores(p, s, n);
    return;
  }
  const int32_t *src = p.src_tables + static_cast<int64_t>(s) * p.src_max_blocks;
  const int32_t *dst = p.dst_tables + static_cast<int64_t>(s) * p.dst_max_blocks;
  bool in_place = false;
  const int shared_blocks = min(p.src_max_blocks, static_cast<int>((n + p.block.d - 1) / p.block.d));
  for (int j = threadIdx.x; j < shared_blocks; j += kMoveThreads) in_place |= src[j] == dst[j];
  if (!__syncthreads_or(in_place)) {
    const int32_t *keep = p.keep + static_cast<int64_t>(s) * p.budget;
    const int lane = threadIdx.x & 31;
    // an item is kRowsPerWarp rows of one array; the next item's slots (kept
    // position, then table entry: two loads in a row) are looked up while this
    // one's rows move
    const int items = (n + kRowsPerWarp - 1) / kRowsPerWarp * p.num_arrays;
    const int step = movers * (kMoveThreads / 32);
    int item = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);
    int64_t f, t;  // of row `lane` of the item, lane < kRowsPerWarp
    auto look_up = [&](int it) {
      f = t = -1;
      const int quad = it / p.num_arrays, i = quad * kRowsPerWarp + lane;
      if (it < items && lane < kRowsPerWarp && i < n) {
        const RowArray &a = p.arrays[it - quad * p.num_arrays];
        f = row_at(p, a, src, p.src_max_blocks, keep[i]);
        t = row_at(p, a, dst, p.dst_max_blocks, i);
        if (f < 0) t = -1;
      }
    };
    look_up(item);
    for (; item < items; item += step) {
      int64_t from[kRowsPerWarp], to[kRowsPerWarp];
#pragma unroll
      for (int u = 0; u < kRowsPerWarp; ++u) {
        from[u] = __shfl_sync(0xffffffffu, f, u);
        to[u] = __shfl_sync(0xffffffffu, t, u);
      }
      look_up(item + step);
      const RowArray &a = p.arrays[item % p.num_arrays];
      if (a.row_bytes % 16 == 0) move_rows<16>(p, a, from, to, lane);
      else if (a.row_bytes % 8 == 0) move_rows<8>(p, a, from, to, lane);
      else move_rows<4>(p, a, from, to, lane);
    }
    return;
  }
  // in place: slices of all arrays in turn
  extern __shared__ uint4 ring[];
  int first = blockIdx.x;
#pragma unroll 1
  for (int k = 0; k < p.num_arrays; ++k) {
    const RowArray &a = p.arrays[k];
    const int per_plane = a.row_bytes > p.slice_bytes ? a.row_bytes / p.slice_bytes : 1, slices = a.planes * per_plane;
    const int bytes = a.row_bytes / per_plane;
    for (; first < slices; first += movers) {
      const int plane = first / per_plane, at = (first - plane * per_plane) * bytes;
      if (bytes % 16 == 0) move_slice<16>(p, a, plane, at, bytes, s, n, ring);
      else if (bytes % 8 == 0) move_slice<8>(p, a, plane, at, bytes, s, n, ring);
      else move_slice<4>(p, a, plane, at, bytes, s, n, ring);
    }
    first -= slices;
  }
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
  p.mark_invalid = a.mark_invalid;
  // one CTA for a short sequence (its passes take less than the cluster's
  // barriers), a cluster for longer ones
  const unsigned C = a.max_context_len <= kSelAlone ? 1 : kSelCluster;
  const size_t per_cta = ((static_cast<size_t>(a.max_context_len) + C - 1) / C + 31) / 32 * 32;
  const bool cached = per_cta * sizeof(uint32_t) <= kSelMaxKeyBytes;
  const auto kernel = cached ? evict_select_kernel<true> : evict_select_kernel<false>;
  const size_t smem = cached ? (per_cta > kSelSmall ? per_cta : kSelSmall) * sizeof(uint32_t) : 0;
  if (smem > 32 * 1024) {  // beside the static arrays
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSelMaxKeyBytes));
    if (e != cudaSuccess) return e;
  }
  if (C == 1) return launch_pdl(kernel, dim3(a.num_seqs), dim3(kSelThreads), smem, stream, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs) * C);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_evict_compact(const EvictCompactArgs &a, cudaStream_t stream) {
  CompactParams p;
  p.num_arrays = a.num_arrays;
  int64_t row_bytes = 0;
  for (int k = 0; k < a.num_arrays; ++k) {
    p.arrays[k] = a.arrays[k];
    p.arrays[k].block_bytes = static_cast<int64_t>(a.arrays[k].planes) * a.block_size * a.arrays[k].row_bytes;
    row_bytes += static_cast<int64_t>(a.arrays[k].planes) * a.arrays[k].row_bytes;
  }
  // in place the slices of a sequence are all that spreads it over the SMs: half
  // as wide where there are too few for four CTAs an SM (in place, one sequence of
  // 8,192 kept rows of 4 KiB takes 37 us with 32 bytes and 52 with 64; 64 of 512
  // rows 80 and 67)
  p.slice_bytes = a.num_seqs * (row_bytes / kSliceBytes) < 4 * static_cast<int64_t>(a.num_sms) ? kSliceBytes / 2 : kSliceBytes;
  int64_t slices = 0;
  for (int k = 0; k < a.num_arrays; ++k)
    slices += static_cast<int64_t>(a.arrays[k].planes) *
              (a.arrays[k].row_bytes > p.slice_bytes ? a.arrays[k].row_bytes / p.slice_bytes : 1);
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
  p.num_blocks = a.num_blocks;
  p.block = fast_div(a.block_size);
  // CTAs a sequence: no more than its slices (in place) or its rows call for,
  // and some 8 an SM in all, so that many sequences do not queue idle CTAs
  const int64_t items = (static_cast<int64_t>(a.budget) + kRowsPerWarp - 1) / kRowsPerWarp * a.num_arrays;
  const int64_t rows = (items + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
  int64_t movers = slices > rows ? slices : rows;
  const int64_t cap = (8 * static_cast<int64_t>(a.num_sms) + a.num_seqs - 1) / a.num_seqs;
  if (movers > cap) movers = cap;
  return launch_pdl(evict_compact_kernel, dim3(static_cast<unsigned>(movers + (a.key_scores != nullptr ? 1 : 0)), a.num_seqs),
                    dim3(kMoveThreads), kRingBytes, stream, p);
}

cudaError_t evict_error_word(uint32_t **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_evict_errors);
}

}  // namespace pkv
