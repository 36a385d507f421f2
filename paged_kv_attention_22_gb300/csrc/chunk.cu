// Attention of chunks of new tokens over the paged cache, on the 5th-generation
// tensor cores (tcgen05, accumulators in TMEM, operands staged by TMA): segments of
// one token, of a few (drafted tokens, the tail of a prompt) or of thousands in one
// call, with a sliding window and sinks.
//
// Work list. A tile is 128 query rows of one KV head: 128 / G tokens times the head's
// G query heads, which are neighbours in the row of a token, so that one TMA box
// loads them in the order (token, head). Its steps are the 128-key tiles that its rows
// see: those that hold sinks, then those from its window's start to its last token's
// position. Tiles are listed in (sequence, KV head, tile) order.
//
// Shares, one CTA per SM. Where several tiles have the same keys and there are tiles
// enough, CTA c takes whole tiles c, c + W, ... of the list's front: CTAs that run side
// by side then pass the same keys at the same time, which reach the SMs through L2 once
// from memory. The steps of the tiles behind, or of all, are cut into one contiguous
// range a CTA, of the length that evens out the CTAs' totals: a few tokens over long
// contexts use every SM, and no CTA is left with the last tile. (All steps in ranges:
// eight chunks of 512 tokens over 7,680 keys 330 us for 250.) A tile cut between ranges leaves its pieces (maximum, sums, unnormalised output) in the workspace, a
// range's first in slot 2k, its last in slot 2k + 1; a second kernel, launched right
// behind, joins them.
//
// 12 warps:
//   warp 0      TMA producer: walks the CTA's share, publishes its pieces to the other
//               warps, and copies Q (two buffers), K and V (two stages each).
//   warp 1      MMAs. S(j + 1) = Q K^T goes out before O += P(j) V(j), into the other of
//               two S buffers in TMEM, so that the tensor pipe computes the next logits
//               while the softmax warps work on these. MMAs complete in order: S(j)
//               complete means that P.V of step j - 2 is. V rows that no row of the tile
//               sees (past the last key; between the sinks and the window) may be absent
//               or hold anything; the warp zeroes them before P.V, for a probability of
//               zero must not meet a NaN. Their logits are masked by selection.
//   warps 4-11  softmax, one row and half of the columns per thread (TMEM lane = row;
//               warps 4-7 the lower half, 8-11 the upper): read S, mask, online softmax in
//               base 2 with a lazy maximum, for which the two threads of a row swap their
//               halves' maxima through shared memory, P as bf16 over S's columns; half of
//               the output's columns each, written once the next piece's first logits have been
//               read, so that its last P.V runs meanwhile.
//
// A few tokens over long contexts are bound by HBM bandwidth: 64 x 5 tokens over 640 keys take
// 37.1 us (floor 25.5), two of 16 over 32,768 keys 52.6 (40.2), of which some 6 us pass before
// the first logits and 4 behind the last. Long chunks are not bound by the tensor pipe (a third
// of its time): a step takes 2,000 cycles, in which an SM takes 64 KB of keys and values, 9 TB/s in
// all. On the eight chunks above, 16 softmax warps with a quarter of the columns each measured
// 267 us, whole rows with the two groups on alternate steps 286, both threads of a row
// reading all of its columns in place of the exchange 263. Two tiles a CTA halve the
// keys' way, but a tile's next logits then wait for its P.V (TMEM holds one S a tile): 247,
// and 8 to 12 us more on the small cases.
//
// P is rounded to bf16 and the output divided by the sum of the rounded
// probabilities, the weights that the products used; the lse comes from the fp32 sum.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {

static __device__ uint32_t g_chunk_errors;

namespace {

constexpr int kD = 128;
constexpr int kRows = 128;                  // query rows a tile
constexpr int kKeys = 128;                  // keys a step
constexpr int kHalfBytes = 128 * 128;       // 128 rows x 64 bf16 (one swizzle column group)
constexpr int kTileBytes = 2 * kHalfBytes;  // 128 rows x 128 bf16
constexpr int kThreads = 384;
constexpr int kMmaWarp = 1, kSoftmaxWarp0 = 4;
constexpr int kDescs = 4;                   // pieces published ahead
constexpr int kDescInts = 16;
constexpr int kMaxWaves = 128;              // whole tiles a CTA, at most

// barriers (8 bytes each): K and V landed, S complete (which frees its K), P written, P.V
// complete (which frees its V), by the parity of the step; Q landed and free, by that of the
// piece; descriptors full and free; of each TMEM quadrant the exchange between its two
// softmax warps; the end
constexpr int kBarK = 0, kBarV = 2, kBarS = 4, kBarP = 6, kBarO = 8, kBarQ = 10, kBarQFree = 12, kBarDesc = 14,
              kBarDescFree = kBarDesc + kDescs, kBarX = kBarDescFree + kDescs, kBarDone = kBarX + 4,
              kNumBars = kBarDone + 1;
constexpr int kDescReaders = 1 + 8;  // the MMA warp, the softmax warps

// A sequence's segment; Lq = 0: nothing to do.
struct Seq {
  int q0, Lq, ctx;
};
// A whole tile of a CTA's share.
struct Wave {
  Seq q;
  int s, head, tile;
};

// shared memory
constexpr int kQOff = 0;                       // two Q tiles
constexpr int kKOff = kQOff + 2 * kTileBytes;  // two K tiles
constexpr int kVOff = kKOff + 2 * kTileBytes;  // two V tiles
constexpr int kEpiWarpBytes = 32 * 64;
constexpr int kEpiOff = kVOff + 2 * kTileBytes;  // staging areas of the softmax warps
constexpr int kBarOff = kEpiOff + 8 * kEpiWarpBytes;
constexpr int kDescOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;
constexpr int kMiscOff = kDescOff + kDescs * kDescInts * 4;  // TMEM address, abort flag, unseen rows of the V tiles
constexpr int kAllOff = kMiscOff + 16;                       // int64: all steps, all tiles
constexpr int kSwapOff = kAllOff + 16;                       // float [6][2][128] by half: maxima of two steps, two sums of two pieces
constexpr int kWaveOff = kSwapOff + 6 * 2 * kRows * 4;       // Wave [kMaxWaves]
constexpr int kSmemBytes = kWaveOff + kMaxWaves * static_cast<int>(sizeof(Wave)) + 1024;  // + slack for alignment
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
// until the first copies, in the place of the V tiles: the list of sequences. The producer's copy
// of V(0) waits for no other warp, so behind build()'s last barrier only the producer reads here.
constexpr int kStepsOff = kVOff;                                          // int64 [S + 1]: steps before
constexpr int kTilesOff = kStepsOff + 8 * (kChunkMaxSeqs + 2);            // int64 [S + 1]: tiles before
constexpr int kSeqOff = kTilesOff + 8 * (kChunkMaxSeqs + 2);              // Seq [S]
constexpr int kShareOff = kSeqOff + static_cast<int>(sizeof(Seq)) * kChunkMaxSeqs;  // int64 [W + 1]: ranges' starts
constexpr int kRankOff = kShareOff + 8 * (kChunkMaxCtas + 2);             // int [W + 1]: ranges before
constexpr int kTotalOff = kRankOff + 4 * (kChunkMaxCtas + 2);             // int64 [warps]
constexpr int kSumOff = kTotalOff + 8 * (kThreads / 32);                  // int [W]
static_assert(kSumOff + 4 * kChunkMaxCtas <= kEpiOff && kTotalOff % 8 == 0, "the list fits the V tiles");
static_assert(kChunkMaxCtas <= kThreads, "a thread for each CTA's share");

constexpr uint32_t kTmemCols = 512;  // S (two), O: 128 columns each; a power of two
constexpr int kTmemO = 256;
constexpr uint32_t kIdescQK = idesc_bf16_f32(kRows, kKeys, 0, 0);  // A = Q K-major, B = K K-major
constexpr uint32_t kIdescPV = idesc_bf16_f32(kRows, kD, 0, 1);     // A = P (TMEM), B = V MN-major
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLazyMax = 8.0f;      // log2 units that the running maximum may lag
constexpr float kFloor = -1e30f;      // finite, below every logit: a row that has seen no key yet

struct ChunkParams {
  const int32_t *cu_q, *lens, *block_tables;
  __nv_bfloat16 *out;
  float *lse;
  float *ws_o;         // [2 ranges, 128, 128]
  float4 *ws_ml;       // [2 ranges, 128]: maximum, sum, sum of the rounded
  ChunkCut *cuts;      // [ranges]: the tile that the start of range k is the first to cut
  FastDiv block;
  int32_t max_blocks, num_seqs, total_q, max_seqlen_q, max_context_len;
  int32_t num_q_heads, num_kv_heads, num_blocks;
  int32_t gqa_log2;    // log2 of the query heads of a KV head
  int32_t lanes_log2;  // lanes that add up one sequence's steps
  int32_t shared_keys; // some segment has several tiles over the same keys
  int32_t window, sinks, box_rows;
  float scale_log2;
};

__device__ __forceinline__ bool wait_(uint32_t bar, uint32_t parity, const volatile int *abort) {
  return mbar_wait(bar, parity, &g_chunk_errors, abort);
}

// Segment s, without rows if it is invalid, which sets `bad`.
__device__ __forceinline__ Seq load_seq(const ChunkParams &p, int s, bool &bad) {
  const int q0 = p.cu_q[s], q1 = p.cu_q[s + 1], ctx = p.lens[s];
  Seq r = {q0, q1 - q0, ctx};
  if (q0 == q1) return r;
  if (q0 < 0 || q1 < q0 || q1 > p.total_q || r.Lq > p.max_seqlen_q || ctx < r.Lq || ctx > p.max_context_len ||
      ctx > static_cast<int64_t>(p.max_blocks) * p.block.d) {
    bad = true;
    r.Lq = 0;
  }
  return r;
}

__device__ __forceinline__ int tile_tokens(const ChunkParams &p) { return kRows >> p.gqa_log2; }

// The key tiles of row tile i: `lead` of them from the first key, then j_start .. n_end - 1;
// lo is the first key of its window.
struct Tile {
  int t0, n_tok;  // its first token within the segment, and its tokens
  int lead, j_start, n_end, lo;
  __device__ __forceinline__ int steps() const { return lead + n_end - j_start; }
};
template <bool kWindowed>
__device__ __forceinline__ Tile tile_of(const ChunkParams &p, const Seq &q, int i) {
  const int diag = q.ctx - q.Lq;
  Tile t;
  t.t0 = i * tile_tokens(p);
  t.n_tok = min(q.Lq - t.t0, tile_tokens(p));
  t.n_end = (diag + t.t0 + t.n_tok + kKeys - 1) / kKeys;
  t.lo = t.j_start = t.lead = 0;
  if constexpr (kWindowed) {
    t.lo = max(0, diag + t.t0 + 1 - p.window);
    t.j_start = t.lo / kKeys;
    t.lead = min((p.sinks + kKeys - 1) / kKeys, t.j_start);
  }
  return t;
}
__device__ __forceinline__ int tiles_of(const ChunkParams &p, const Seq &q) {
  return (q.Lq + tile_tokens(p) - 1) / tile_tokens(p);
}

// a / b for 0 <= a, 0 < b, with 32-bit division where it does.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// The last s in [0, n) with before[s] <= x.
__device__ __forceinline__ int find(const int64_t *before, int n, int64_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Inclusive prefix sums of a[1 .. n] in place, a[0] = 0, and the last of them; one warp.
__device__ __forceinline__ int64_t scan(int64_t *a, int n, int lane) {
  int64_t carry = 0;
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane;
    int64_t x = i < n ? a[i + 1] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (i < n) a[i + 1] = carry + x;
    carry += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) a[0] = 0;
  return carry;
}

// What the whole call comes to, as every thread knows it. Without whole tiles (front == 0)
// range c starts at step c * even; else the starts and ranks are in shared memory.
struct Shares {
  int64_t U, even;  // steps in all, and the even share of a CTA
  int W;            // CTAs with work
  int waves;        // whole tiles of each
  int front;
};

// Builds the list and the shares; the whole CTA. Afterwards this CTA's whole tiles are in
// shared memory. No work if some thread says `skip`.
template <bool kWindowed>
__device__ __forceinline__ Shares build(const ChunkParams &p, uint8_t *smem, bool skip) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  int64_t *steps = reinterpret_cast<int64_t *>(smem + kStepsOff);
  int64_t *tiles = reinterpret_cast<int64_t *>(smem + kTilesOff);
  Seq *seqs = reinterpret_cast<Seq *>(smem + kSeqOff);
  int64_t *starts = reinterpret_cast<int64_t *>(smem + kShareOff);
  int *ranks = reinterpret_cast<int *>(smem + kRankOff);
  Wave *list = reinterpret_cast<Wave *>(smem + kWaveOff);
  int *sums = reinterpret_cast<int *>(smem + kSumOff);
  int64_t *totals = reinterpret_cast<int64_t *>(smem + kTotalOff);
  volatile int64_t *all_of = reinterpret_cast<volatile int64_t *>(smem + kAllOff);
  const int lanes = 1 << p.lanes_log2, sub = tid & (lanes - 1);
  bool bad = false;
  for (int base = 0; base < p.num_seqs; base += kThreads >> p.lanes_log2) {
    const int s = base + (tid >> p.lanes_log2);
    int64_t n = 0;
    if (s < p.num_seqs) {
      const Seq q = load_seq(p, s, bad);
      const int n_tiles = tiles_of(p, q);
      for (int i = sub; i < n_tiles; i += lanes) n += tile_of<kWindowed>(p, q, i).steps();
      if (sub == 0) {
        seqs[s] = q;
        tiles[s + 1] = static_cast<int64_t>(n_tiles) * p.num_kv_heads;
      }
    }
    for (int off = lanes >> 1; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
    if (s < p.num_seqs && sub == 0) steps[s + 1] = n * p.num_kv_heads;
  }
  if (__syncthreads_or(skip)) return Shares{};
  if (bad && cta == 0 && sub == 0) atomicOr(&g_chunk_errors, kErrSeqlens);
  if (warp == 0 || (warp == 1 && p.shared_keys)) {
    const int64_t all = scan(warp == 0 ? steps : tiles, p.num_seqs, lane);
    if (lane == 0) all_of[warp] = all;
  }
  __syncthreads();
  // The ways out that pass no other barrier read no more of the list than this: a late warp may
  // be here when V(0) lands there.
  const int64_t U = all_of[0];
  Shares r;
  r.U = U;
  r.W = static_cast<int>(min(static_cast<int64_t>(gridDim.x), U));
  r.waves = r.front = 0;
  r.even = r.W == 0 ? 0 : quotient(U + r.W - 1, r.W);
  if (r.W == 0 || !p.shared_keys) return r;
  // Tile i of the list (the rows of q are fewer than 2^31, so are the tiles), found from
  // a sequence at or before it.
  const int n_tiles = static_cast<int>(all_of[1]);
  auto locate = [&](int i, int from) {
    Wave w;
    w.s = from;
    while (tiles[w.s + 1] <= i) ++w.s;  // the last has tiles[] = n_tiles
    w.q = seqs[w.s];
    const uint32_t at = i - static_cast<int>(tiles[w.s]), n = tiles_of(p, w.q);
    w.head = at / n;
    w.tile = at - w.head * n;
    return w;
  };
  // Whole tiles as far as no CTA gets more than its even share, and one more each is left
  // to even out with. (Fewer than 2^31 steps: at most kMaxWaves tiles of 2^23.)
  int mine = 0;  // thread c: steps of CTA c's whole tiles
  for (r.waves = min(n_tiles / r.W - 1, kMaxWaves); r.waves > 0; r.waves >>= 1) {
    if (tid < r.W) sums[tid] = 0;
    __syncthreads();
    int at = 0;
    for (int i = tid; i < r.waves * r.W; i += kThreads) {
      if (i == tid) at = find(tiles, p.num_seqs, tid);
      const Wave x = locate(i, at);
      at = x.s;
      atomicAdd(&sums[i % r.W], tile_of<kWindowed>(p, x.q, x.tile).steps());
    }
    __syncthreads();
    mine = tid < r.W ? sums[tid] : 0;
    if (!__syncthreads_or(mine > r.even)) break;
  }
  if (r.waves <= 0) {
    r.waves = 0;
    return r;
  }
  if (tid < r.waves) list[tid] = locate(cta + tid * r.W, find(tiles, p.num_seqs, cta + tid * r.W));
  // the whole tiles are in front of the ranges, of which thread c's is what CTA c may still take
  const int64_t rest = tid < r.W ? r.even - mine : 0;
  int64_t before = rest;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, before, off);
    if (lane >= off) before += y;
  }
  if (lane == 31) totals[warp] = before;
  __syncthreads();
  int64_t all = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += totals[w];
    all += totals[w];
  }
  const int64_t front = r.even * r.W - all;
  const int64_t start = min(front + before - rest, U), end = min(front + before, U);
  const uint32_t some = __ballot_sync(0xffffffffu, tid < r.W && end > start);
  if (lane == 0) sums[warp] = __popc(some);
  if (tid < r.W) starts[tid] = start;
  if (tid == r.W - 1) starts[r.W] = U;
  __syncthreads();
  int rank = __popc(some & ((1u << lane) - 1));
  for (int w = 0; w < warp; ++w) rank += sums[w];
  if (tid < r.W) ranks[tid] = rank;
  if (tid == r.W - 1) ranks[r.W] = rank + (end > start ? 1 : 0);
  __syncthreads();
  r.front = 1;
  return r;
}

// A piece as the producer publishes it: `steps` steps from `first` of a tile's.
struct Piece {
  int steps;       // 0: no more pieces
  int first, lead, j_start;
  int pos;         // position of the tile's first token
  int row, n_tok;  // its first token among all, and its tokens
  int head;        // KV head
  int slot;        // where its partial result goes, or -1: it is the whole tile
  __device__ __forceinline__ int key_tile(int j) const {  // of the piece's step j
    const int k = first + j;
    return k < lead ? k : k - lead + j_start;
  }
};
constexpr int kPieceInts = sizeof(Piece) / 4;
static_assert(kPieceInts <= kDescInts, "a piece fits its slot");

// Descriptor n, the first kInts ints of it, once its barrier's phase is complete.
template <int kInts>
__device__ __forceinline__ void read_piece(int n, const uint8_t *smem, uint32_t bars, int lane, Piece &d) {
  const int i = n % kDescs;
  const volatile int *src = reinterpret_cast<const volatile int *>(smem + kDescOff) + i * kDescInts;
  int *dst = reinterpret_cast<int *>(&d);
#pragma unroll
  for (int k = 0; k < kInts; ++k) dst[k] = src[k];
  __syncwarp();
  if (lane == 0) mbar_arrive(bars + 8 * (kBarDescFree + i));
}

// 16 words a lane through the warp's staging area to rows of 64 bytes each, 16-byte
// chunk c of row i at c ^ ((i >> 1) & 3), which keeps both sides free of bank
// conflicts; `to` gives a row's address.
template <typename To>
__device__ __forceinline__ void store_rows(const uint32_t *w, uint32_t scr, int n_valid, int lane, To to) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(scr + lane * 64 + ((k ^ ((lane >> 1) & 3)) * 16)),
                 "r"(w[4 * k]), "r"(w[4 * k + 1]), "r"(w[4 * k + 2]), "r"(w[4 * k + 3])
                 : "memory");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 8 * i + (lane >> 2), c = lane & 3;
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(scr + row * 64 + ((c ^ ((row >> 1) & 3)) * 16))
                 : "memory");
    if (row < n_valid) *reinterpret_cast<uint4 *>(to(row) + c * 16) = v;
  }
  __syncwarp();
}

template <bool kWindowed>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const ChunkParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem), bars = sbase + kBarOff;
  auto bar = [&](int i) { return bars + 8u * i; };
  volatile int *abort = reinterpret_cast<volatile int *>(smem + kMiscOff + 4);
  volatile uint32_t *unseen = reinterpret_cast<volatile uint32_t *>(smem + kMiscOff + 8);  // [2]
  auto fail = [&]() {
    *abort = 1;
    atomicOr(&g_chunk_errors, kErrTimeout);
  };
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      int count = 1;
      if (i >= kBarP && i < kBarP + 2) count = 8;
      if (i >= kBarDescFree && i < kBarDescFree + kDescs) count = kDescReaders;
      if (i >= kBarX && i < kBarX + 4) count = 2;
      mbar_init(bar(i), count);
    }
    *abort = 0;
    fence_barrier_init();
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sbase + kMiscOff, kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  tc_fence_before();
  // a CTA gave up waiting (in this or an earlier launch): skip the work until the
  // error word is read and cleared; decided once per CTA
  const Shares shares = build<kWindowed>(
      p, smem, tid == 0 && (*reinterpret_cast<volatile uint32_t *>(&g_chunk_errors) & kErrTimeout));
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kMiscOff);
  const int cta = blockIdx.x;
  const bool works = cta < shares.W;
  const int *ranks = reinterpret_cast<const int *>(smem + kRankOff);
  // ranges that no CTA has cut nothing
  if (tid == 0 && cta >= (shares.front ? ranks[shares.W]
                                       : shares.W == 0 ? 0 : static_cast<int>(quotient(shares.U + shares.even - 1, shares.even))))
    p.cuts[cta].pieces = 0;

  if (warp == 0 && works) {
    // -------------------------------------------------------------- TMA producer
    auto wait_all = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait_(bar(i), parity, abort)); };
    const Wave *waves = reinterpret_cast<const Wave *>(smem + kWaveOff);
    volatile int *descs = reinterpret_cast<volatile int *>(smem + kDescOff);
    // the range: where it starts (s, head, i, first) and its length
    const int64_t *starts = reinterpret_cast<const int64_t *>(smem + kShareOff);
    auto start = [&](int c) { return shares.front ? starts[c] : min(c * shares.even, shares.U); };
    auto rank_of = [&](int c) { return shares.front ? ranks[c] : c; };
    const int64_t u_lo = start(cta);
    const int rank = rank_of(cta);
    int left = static_cast<int>(start(cta + 1) - u_lo);  // steps that no piece has yet
    int s = 0, head = 0, i = 0, n_tiles = 0, first = 0;
    Seq q = {0, 0, 0};
    if (left > 0) {
      const int64_t *steps = reinterpret_cast<const int64_t *>(smem + kStepsOff);
      s = find(steps, p.num_seqs, u_lo);  // it has steps
      q = reinterpret_cast<const Seq *>(smem + kSeqOff)[s];
      n_tiles = tiles_of(p, q);
      int64_t skip = u_lo - steps[s];
      const int64_t per_head = quotient(steps[s + 1] - steps[s], p.num_kv_heads);
      head = static_cast<int>(quotient(skip, per_head));
      skip -= head * per_head;
      for (i = 0; n_tiles > 1; i += 32) {  // the tile that holds step `skip` of the head: 32 at a time
        const int n = i + lane < n_tiles ? tile_of<kWindowed>(p, q, i + lane).steps() : 0;
        int incl = n;  // 32 tiles have fewer than 2^31 steps
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += x;
        }
        const uint32_t beyond = __ballot_sync(0xffffffffu, incl > skip);
        if (beyond != 0 || i + 32 >= n_tiles) {  // the step lies within the head: some lane is beyond it
          const int at = max(__ffs(beyond) - 1, 0);
          skip -= __shfl_sync(0xffffffffu, incl - n, at);
          i += at;
          break;
        }
        skip -= __shfl_sync(0xffffffffu, incl, 31);
      }
      first = static_cast<int>(skip);
    }
    // The tile that the range's start cuts, if no range before does, for the joining kernel.
    auto record_cut = [&](const Seq &sq, int at, int kv_head, int from) {
      auto owner = [&](int64_t u) {
        return shares.front ? find(starts, shares.W, u) : static_cast<int>(quotient(u, shares.even));
      };
      ChunkCut cut = {};
      const int64_t P0 = u_lo - from;
      if (from > 0) {
        const int before = owner(u_lo - 1);  // the range before
        if (start(before) <= P0) {
          const Tile t = tile_of<kWindowed>(p, sq, at);
          cut.pieces = rank_of(owner(P0 + t.steps() - 1)) - rank_of(before) + 1;
          cut.slot0 = 2 * rank_of(before) + (start(before) < P0 ? 1 : 0);
          cut.head = kv_head;
          cut.row = sq.q0 + t.t0;
          cut.n_tok = t.n_tok;
        }
      }
      if (lane == 0) p.cuts[rank] = cut;
    };
    const Seq cut_q = q;
    const int cut_tile = i, cut_head = head;
    const bool in_a_range = left > 0;
    struct Work {  // a piece, as its copies need it
      Piece d;
      const int32_t *table;  // of its sequence
      int lo, ctx;           // the first key of its window, the sequence's keys
    };
    int n_pieces = 0;
    bool in_range = false;  // a piece of the range has been published
    // The next piece into x, published; false if a wait gave up.
    auto next_piece = [&](Work &x) -> bool {
      const int slot = n_pieces % kDescs;
      Piece &d = x.d;
      d.steps = 0;
      const bool wave = n_pieces < shares.waves;
      if (wave || left > 0) {
        Seq sq;
        int at, xs, from = 0;
        if (wave) {
          const Wave w = waves[n_pieces];
          sq = w.q, at = w.tile, xs = w.s, d.head = w.head;
        } else {
          if (in_range && ++i == n_tiles) {
            i = 0;
            if (++head == p.num_kv_heads) {
              head = 0;
              bool bad;
              do q = load_seq(p, ++s, bad);  // steps are left, so a sequence has them
              while (q.Lq == 0);
              n_tiles = tiles_of(p, q);
            }
          }
          if (!in_range) from = first;
          sq = q, at = i, xs = s, d.head = head;
        }
        const Tile t = tile_of<kWindowed>(p, sq, at);
        const int all = t.steps();
        d.steps = wave ? all : min(all - from, left);
        d.first = from;
        d.lead = t.lead;
        d.j_start = t.j_start;
        d.pos = sq.ctx - sq.Lq + t.t0;
        d.row = sq.q0 + t.t0;
        d.n_tok = t.n_tok;
        d.slot = d.steps == all ? -1 : 2 * rank + (in_range ? 1 : 0);
        x.table = p.block_tables + static_cast<int64_t>(xs) * p.max_blocks;
        x.lo = t.lo;
        x.ctx = sq.ctx;
        if (!wave) {
          left -= d.steps;
          in_range = true;
        }
      }
      if (n_pieces >= kDescs && !wait_all(kBarDescFree + slot, ((n_pieces / kDescs) - 1) & 1)) return false;
      if (lane == 0) {
        const int *src = reinterpret_cast<const int *>(&d);
#pragma unroll
        for (int k = 0; k < kPieceInts; ++k) descs[slot * kDescInts + k] = src[k];
        mbar_arrive(bar(kBarDesc + slot));  // publishes it
      }
      __syncwarp();
      ++n_pieces;
      return true;
    };
    // Lane b < 128 / box_rows owns the b-th box of every key tile: it reads that
    // box's table entry a step ahead and issues the box's copies; lane 0 arms the
    // barriers. Boxes that no row of the tile sees are left out.
    const int box_rows = p.box_rows;
    auto key_of = [&](const Work &x, int j) { return x.d.key_tile(j) * kKeys + lane * box_rows; };
    auto wanted = [&](const Work &x, int j) {
      const int k = key_of(x, j);
      return lane * box_rows < kKeys && k < x.ctx && (!kWindowed || k + box_rows > x.lo || k < p.sinks);
    };
    auto entry = [&](const Work &x, int j) {
      return wanted(x, j) ? __ldg(x.table + fast_quotient(key_of(x, j), p.block)) : -1;
    };
    Work cur = {}, next = {};
    bool good = next_piece(cur);
    int32_t blk = cur.d.steps > 0 ? entry(cur, 0) : -1;
    int g = 0;  // steps so far
    // V goes out a step behind K: the next K is wanted first, and its stage is free first
    int32_t v_row = -1;
    uint32_t v_bytes = 0, v_unseen = 0;
    int v_head = 0;
    auto load_v = [&](int step) -> bool {
      const int b = step & 1;
      // P.V of step - 2 has been the last to read this V tile
      if (step >= 2 && !wait_all(kBarO + b, ((step >> 1) - 1) & 1)) return false;
      if (lane == 0) {
        unseen[b] = v_unseen;
        mbar_arrive_expect_tx(bar(kBarV + b), v_bytes);  // publishes `unseen` as well
      }
      __syncwarp();
      if (v_row >= 0) {
        const uint32_t at = sbase + kVOff + b * kTileBytes + lane * box_rows * 128;
        tma_load_3d(at, &v_map, bar(kBarV + b), 0, v_head, v_row);
        tma_load_3d(at + kHalfBytes, &v_map, bar(kBarV + b), 64, v_head, v_row);
      }
      return true;
    };
    for (int piece = 0; good && cur.d.steps > 0; ++piece) {
      const int steps = cur.d.steps, kv_head = cur.d.head, qb = piece & 1;
      if (piece >= 2 && !(good = wait_all(kBarQFree + qb, ((piece >> 1) - 1) & 1))) break;
      if (lane == 0) {
        const uint32_t dst = sbase + kQOff + qb * kTileBytes;
        mbar_arrive_expect_tx(bar(kBarQ + qb), kTileBytes);
        tma_load_3d(dst, &q_map, bar(kBarQ + qb), 0, kv_head << p.gqa_log2, cur.d.row);
        tma_load_3d(dst + kHalfBytes, &q_map, bar(kBarQ + qb), 64, kv_head << p.gqa_log2, cur.d.row);
      }
      __syncwarp();
      for (int j = 0; good && j < steps; ++j, ++g) {
        const int k0 = cur.d.key_tile(j) * kKeys;
        // V rows that no row of the tile sees: from .. to - 1 and end ..
        const uint32_t from = static_cast<uint32_t>(min(max(p.sinks - k0, 0), kKeys));
        const uint32_t to = static_cast<uint32_t>(min(max(cur.lo - k0, 0), kKeys));
        const uint32_t end = static_cast<uint32_t>(min(cur.ctx - k0, kKeys));
        int32_t row = -1;  // cache row of this lane's box
        if (wanted(cur, j)) {
          if (blk >= 0 && blk < p.num_blocks) {
            const uint32_t key = key_of(cur, j);
            row = blk * static_cast<int32_t>(p.block.d) + (key - fast_quotient(key, p.block) * p.block.d);
          } else {
            atomicOr(&g_chunk_errors, kErrBlock);
          }
        }
        // the entry of the next step, which may be the next piece's first
        if (j + 1 < steps)
          blk = entry(cur, j + 1);
        else if (j > 0)
          blk = next.d.steps > 0 ? entry(next, 0) : -1;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, row >= 0)) * 2u * box_rows * 128u;
        const int b = g & 1;
        // S of step g - 2 has been the last to read this K tile
        if (g >= 2) good = good && wait_all(kBarS + b, ((g >> 1) - 1) & 1);
        if (!good) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(kBarK + b), bytes);
        __syncwarp();
        if (row >= 0) {
          const uint32_t at = sbase + kKOff + b * kTileBytes + lane * box_rows * 128;
          tma_load_3d(at, &k_map, bar(kBarK + b), 0, kv_head, row);
          tma_load_3d(at + kHalfBytes, &k_map, bar(kBarK + b), 64, kv_head, row);
        }
        if (g == 0) {
          if (in_a_range) record_cut(cut_q, cut_tile, cut_head, first);
          __syncwarp();
          fence_proxy_async_smem();  // the copies of V overwrite the list
        }
        if (j == 0) {  // the next piece is known before the other warps are done with this one
          if (!(good = next_piece(next))) break;
          if (steps == 1) blk = next.d.steps > 0 ? entry(next, 0) : -1;
        }
        if (g >= 1 && !(good = load_v(g - 1))) break;
        v_row = row;
        v_bytes = bytes;
        v_head = kv_head;
        v_unseen = (from < to ? from | to << 8 : 0) | end << 16;
      }
      cur = next;
    }
    if (good && g >= 1) good = load_v(g - 1);
    if (!good) {
      if (lane == 0) fail();
      // copies that nobody waits for any more land in this CTA's memory: outlast them
      for (int k = 0; k < 200; ++k) __nanosleep(1000);
    }
  } else if (warp == kMmaWarp && works) {
    // -------------------------------------------------------------- MMA issuer
    // The whole warp runs the loop and its waits (warp-uniform control flow) and
    // one elected lane, always the same, issues every MMA and commit. The operand
    // descriptors are 32-bit low halves over one common high half.
    const uint32_t desc_hi = static_cast<uint32_t>(smem_desc_sw128(sbase, 16, 1024) >> 32);
    const uint32_t lo0 = static_cast<uint32_t>(smem_desc_sw128(sbase, 16, 1024));
    constexpr uint32_t kVLbo = static_cast<uint32_t>((kHalfBytes - 16) >> 4) << 16;
    bool good = true;
    int n = 0;  // pieces read
    // steps of the next piece, in a uniform register (0: none)
    auto read = [&]() -> int {
      const bool ok = wait_(bar(kBarDesc + n % kDescs), (n / kDescs) & 1, abort);
      if (!(good = __all_sync(0xffffffffu, ok))) return 0;
      const int steps = reinterpret_cast<const volatile int *>(smem + kDescOff)[n % kDescs * kDescInts];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarDescFree + n % kDescs));
      ++n;
      return static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(steps)));
    };
    // S of step g; opens, closes: the first, the last of piece `piece`
    auto issue_s = [&](int g, int piece, bool opens, bool closes) {
      const int b = g & 1, qb = piece & 1;
      bool ok = !opens || wait_(bar(kBarQ + qb), (piece >> 1) & 1, abort);
      ok = wait_(bar(kBarK + b), (g >> 1) & 1, abort) && ok;
      if (!(good = __all_sync(0xffffffffu, ok && good))) return;
      const uint32_t qd = lo0 + (kQOff >> 4) + qb * (kTileBytes >> 4), kd = lo0 + (kKOff >> 4) + b * (kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off16 = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
          mma_bf16_ss(tmem + b * kKeys, qd + off16, kd + off16, desc_hi, kIdescQK, kk > 0);
        }
        mma_commit(bar(kBarS + b));
        if (closes) mma_commit(bar(kBarQFree + qb));
      }
      __syncwarp();
    };
    auto issue_pv = [&](int g, bool opens) {
      const int b = g & 1;
      bool ok = wait_(bar(kBarV + b), (g >> 1) & 1, abort);
      if (!(good = __all_sync(0xffffffffu, ok && good))) return;
      const uint32_t u = unseen[b];
      if (u != kKeys << 16) {
        const uint32_t tile = sbase + kVOff + b * kTileBytes;
        auto zero = [&](int from, int to) {
          for (int i = from * 16 + lane; i < to * 16; i += 32) {
            const uint32_t addr = tile + ((i & 8) ? kHalfBytes : 0) + (i >> 4) * 128 + (i & 7) * 16;
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
          }
        };
        __syncwarp();
        zero(u & 255, (u >> 8) & 255);
        zero(u >> 16, kKeys);
        fence_proxy_async_smem();
      }
      ok = wait_(bar(kBarP + b), (g >> 1) & 1, abort);
      if (!(good = __all_sync(0xffffffffu, ok && good))) return;
      tc_fence_after();
      const uint32_t vd = lo0 + (kVOff >> 4) + b * (kTileBytes >> 4) + kVLbo, old = opens ? 0u : 1u;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_bf16_ts(tmem + kTmemO, tmem + b * kKeys + (kk >> 2) * 64 + (kk & 3) * 8, vd + ((kk * 16 * 128) >> 4), desc_hi, kIdescPV,
                      kk > 0 ? 1u : old);
        mma_commit(bar(kBarO + b));
      }
      __syncwarp();
    };
    int g = 0, j = 0, steps = read();
    bool more = good && steps > 0;
    if (more) issue_s(0, 0, true, steps == 1);
#pragma unroll 1
    while (good && more) {
      const bool opens = j == 0;
      if (++j == steps) {
        steps = read();
        more = steps > 0;
        j = 0;
      }
      if (good && more) issue_s(g + 1, n - 1, j == 0, j + 1 == steps);
      if (good) issue_pv(g, opens);
      ++g;
    }
    // every copy that this CTA needs has landed: the next kernel may start launching
    if (lane == 0) griddep_launch_dependents();
    // every MMA issued here has completed, and its commits arrived, before the CTA ends
    if (elect_one()) mma_commit(bar(kBarDone));
    __syncwarp();
    auto wait_all = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait_(bar(i), parity, abort)); };
    if (!wait_all(kBarDone, 0)) good = false;
    for (int x = max(g - 2, 0); good && x < g; ++x)
      good = wait_all(kBarS + (x & 1), (x >> 1) & 1) && wait_all(kBarO + (x & 1), (x >> 1) & 1);
    for (int x = max(n - 3, 0); good && x < n - 1; ++x) good = wait_all(kBarQFree + (x & 1), (x >> 1) & 1);
    if (!good && lane == 0) fail();
  } else if (warp >= kSoftmaxWarp0 && works) {
    // -------------------------------------------------------------- softmax
    const int half = (warp - kSoftmaxWarp0) >> 2;  // of the columns
    const int quad = warp & 3;                     // TMEM lane quadrant this warp may access
    const int r = quad * 32 + lane;                // row within the tile == TMEM lane
    const int tok0 = (quad * 32) >> p.gqa_log2, tok = r >> p.gqa_log2;  // the warp's first token, the row's
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tO = tmem + kTmemO + half * 64 + lane_off;
    const uint32_t scr = sbase + kEpiOff + (warp - kSoftmaxWarp0) * kEpiWarpBytes;
    // by half: maxima of two steps, then two sums of two pieces
    volatile float *swap = reinterpret_cast<volatile float *>(smem + kSwapOff) + r;
    const uint32_t masked = p.scale_log2 < 0.f ? 0x7F800000u : 0xFF800000u;  // times the scale: -inf
    bool good = true;
    int g = 0;
    uint32_t x_par = 0;  // parity of the next exchange
    // Both warps of the quadrant have come to offer(), and see what the other wrote before.
    auto offer = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarX + quad));
    };
    auto meet = [&]() -> bool {
      const bool ok = __all_sync(0xffffffffu, wait_(bar(kBarX + quad), x_par, abort));
      x_par ^= 1;
      return ok;
    };
    Piece d;
    bool live = false;
    int lim = 0;  // last key this row sees
    uint32_t x[64];  // the thread's logits of the step
    // Reads those of the piece's step j, step h of the CTA, masked as -inf once scaled, and
    // offers their maximum to the other half's warp.
    auto logits = [&](int j, int h) -> bool {
      const int b = h & 1;
      if (!__all_sync(0xffffffffu, wait_(bar(kBarS + b), (h >> 1) & 1, abort))) return false;
      tc_fence_after();
      const uint32_t tS = tmem + b * kKeys + half * 64 + lane_off;
      tmem_ld32(tS, reinterpret_cast<uint32_t(&)[32]>(x[0]));
      tmem_ld32(tS + 32, reinterpret_cast<uint32_t(&)[32]>(x[32]));
      const int k0 = d.key_tile(j) * kKeys + half * 64;  // the thread's first key
      bool some = k0 + 63 > d.pos + tok0;  // some key is masked for some row of the warp
      if constexpr (kWindowed)  // the largest first key of the warp's rows
        some = some || (k0 <= d.pos + tok0 + (31 >> p.gqa_log2) - p.window && k0 + 64 > p.sinks);
      tmem_wait_ld();
      if (some) {
        const int keep = lim - k0;  // columns up to it are at or before the row's position
        auto below = [](int i) { return i <= 0 ? 0u : i >= 32 ? 0xffffffffu : (1u << i) - 1; };
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t seen = below(keep + 1 - c);  // as bits
          if constexpr (kWindowed)              // but for those between the sinks and the window
            seen &= ~below(keep - p.window + 1 - c) | below(p.sinks - k0 - c);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(seen >> i & 1)) x[c + i] = masked;
        }
      }
      float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (p.scale_log2 >= 0.f) {
#pragma unroll
        for (int i = 0; i < 64; i += 2)
          a[(i >> 1) & 3] = fmax3(a[(i >> 1) & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
      } else {
#pragma unroll
        for (int i = 0; i < 64; ++i) a[i & 3] = fmaxf(a[i & 3], -__uint_as_float(x[i]));
      }
      // -inf stays -inf; two steps' worth of places: a warp may be a step ahead of the
      // other's reading
      swap[(b * 2 + half) * kRows] =
          fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * fabsf(p.scale_log2);
      offer();
      return true;
    };
    // A piece whose output is still to be written. That is done when the next piece's first
    // logits have been read: its last P.V runs meanwhile, and one exchange serves both.
    struct Ended {
      int slot, row, n_tok, head;
      float m, l, lr;
    } e = {};
    bool ended = false;
    auto finish = [&](int n) -> bool {  // e is piece n, its last step g - 1
      // The next P.V, which overwrites O, waits for this warp's next P.
      const int b = (g - 1) & 1;
      if (!__all_sync(0xffffffffu, wait_(bar(kBarO + b), ((g - 1) >> 1) & 1, abort))) return false;
      tc_fence_after();
      const volatile float *sums = swap + (4 + (n & 1) * 4 + 1 - half) * kRows;
      const float l = e.l + sums[0], lr = e.lr + sums[2 * kRows];
      const int n_valid = min(32, (e.n_tok - tok0) << p.gqa_log2);
      const float inv = e.slot < 0 ? 1.f / lr : 1.f;
      const int64_t row0 = static_cast<int64_t>(e.row + tok0) * p.num_q_heads + (static_cast<int64_t>(e.head) << p.gqa_log2);
#pragma unroll 1
      for (int c = 0; c < 64; c += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
        const int col = half * 64 + c;
        if (e.slot < 0) {
          uint32_t y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            y[i] = pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
          store_rows(y, scr, n_valid, lane, [&](int i) {
            const int64_t at = row0 + static_cast<int64_t>(i >> p.gqa_log2) * p.num_q_heads + (i & ((1 << p.gqa_log2) - 1));
            return reinterpret_cast<uint8_t *>(p.out + at * kD + col);
          });
        } else {
          float *dst = p.ws_o + (static_cast<int64_t>(e.slot) * kRows + quad * 32) * kD + col;
          store_rows(o, scr, n_valid, lane, [&](int i) { return reinterpret_cast<uint8_t *>(dst + i * kD); });
          store_rows(o + 16, scr, n_valid, lane, [&](int i) { return reinterpret_cast<uint8_t *>(dst + i * kD + 16); });
        }
      }
      if (tok < e.n_tok && half == 0) {
        if (e.slot >= 0)
          p.ws_ml[static_cast<int64_t>(e.slot) * kRows + r] = make_float4(e.m, l, lr, 0.f);
        else if (p.lse != nullptr)
          p.lse[row0 + static_cast<int64_t>(lane >> p.gqa_log2) * p.num_q_heads + (lane & ((1 << p.gqa_log2) - 1))] =
              (e.m + log2f(l)) * kLn2;
      }
      return true;
    };
#pragma unroll 1
    for (int n = 0;; ++n) {
      if (!(good = __all_sync(0xffffffffu, wait_(bar(kBarDesc + n % kDescs), (n / kDescs) & 1, abort)))) break;
      read_piece<kPieceInts>(n, smem, bars, lane, d);
      const bool any = d.steps > 0 && tok0 < d.n_tok;  // some row of the warp is live
      live = tok < d.n_tok;
      lim = d.pos + tok;
      if (any) {
        if (!(good = logits(0, g))) break;
      } else if (ended) {
        offer();
      }
      if ((any || ended) && !(good = meet())) break;
      if (ended && !(good = finish(n - 1))) break;
      ended = any;
      if (d.steps == 0) break;
      if (!any) {
        tc_fence_before();  // finish() may have read O, which this piece's first P.V overwrites
        __syncwarp();
        for (int j = 0; j < d.steps && good; ++j, ++g) {
          good = __all_sync(0xffffffffu, wait_(bar(kBarS + (g & 1)), (g >> 1) & 1, abort));
          if (lane == 0) mbar_arrive(bar(kBarP + (g & 1)));
        }
        if (!good) break;
        continue;
      }
      float m = kFloor, l = 0.f, lr = 0.f;
#pragma unroll 1
      for (int j = 0; j < d.steps; ++j, ++g) {
        const int b = g & 1;
        // The running maximum moves only where it is exceeded by more than 2^8: the
        // warps then rescale O. A piece's first step always does.
        const float mx = fmaxf(swap[b * 2 * kRows], swap[(b * 2 + 1) * kRows]);
        if (__any_sync(0xffffffffu, live && !(mx <= m + kLazyMax))) {
          const float m_new = fmaxf(m, mx);
          if (j > 0) {
            // O holds every step up to j - 1 once that P.V is complete
            if (!(good = __all_sync(0xffffffffu, wait_(bar(kBarO + (b ^ 1)), ((g - 1) >> 1) & 1, abort)))) break;
            tc_fence_after();
            const float alpha = fast_exp2(m - m_new);
#pragma unroll 1
            for (int c = 0; c < 64; c += 16) {
              uint32_t o[16];
              tmem_ld16(tO + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(tO + c, o);
            }
            l *= alpha;
            lr *= alpha;
          }
          m = m_new;
        }
        // P = 2^(x * scale - m), packed two per column over the first columns of the
        // thread's own half, and the sum of the fp32 values over eight chains.
        uint32_t pk[32];
        {
          const uint32_t tP = tmem + b * kKeys + half * 64 + lane_off;
          float s8[8] = {};
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            float e[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) e[i] = fast_exp2(fmaf(__uint_as_float(x[c + i]), p.scale_log2, -m));
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[c / 2 + i] = pack_bf16x2(e[2 * i], e[2 * i + 1]);
            tmem_st16(tP + c / 2, reinterpret_cast<uint32_t(&)[16]>(pk[c / 2]));
#pragma unroll
            for (int i = 0; i < 32; ++i) s8[i & 7] += e[i];
          }
          l += ((s8[0] + s8[1]) + (s8[2] + s8[3])) + ((s8[4] + s8[5]) + (s8[6] + s8[7]));
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarP + b));
        const bool more = j + 1 < d.steps;
        if (more && !(good = logits(j + 1, g + 1))) break;
        // the sum of the rounded values, while the other half's maximum is on its way
        {
          float r8[8] = {};
#pragma unroll
          for (int i = 0; i < 32; ++i) add_bf16x2_to_f32(r8[2 * (i & 3)], r8[2 * (i & 3) + 1], pk[i]);
          lr += ((r8[0] + r8[1]) + (r8[2] + r8[3])) + ((r8[4] + r8[5]) + (r8[6] + r8[7]));
        }
        if (more && !(good = meet())) break;
      }
      if (!good) break;
      // (in the other piece's places the other warp may still be reading)
      swap[(4 + (n & 1) * 4 + half) * kRows] = l;
      swap[(6 + (n & 1) * 4 + half) * kRows] = lr;
      e = {d.slot, d.row, d.n_tok, d.head, m, l, lr};
    }
    if (!good && lane == 0) fail();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the pieces of the tiles that ranges cut: CTA (k, y) takes rows kJoinRows y ..
// of the tile that the start of range k + 1 is the first to cut, a warp a row, four dims
// a lane. Piece x > 0 is in slot 2 (range of piece 0 + x).
constexpr int kJoinWarps = 4;
constexpr int kJoinRows = 4;
// Pieces whose outputs are in flight, where there are more than two (most tiles are cut once). 20
// rows over 32,000 keys, one tile over every SM, take 25 us in all, with 4 of them 34; with 16
// registers run short where there are many rows (23 ragged segments 71 us for 66). Few rows
// split between a CTA's warps: 19 and 54 us on that tile and the two documents, here 25 and 52.
constexpr int kJoinLoads = 8;

__global__ void __launch_bounds__(kJoinWarps * 32) chunk_join_kernel(const ChunkParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // after a timeout (in the kernel just before this one, or in an earlier launch,
  // which made that kernel skip its work) the pieces are stale: write nothing
  if (*reinterpret_cast<volatile uint32_t *>(&g_chunk_errors) & kErrTimeout) return;
  const ChunkCut cut = p.cuts[blockIdx.x + 1];
  const int rows = min(cut.n_tok << p.gqa_log2, kJoinRows * (static_cast<int>(blockIdx.y) + 1));
  if (cut.pieces == 0) return;
  for (int r = kJoinRows * blockIdx.y + warp; r < rows; r += kJoinWarps) {
    // piece x > 0 is 2 x slots behind the even slot of piece 0's range
    const int64_t even = static_cast<int64_t>(cut.slot0 & ~1) * kRows + r;
    const float4 *ml0 = p.ws_ml + even, *o0 = reinterpret_cast<const float4 *>(p.ws_o + even * kD) + lane;
    auto rows_on = [&](int x) { return x == 0 ? (cut.slot0 & 1) * kRows : 2 * x * kRows; };
    float M = kFloor, l = 0.f, lr = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    // pieces base .. base + kLoads - 1, the loads of all in flight; past the last, that one
    // again with no weight
    auto join = [&](auto loads, int base) {
      constexpr int kLoads = decltype(loads)::value;
      float4 ml[kLoads], o[kLoads];
      float top = M;
#pragma unroll
      for (int x = 0; x < kLoads; ++x) {
        const int i = rows_on(min(base + x, cut.pieces - 1));
        ml[x] = ml0[i];
        o[x] = o0[i * (kD / 4)];
      }
#pragma unroll
      for (int x = 0; x < kLoads; ++x) {
        if (base + x >= cut.pieces) ml[x].x = -INFINITY;
        top = fmaxf(top, ml[x].x);
      }
      const float old = fast_exp2(M - top);
      M = top;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= old;
      l *= old;
      lr *= old;
#pragma unroll
      for (int x = 0; x < kLoads; ++x) {
        const float f = fast_exp2(ml[x].x - M);
        acc[0] = fmaf(o[x].x, f, acc[0]);
        acc[1] = fmaf(o[x].y, f, acc[1]);
        acc[2] = fmaf(o[x].z, f, acc[2]);
        acc[3] = fmaf(o[x].w, f, acc[3]);
        l = fmaf(ml[x].y, f, l);
        lr = fmaf(ml[x].z, f, lr);
      }
    };
    if (cut.pieces <= 2)
      join(std::integral_constant<int, 2>{}, 0);
    else
      for (int base = 0; base < cut.pieces; base += kJoinLoads) join(std::integral_constant<int, kJoinLoads>{}, base);
    const float inv = 1.f / lr;
    const int64_t row = static_cast<int64_t>(cut.row + (r >> p.gqa_log2)) * p.num_q_heads +
                        (static_cast<int64_t>(cut.head) << p.gqa_log2) + (r & ((1 << p.gqa_log2) - 1));
    uint2 v;
    v.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    v.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2 *>(p.out + row * kD + lane * 4) = v;
    if (lane == 0 && p.lse != nullptr) p.lse[row] = (M + log2f(l)) * kLn2;
  }
}

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

}  // namespace

cudaError_t launch_chunk(const ChunkArgs &a, const CUtensorMap &q_map, const CUtensorMap &k_map,
                         const CUtensorMap &v_map, cudaStream_t stream) {
  ChunkParams p;
  p.cu_q = a.cu_seqlens_q;
  p.lens = a.context_lens;
  p.block_tables = a.block_tables;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.ws_o = a.ws_o;
  p.ws_ml = reinterpret_cast<float4 *>(a.ws_ml);
  p.cuts = a.cuts;
  p.block = fast_div(a.block_size);
  p.max_blocks = a.max_blocks;
  p.num_seqs = a.num_seqs;
  p.total_q = a.total_q;
  p.max_seqlen_q = a.max_seqlen_q;
  p.max_context_len = a.max_context_len;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.num_blocks = a.num_blocks;
  p.gqa_log2 = log2_of(a.num_q_heads / a.num_kv_heads);
  const int tokens = kRows >> p.gqa_log2;
  const int tiles = (a.max_seqlen_q - 1) / tokens + 1;  // of the longest segment
  p.lanes_log2 = tiles >= 32 ? 5 : log2_of(tiles);
  p.shared_keys = tiles > 1;
  p.window = a.window;
  p.sinks = a.sinks;
  p.box_rows = prefill_box_rows(a.block_size);
  // a factor of zero would make NaN of masked logits: the smallest normal number
  // gives the same weights to any logits below 10^30
  p.scale_log2 = a.scale_log2 == 0.f ? 1.17549435e-38f : a.scale_log2;
  const auto kernel = a.window > 0 ? chunk_kernel<true> : chunk_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(a.num_ctas), dim3(kThreads), kSmemBytes, stream, q_map, k_map, v_map, p);
  // tiles of one step have no boundary inside
  if (e != cudaSuccess || a.num_ctas < 2 || (tiles == 1 && a.max_context_len <= kKeys)) return e;
  const int rows = static_cast<int>(std::min<int64_t>(kRows, static_cast<int64_t>(a.max_seqlen_q) << p.gqa_log2));
  return launch_pdl(chunk_join_kernel, dim3(a.num_ctas - 1, (rows + kJoinRows - 1) / kJoinRows),
                    dim3(kJoinWarps * 32), 0, stream, p);
}

cudaError_t chunk_error_word(uint32_t **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_chunk_errors);
}

}  // namespace pkv
