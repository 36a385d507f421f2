// Attention of chunks of new tokens over the paged cache, on the 5th-generation
// tensor cores (tcgen05, accumulators in TMEM, operands staged by TMA): segments of
// one token, of a few (drafted tokens, the tail of a prompt) or of thousands in one
// call, with a sliding window and sinks.
//
// Work list. A tile is 128 query rows of one KV head: 128 / G tokens times the head's
// G query heads, which are neighbours in the row of a token, so that one TMA box
// loads them in the order (token, head). A tile's steps are the 128-key tiles that
// its rows see: those that hold sinks, then those from its window's start to its
// last token's position. The steps of all tiles, listed in (sequence, KV head, tile,
// step) order, are cut into equal contiguous ranges, one per CTA (one CTA per SM),
// whatever the lengths: a few tokens over long contexts use every SM, and long
// chunks, many tiles a CTA, have no tail. A tile cut by a range boundary leaves its
// pieces (maximum, sums, unnormalised output) in the workspace, a CTA's first in slot
// 2c, its last in slot 2c + 1; a second kernel, launched right behind, joins them.
//
// 8 warps:
//   warp 0     TMA producer: Q tiles (two buffers), K and V tiles (two each).
//   warp 1     MMAs. S(j + 1) = Q K(j + 1)^T goes out before O += P(j) V(j), into
//              the other of two S buffers in TMEM, so that the tensor pipe computes the
//              next logits while the softmax warps work on these. MMAs complete in
//              order: S(j) complete means that P.V of step j - 2 is. While it
//              waits for P(j) it zeroes the V rows that no row of the segment sees (past
//              the last key; between the sinks and the window), which may be absent or
//              hold anything: a probability of zero must not meet a NaN. Their
//              logits are masked by selection.
//   warp 2     walks the range and publishes its pieces to the other warps.
//   warps 4-7  softmax, one row per thread (TMEM lane = row): read S, mask, online
//              softmax in base 2 with a lazy maximum, P as bf16 over S's columns; at
//              the end of a piece the output.
//
// P is rounded to bf16 and the output divided by the sum of the rounded
// probabilities, the weights that the products used; the lse comes from the fp32 sum.
#include <algorithm>
#include <cmath>

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
constexpr int kThreads = 256;
constexpr int kDescs = 4;                   // pieces published ahead
constexpr int kDescInts = 16;

// shared memory
constexpr int kQOff = 0;                            // two Q tiles
constexpr int kKOff = kQOff + 2 * kTileBytes;       // two K tiles
constexpr int kVOff = kKOff + 2 * kTileBytes;       // two V tiles
constexpr int kEpiWarpBytes = 32 * 128;
constexpr int kEpiOff = kVOff + 2 * kTileBytes;     // staging areas of the four softmax warps
constexpr int kBarOff = kEpiOff + 4 * kEpiWarpBytes;
// barriers (8 bytes each), those of steps and Q buffers in pairs by parity: K and V
// landed, S complete (which frees its K), P written, P.V complete (which frees its V),
// Q landed, Q free; descriptors full and empty; the end
constexpr int kBarK = 0, kBarV = 2, kBarS = 4, kBarP = 6, kBarO = 8, kBarQ = 10, kBarQFree = 12, kBarDesc = 14, kBarDescFree = kBarDesc + kDescs, kBarDone = kBarDescFree + kDescs, kNumBars = kBarDone + 1;
constexpr int kDescOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;
constexpr int kMiscOff = kDescOff + kDescs * kDescInts * 4;  // TMEM address, abort flag
constexpr int kPrefixOff = kMiscOff + 16;                    // int64 [S + 1]
constexpr int smem_bytes(int num_seqs) { return kPrefixOff + 8 * (num_seqs + 1) + 1024; }  // + slack for alignment
static_assert(smem_bytes(kChunkMaxSeqs) <= 227 * 1024, "shared memory per CTA");

constexpr uint32_t kTmemCols = 512;  // S (two), O: 128 columns each; a power of two
constexpr int kTmemO = 256;
constexpr uint32_t kIdescQK = idesc_bf16_f32(kRows, kKeys, 0, 0);  // A = Q K-major, B = K K-major
constexpr uint32_t kIdescPV = idesc_bf16_f32(kRows, kD, 0, 1);     // A = P (TMEM), B = V MN-major
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLazyBound = 256.0f;  // the largest sum of a row's step taken with an old maximum
constexpr float kFloor = -1e30f;      // finite, below every logit: a row that has seen no key yet

struct ChunkParams {
  const int32_t *cu_q, *lens, *block_tables;
  __nv_bfloat16 *out;
  float *lse;
  float *ws_o;         // [2 grid, 128, 128]
  float4 *ws_ml;       // [2 grid, 128]: maximum, sum, sum of the rounded
  ChunkCut *cuts;      // [grid]: the tile that boundary c is the first to cut
  FastDiv block;
  int32_t max_blocks, num_seqs, total_q, max_seqlen_q, max_context_len;
  int32_t num_q_heads, num_kv_heads, num_blocks;
  int32_t gqa_log2;    // log2 of the query heads of a KV head
  int32_t lanes_log2;  // lanes that add up one sequence's steps
  int32_t window, sinks, box_rows;
  float scale_log2;    // > 0; the sign is in flip
  uint32_t flip;       // sign bit of the logits' factor
};

__device__ __forceinline__ bool wait_(uint32_t bar, uint32_t parity, const volatile int *abort) {
  return mbar_wait(bar, parity, &g_chunk_errors, abort);
}

// A sequence's segment; Lq = 0: nothing to do.
struct Seq {
  int q0, Lq, ctx;
};
__device__ __forceinline__ Seq load_seq(const ChunkParams &p, int s, bool raise) {
  const int q0 = p.cu_q[s], q1 = p.cu_q[s + 1], ctx = p.lens[s];
  Seq r = {q0, q1 - q0, ctx};
  if (q0 == q1) return r;
  if (q0 < 0 || q1 < q0 || q1 > p.total_q || r.Lq > p.max_seqlen_q || ctx < r.Lq || ctx > p.max_context_len ||
      ctx > static_cast<int64_t>(p.max_blocks) * p.block.d) {
    if (raise) atomicOr(&g_chunk_errors, kErrSeqlens);
    r.Lq = 0;
  }
  return r;
}

// The key tiles of row tile rt: lead of them from the first key, then j_start ..
// n_end - 1; lo is the first key of its window.
struct Tile {
  int lead, j_start, n_end, lo;
  __device__ __forceinline__ int steps() const { return lead + n_end - j_start; }
};
__device__ __forceinline__ int tile_tokens(const ChunkParams &p) { return kRows >> p.gqa_log2; }
__device__ __forceinline__ Tile tile_of(const ChunkParams &p, int Lq, int ctx, int rt) {
  const int diag = ctx - Lq, t0 = rt * tile_tokens(p);
  Tile t;
  t.n_end = (diag + min(Lq, t0 + tile_tokens(p)) + kKeys - 1) / kKeys;
  t.lo = p.window > 0 ? max(0, diag + t0 + 1 - p.window) : 0;
  t.j_start = t.lo / kKeys;
  t.lead = min((p.sinks + kKeys - 1) / kKeys, t.j_start);
  return t;
}
__device__ __forceinline__ int row_tiles(const ChunkParams &p, int Lq) {
  return (Lq + tile_tokens(p) - 1) / tile_tokens(p);
}

// First step of CTA c's range among W CTAs over U steps (W <= U), and the CTA
// whose range holds step u.
__device__ __forceinline__ int64_t range_start(int64_t c, int64_t W, int64_t U) { return c * U / W; }
__device__ __forceinline__ int64_t owner_of(int64_t u, int64_t W, int64_t U) { return ((u + 1) * W + U - 1) / U - 1; }

// prefix[s] = steps of the sequences before s, for all s <= num_seqs; the whole CTA.
__device__ __forceinline__ void build_prefix(const ChunkParams &p, int64_t *prefix, bool raise) {
  const int tid = threadIdx.x, lanes = 1 << p.lanes_log2, sub = tid & (lanes - 1);
  for (int base = 0; base < p.num_seqs; base += kThreads >> p.lanes_log2) {
    const int s = base + (tid >> p.lanes_log2);
    int64_t n = 0;
    if (s < p.num_seqs) {
      const Seq q = load_seq(p, s, raise && sub == 0);
      const int n_rt = row_tiles(p, q.Lq);
      for (int rt = sub; rt < n_rt; rt += lanes) n += tile_of(p, q.Lq, q.ctx, rt).steps();
    }
    for (int off = lanes >> 1; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
    if (s < p.num_seqs && sub == 0) prefix[s + 1] = n * p.num_kv_heads;
  }
  __syncthreads();
  if (tid < 32) {
    int64_t carry = 0;
    for (int base = 0; base < p.num_seqs; base += 32) {
      const int s = base + tid;
      int64_t n = s < p.num_seqs ? prefix[s + 1] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, n, off);
        if (tid >= off) n += v;
      }
      if (s < p.num_seqs) prefix[s + 1] = carry + n;
      carry += __shfl_sync(0xffffffffu, n, 31);
    }
    if (tid == 0) prefix[0] = 0;
  }
  __syncthreads();
}

// A piece as the walker publishes it: steps first .. first + steps - 1 of a tile.
struct Piece {
  int steps;       // 0: no more pieces
  int first;
  int s, head;     // table row, KV head
  int row, n_tok;  // the tile's first token among all, and its tokens
  int pos;         // position of its first token
  int ctx, lead, j_start, lo;
  int slot;        // where its partial result goes, or -1: it is the whole tile
  __device__ __forceinline__ int key_tile(int j) const {  // of the piece's step j
    const int k = first + j;
    return k < lead ? k : k - lead + j_start;
  }
};
// The rows of a key tile that no row of the segment sees: from .. to - 1 (between sinks and
// window) and end .. (past the last key).
struct Unseen {
  int from, to, end;
  __device__ __forceinline__ Unseen(const Piece &d, int j, int sinks) {
    const int k0 = d.key_tile(j) * kKeys;
    from = max(sinks - k0, 0);
    to = min(d.lo - k0, kKeys);
    end = min(d.ctx - k0, kKeys);
  }
};
static_assert(sizeof(Piece) <= kDescInts * 4, "a piece fits its slot");

// The pieces of one CTA as a role reads them.
struct PieceReader {
  int n = 0;  // pieces read
  __device__ __forceinline__ bool next(uint8_t *smem, uint32_t bars, const volatile int *abort, int lane, Piece &d) {
    const int i = n % kDescs;
    if (!__all_sync(0xffffffffu, wait_(bars + 8 * (kBarDesc + i), (n / kDescs) & 1, abort))) return false;
    const volatile int *src = reinterpret_cast<const volatile int *>(smem + kDescOff) + i * kDescInts;
    int *dst = reinterpret_cast<int *>(&d);
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(Piece) / 4); ++k) dst[k] = src[k];
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * (kBarDescFree + i));
    ++n;
    return true;
  }
};
constexpr int kDescReaders = 2 + 4;  // producer, MMA and softmax warps

// 32 columns a lane through the warp's staging area to rows of 128 bytes each:
// words w[8 k .. 8 k + 3] and so on in 16-byte chunks, chunk c of row i at c ^ (i & 7),
// which keeps both sides free of bank conflicts; `to` gives a row's address.
template <typename To>
__device__ __forceinline__ void store_rows(const uint32_t (&w)[32], uint32_t scr, int n_valid, int lane, To to) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(scr + lane * 128 + ((k ^ (lane & 7)) * 16)),
                 "r"(w[4 * k]), "r"(w[4 * k + 1]), "r"(w[4 * k + 2]), "r"(w[4 * k + 3])
                 : "memory");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 4 * i + (lane >> 3), c = lane & 7;
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(scr + row * 128 + ((c ^ (row & 7)) * 16))
                 : "memory");
    if (row < n_valid) *reinterpret_cast<uint4 *>(to(row) + c * 16) = v;
  }
  __syncwarp();
}

__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const ChunkParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + kBarOff;
  auto bar = [&](int i) { return bars + 8u * i; };
  volatile int *abort = reinterpret_cast<volatile int *>(smem + kMiscOff + 4);
  int64_t *prefix = reinterpret_cast<int64_t *>(smem + kPrefixOff);
  auto fail = [&]() {
    *abort = 1;
    atomicOr(&g_chunk_errors, kErrTimeout);
  };

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool softmax = i >= kBarP && i < kBarP + 2;
      const bool readers = i >= kBarDescFree && i < kBarDescFree + kDescs;
      mbar_init(bar(i), softmax ? 4 : readers ? kDescReaders : 1);
    }
    *abort = 0;
    fence_barrier_init();
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  if (warp == 1) {
    tmem_alloc(sbase + kMiscOff, kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  tc_fence_before();
  // a CTA gave up waiting (in this or an earlier launch): skip the work until the
  // error word is read and cleared; decided once per CTA
  const bool skipped =
      __syncthreads_or(tid == 0 && (*reinterpret_cast<volatile uint32_t *>(&g_chunk_errors) & kErrTimeout));
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kMiscOff);

  const int64_t cta = blockIdx.x;
  if (!skipped) build_prefix(p, prefix, cta == 0);
  const int64_t U = skipped ? 0 : prefix[p.num_seqs];
  const int64_t W = min(static_cast<int64_t>(gridDim.x), U);
  if (cta >= W && tid == 0) p.cuts[cta].pieces = 0;

  if (cta < W) {
    if (warp == 2) {
      // ------------------------------------------------------------ walker
      const int64_t u_lo = range_start(cta, W, U);
      int64_t left = range_start(cta + 1, W, U) - u_lo;
      int lo = 0, hi = p.num_seqs - 1;  // the last s with prefix[s] <= u_lo: it has steps
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= u_lo) lo = mid; else hi = mid - 1;
      }
      int s = lo;
      Seq q = load_seq(p, s, false);
      int n_rt = row_tiles(p, q.Lq);
      const int64_t per_head = (prefix[s + 1] - prefix[s]) / p.num_kv_heads;
      const int64_t in_seq = u_lo - prefix[s];
      int head = static_cast<int>(in_seq / per_head);
      int64_t skip = in_seq - head * per_head;
      int rt = 0;
      for (;; rt += 32) {  // the row tile that holds step `skip` of the head: 32 at a time
        const int n = rt + lane < n_rt ? tile_of(p, q.Lq, q.ctx, rt + lane).steps() : 0;
        int64_t incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += v;
        }
        const uint32_t beyond = __ballot_sync(0xffffffffu, incl > skip);
        if (beyond != 0) {
          const int at = __ffs(beyond) - 1;
          skip -= __shfl_sync(0xffffffffu, incl - n, at);
          rt += at;
          break;
        }
        skip -= __shfl_sync(0xffffffffu, incl, 31);
        if (rt + 32 >= n_rt) break;  // not reached: the step lies within the head
      }
      int first = static_cast<int>(skip);
      for (int n = 0;; ++n) {
        Piece d;
        d.steps = 0;
        if (left > 0) {
          const Tile t = tile_of(p, q.Lq, q.ctx, rt);
          const int all = t.steps();
          d.steps = static_cast<int>(min(static_cast<int64_t>(all - first), left));
          d.first = first;
          d.s = s;
          d.head = head;
          d.row = q.q0 + rt * tile_tokens(p);
          d.n_tok = min(tile_tokens(p), q.Lq - rt * tile_tokens(p));
          d.pos = q.ctx - q.Lq + rt * tile_tokens(p);
          d.ctx = q.ctx;
          d.lead = t.lead;
          d.j_start = t.j_start;
          d.lo = t.lo;
          d.slot = d.steps == all ? -1 : static_cast<int>(2 * cta) + (n == 0 ? 0 : 1);
          if (n == 0 && lane == 0) {
            // the tile that this CTA's boundary cuts, if no boundary before does
            ChunkCut cut = {};
            const int64_t P0 = u_lo - first;
            if (first > 0 && range_start(cta - 1, W, U) <= P0) {
              cut.pieces = static_cast<int32_t>(owner_of(P0 + all - 1, W, U) - (cta - 1) + 1);
              cut.slot0 = static_cast<int32_t>(2 * (cta - 1) + (range_start(cta - 1, W, U) < P0 ? 1 : 0));
              cut.head = head;
              cut.row = d.row;
              cut.n_tok = d.n_tok;
            }
            p.cuts[cta] = cut;
          }
        }
        const int i = n % kDescs;
        if (n >= kDescs &&
            !__all_sync(0xffffffffu, wait_(bar(kBarDescFree + i), ((n / kDescs) - 1) & 1, abort))) {
          if (lane == 0) fail();
          break;
        }
        if (lane == 0) {
          volatile int *dst = reinterpret_cast<volatile int *>(smem + kDescOff) + i * kDescInts;
          const int *src = reinterpret_cast<const int *>(&d);
#pragma unroll
          for (int k = 0; k < static_cast<int>(sizeof(Piece) / 4); ++k) dst[k] = src[k];
          mbar_arrive(bar(kBarDesc + i));  // publishes it
        }
        __syncwarp();
        if (d.steps == 0) break;
        left -= d.steps;
        first = 0;
        if (left > 0 && ++rt == n_rt) {
          rt = 0;
          if (++head == p.num_kv_heads) {
            head = 0;
            do {
              ++s;
            } while (prefix[s + 1] == prefix[s]);  // steps are left, so a sequence has them
            q = load_seq(p, s, false);
            n_rt = row_tiles(p, q.Lq);
          }
        }
      }
    } else if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      // Lane b < 128 / box_rows owns the b-th box of every key tile: it reads that
      // box's table entry a step ahead and issues the box's copies; lane 0 arms the
      // barriers. Boxes that no row of the segment sees are left out.
      const int box_rows = p.box_rows, n_boxes = kKeys / box_rows;
      PieceReader reader;
      Piece d;
      bool good = true;
      int gk = 0;  // steps of this CTA so far
      while (good && (good = reader.next(smem, bars, abort, lane, d)) && d.steps > 0) {
        const int piece = reader.n - 1, qb = piece & 1;
        const int32_t *table = p.block_tables + static_cast<int64_t>(d.s) * p.max_blocks;
        auto key_of = [&](int j) { return d.key_tile(j) * kKeys + lane * box_rows; };
        auto wanted = [&](int j) {
          if (lane >= n_boxes || j >= d.steps) return false;
          const int k = key_of(j);
          return k < d.ctx && (k + box_rows > d.lo || k < p.sinks);
        };
        auto entry = [&](int j) { return wanted(j) ? __ldg(table + fast_quotient(key_of(j), p.block)) : -1; };
        int32_t blk = entry(0);
        if (piece >= 2 &&
            !__all_sync(0xffffffffu, wait_(bar(kBarQFree + qb), ((piece >> 1) - 1) & 1, abort))) {
          good = false;
          break;
        }
        if (lane == 0) {
          const uint32_t dst = sbase + kQOff + qb * kTileBytes;
          mbar_arrive_expect_tx(bar(kBarQ + qb), kTileBytes);
          tma_load_3d(dst, &q_map, bar(kBarQ + qb), 0, d.head << p.gqa_log2, d.row);
          tma_load_3d(dst + kHalfBytes, &q_map, bar(kBarQ + qb), 64, d.head << p.gqa_log2, d.row);
        }
        for (int j = 0; j < d.steps; ++j, ++gk) {
          const int32_t next = entry(j + 1);
          int32_t row = -1;  // cache row of this lane's box
          if (wanted(j)) {
            if (blk >= 0 && blk < p.num_blocks) {
              const uint32_t key = key_of(j);
              row = blk * static_cast<int32_t>(p.block.d) + (key - fast_quotient(key, p.block) * p.block.d);
            } else {
              atomicOr(&g_chunk_errors, kErrBlock);
            }
          }
          blk = next;
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, row >= 0)) * 2u * box_rows * 128u;
          const int b = gk & 1;
          const uint32_t at = b * kTileBytes + lane * box_rows * 128;
          // S of step gk - 2 has been the last to read this K tile, P.V this V tile
          if (gk >= 2 && !__all_sync(0xffffffffu, wait_(bar(kBarS + b), ((gk >> 1) - 1) & 1, abort))) {
            good = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(kBarK + b), bytes);
          __syncwarp();
          if (row >= 0) {
            tma_load_3d(sbase + kKOff + at, &k_map, bar(kBarK + b), 0, d.head, row);
            tma_load_3d(sbase + kKOff + at + kHalfBytes, &k_map, bar(kBarK + b), 64, d.head, row);
          }
          if (gk >= 2 && !__all_sync(0xffffffffu, wait_(bar(kBarO + b), ((gk >> 1) - 1) & 1, abort))) {
            good = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(kBarV + b), bytes);
          __syncwarp();
          if (row >= 0) {
            tma_load_3d(sbase + kVOff + at, &v_map, bar(kBarV + b), 0, d.head, row);
            tma_load_3d(sbase + kVOff + at + kHalfBytes, &v_map, bar(kBarV + b), 64, d.head, row);
          }
        }
      }
      // every copy of this CTA is issued: the next kernel may start launching
      if (lane == 0) griddep_launch_dependents();
      if (!good && lane == 0) fail();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp runs the loop and its waits (warp-uniform control flow) and
      // one elected lane, always the same, issues every MMA and commit. The operand
      // descriptors are 32-bit low halves over one common high half.
      auto wait_all = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait_(bar(i), parity, abort)); };
      const uint32_t desc_hi = static_cast<uint32_t>(smem_desc_sw128(sbase, 16, 1024) >> 32);
      const uint32_t lo0 = static_cast<uint32_t>(smem_desc_sw128(sbase, 16, 1024));
      constexpr uint32_t kVLbo = static_cast<uint32_t>((kHalfBytes - 16) >> 4) << 16;
      auto desc = [&](int off) { return lo0 + static_cast<uint32_t>(off >> 4); };
      auto issue_s = [&](int gk, int piece, bool opens, bool closes) -> bool {
        const int b = gk & 1, qb = piece & 1;
        if (opens && !wait_all(kBarQ + qb, (piece >> 1) & 1)) return false;
        if (!wait_all(kBarK + b, (gk >> 1) & 1)) return false;
        const uint32_t qd = desc(kQOff + qb * kTileBytes), kd = desc(kKOff + b * kTileBytes);
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
        return true;
      };
      auto issue_pv = [&](int gk, bool opens, const Unseen &u) -> bool {
        const int b = gk & 1;
        if (!wait_all(kBarV + b, (gk >> 1) & 1)) return false;
        if (u.from < u.to || u.end < kKeys) {
          auto zero = [&](int from, int to) {
            const uint32_t base = sbase + kVOff + b * kTileBytes;
            for (int i = from * 16 + lane; i < to * 16; i += 32) {
              const uint32_t addr = base + ((i & 8) ? kHalfBytes : 0) + (i >> 4) * 128 + (i & 7) * 16;
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
            }
          };
          zero(u.from, u.to);
          zero(u.end, kKeys);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!wait_all(kBarP + b, (gk >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t vd = desc(kVOff + b * kTileBytes) + kVLbo;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_bf16_ts(tmem + kTmemO, tmem + b * kKeys + kk * 8, vd + ((kk * 16 * 128) >> 4), desc_hi, kIdescPV,
                        (!opens || kk > 0) ? 1u : 0u);
          mma_commit(bar(kBarO + b));
        }
        __syncwarp();
        return true;
      };
      PieceReader reader;
      Piece d;
      bool good = reader.next(smem, bars, abort, lane, d);
      bool more = good && d.steps > 0;
      int gk = 0, j = 0;
      if (more) good = issue_s(0, 0, true, d.steps == 1);
      while (good && more) {
        const bool opens = j == 0;
        const Unseen unseen(d, j, p.sinks);
        if (++j == d.steps) {
          good = reader.next(smem, bars, abort, lane, d);
          more = good && d.steps > 0;
          j = 0;
        }
        if (good && more) good = issue_s(gk + 1, reader.n - 1, j == 0, j == d.steps - 1);
        if (good) good = issue_pv(gk, opens, unseen);
        ++gk;
      }
      // every MMA issued here has completed, and its commits arrived, before the CTA ends
      if (elect_one()) mma_commit(bar(kBarDone));
      __syncwarp();
      if (!wait_all(kBarDone, 0)) good = false;
      for (int g = max(gk - 2, 0); good && g < gk; ++g)
        good = wait_all(kBarS + (g & 1), (g >> 1) & 1) && wait_all(kBarO + (g & 1), (g >> 1) & 1);
      for (int n = max(reader.n - 3, 0); good && n < reader.n - 1; ++n)
        good = wait_all(kBarQFree + (n & 1), (n >> 1) & 1);
      if (!good && lane == 0) fail();
    } else if (warp >= 4) {
      // ------------------------------------------------------------ softmax
      const int quad = warp & 3;       // TMEM lane quadrant this warp may access
      const int r = quad * 32 + lane;  // row within the tile == TMEM lane
      const int tok = r >> p.gqa_log2, h = r & ((1 << p.gqa_log2) - 1);
      const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
      const uint32_t tO = tmem + kTmemO + lane_off;
      const uint32_t scr = sbase + kEpiOff + quad * kEpiWarpBytes;
      const uint64_t scl = f32x2(p.scale_log2, p.scale_log2);
      PieceReader reader;
      Piece d;
      bool good = true;
      int gk = 0;
      while (good && (good = reader.next(smem, bars, abort, lane, d)) && d.steps > 0) {
        const bool live = tok < d.n_tok;
        const bool any = (quad * 32) >> p.gqa_log2 < d.n_tok;  // some row of the warp is
        const int lim = d.pos + tok;                           // last key this row sees
        const int first = p.window > 0 ? lim - p.window + 1 : 0;
        // of the warp's rows: the smallest last key and the largest first one
        const int lim_min = d.pos + ((quad * 32) >> p.gqa_log2);
        const int first_max = p.window > 0 ? d.pos + ((quad * 32 + 31) >> p.gqa_log2) - p.window + 1 : 0;
        float m = kFloor, l = 0.f, lr = 0.f;
        for (int j = 0; j < d.steps; ++j, ++gk) {
          const int b = gk & 1;
          if (!__all_sync(0xffffffffu, wait_(bar(kBarS + b), (gk >> 1) & 1, abort))) {
            good = false;
            break;
          }
          if (any) {
            tc_fence_after();
            const uint32_t tS = tmem + b * kKeys + lane_off;
            const int k0 = d.key_tile(j) * kKeys;
            uint32_t x[kKeys];
#pragma unroll
            for (int c = 0; c < kKeys; c += 32) tmem_ld32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(&x[c]));
            tmem_wait_ld();
            if (p.flip != 0) {
#pragma unroll
              for (int c = 0; c < kKeys; ++c) x[c] ^= 0x80000000u;
            }
            // masked logits become -inf, their probabilities 0
            if (k0 + kKeys - 1 > lim_min || (k0 < first_max && k0 + kKeys > p.sinks)) {
              const int keep = lim - k0, skip = first - k0, sink = p.sinks - k0;
#pragma unroll
              for (int c = 0; c < kKeys; ++c)
                if (c > keep || (c < skip && c >= sink)) x[c] = 0xFF800000u;
            }
            // P = 2^(x * scale - mm), packed two per column over the first 64 columns
            // of S; ts and tr get the row's sums of the fp32 and of the rounded values
            auto exps = [&](float mm, float &ts, float &tr) {
              const uint64_t nm = f32x2(-mm, -mm);
              uint64_t s0 = 0, s1 = 0;
              float r0l = 0.f, r0h = 0.f, r1l = 0.f, r1h = 0.f;
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  const int k = hf * 64 + 2 * c;
                  const uint64_t e = fma2(f32x2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), scl, nm);
                  const float p0 = fast_exp2(f32x2_lo(e)), p1 = fast_exp2(f32x2_hi(e));
                  pk[c] = pack_bf16x2(p0, p1);
                  if (c & 1) {
                    add2(s1, f32x2(p0, p1));
                    add_bf16x2_to_f32(r1l, r1h, pk[c]);
                  } else {
                    add2(s0, f32x2(p0, p1));
                    add_bf16x2_to_f32(r0l, r0h, pk[c]);
                  }
                }
                tmem_st32(tS + hf * 32, pk);
              }
              add2(s0, s1);
              ts = f32x2_lo(s0) + f32x2_hi(s0);
              tr = (r0l + r1l) + (r0h + r1h);
            };
            // First with the row's current maximum; if some row's probabilities then sum
            // to more than 2^8 (a logit well above m), the warp takes the exact maximum,
            // rescales O and recomputes P over what it wrote. A piece's first step
            // always takes the maximum.
            float ts, tr;
            bool exact = j == 0;
#pragma unroll 1
            for (;;) {
              if (exact) {
                float a[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] = __uint_as_float(x[i]);
#pragma unroll
                for (int c = 8; c < kKeys; c += 16)
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    a[i] = fmax3(a[i], __uint_as_float(x[c + i]), __uint_as_float(x[c + 8 + i]));
                const float mx = fmax3(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
                const float m_new = fmaxf(m, mx * p.scale_log2);  // -inf stays -inf
                if (j > 0) {
                  // O holds every step up to j - 1 once that P.V is complete
                  if (!__all_sync(0xffffffffu, wait_(bar(kBarO + (b ^ 1)), ((gk - 1) >> 1) & 1, abort))) {
                    good = false;
                    break;
                  }
                  tc_fence_after();
                  const float alpha = fast_exp2(m - m_new);
#pragma unroll 1
                  for (int c = 0; c < kD; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                    tmem_st32(tO + c, o);
                  }
                  tmem_wait_st();
                  l *= alpha;
                  lr *= alpha;
                }
                m = m_new;
              }
              exps(m, ts, tr);
              if (exact || !__any_sync(0xffffffffu, live && !(ts <= kLazyBound))) break;
              exact = true;
            }
            if (!good) break;
            l += ts;
            lr += tr;
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarP + b));
        }
        if (!good) break;
        const int last = gk - 1;
        if (!any) continue;
        if (!__all_sync(0xffffffffu, wait_(bar(kBarO + (last & 1)), (last >> 1) & 1, abort))) {
          good = false;
          break;
        }
        tc_fence_after();
        const int n_valid = min(32, (d.n_tok << p.gqa_log2) - quad * 32);
        if (d.slot < 0) {
          const float inv = 1.f / lr;
          const int64_t head0 = static_cast<int64_t>(d.head) << p.gqa_log2;
          auto to = [&](int i, int half) {
            const int ri = quad * 32 + i;
            const int64_t at = static_cast<int64_t>(d.row + (ri >> p.gqa_log2)) * p.num_q_heads + head0 +
                               (ri & ((1 << p.gqa_log2) - 1));
            return reinterpret_cast<uint8_t *>(p.out + at * kD + half * 64);
          };
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            uint32_t o[64], w[32];
            tmem_ld32(tO + half * 64, *reinterpret_cast<uint32_t(*)[32]>(&o[0]));
            tmem_ld32(tO + half * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&o[32]));
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              w[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
            store_rows(w, scr, n_valid, lane, [&](int i) { return to(i, half); });
          }
          if (live && p.lse != nullptr)
            p.lse[static_cast<int64_t>(d.row + tok) * p.num_q_heads + head0 + h] = (m + log2f(l)) * kLn2;
        } else {
          float *dst = p.ws_o + (static_cast<int64_t>(d.slot) * kRows + quad * 32) * kD;
#pragma unroll 1
          for (int c = 0; c < kD; c += 32) {
            uint32_t o[32];
            tmem_ld32(tO + c, o);
            tmem_wait_ld();
            store_rows(o, scr, n_valid, lane, [&](int i) { return reinterpret_cast<uint8_t *>(dst + i * kD + c); });
          }
          if (live) p.ws_ml[static_cast<int64_t>(d.slot) * kRows + r] = make_float4(m, l, lr, 0.f);
        }
      }
      if (!good && lane == 0) fail();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the pieces of the tiles that range boundaries cut: CTA (c, y) takes rows
// kJoinRows y .. of the tile that boundary c + 1 is the first to cut, a warp a row,
// four dims a lane. Piece x > 0 is in slot 2 (cta of piece 0 + x).
constexpr int kJoinWarps = 4;
constexpr int kJoinRows = 8;
constexpr int kJoinLoads = 8;  // pieces whose outputs are in flight

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
    auto at = [&](int x) {
      const int64_t slot = x == 0 ? cut.slot0 : 2 * (static_cast<int64_t>(cut.slot0 >> 1) + x);
      return slot * kRows + r;
    };
    float M = kFloor;
    for (int x = lane; x < cut.pieces; x += 32) M = fmaxf(M, p.ws_ml[at(x)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float l = 0.f, lr = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int base = 0; base < cut.pieces; base += 32) {
      float f = 0.f;
      if (base + lane < cut.pieces) {
        const float4 ml = p.ws_ml[at(base + lane)];
        // a piece that the row sees nothing of has a sum of 0 and an output of zeros
        f = fast_exp2(ml.x - M);
        l = fmaf(ml.y, f, l);
        lr = fmaf(ml.z, f, lr);
      }
      const int n = min(32, cut.pieces - base);
      for (int x0 = 0; x0 < n; x0 += kJoinLoads) {
        float4 o[kJoinLoads];
#pragma unroll
        for (int x = 0; x < kJoinLoads; ++x)
          o[x] = x0 + x < n ? reinterpret_cast<const float4 *>(p.ws_o + at(base + x0 + x) * kD)[lane]
                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < kJoinLoads; ++x) {
          const float fx = __shfl_sync(0xffffffffu, f, (x0 + x) & 31);
          acc[0] = fmaf(o[x].x, fx, acc[0]);
          acc[1] = fmaf(o[x].y, fx, acc[1]);
          acc[2] = fmaf(o[x].z, fx, acc[2]);
          acc[3] = fmaf(o[x].w, fx, acc[3]);
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, off);
      lr += __shfl_xor_sync(0xffffffffu, lr, off);
    }
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
  const int tiles = (a.max_seqlen_q - 1) / tokens + 1;  // row tiles of the longest segment
  p.lanes_log2 = tiles >= 32 ? 5 : log2_of(tiles);
  p.window = a.window;
  p.sinks = a.sinks;
  p.box_rows = prefill_box_rows(a.block_size);
  p.flip = a.scale_log2 < 0.f ? 1u : 0u;
  // a factor of zero would make NaN of masked logits: the smallest normal number
  // gives the same weights to any logits below 10^30
  p.scale_log2 = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);
  // the limit is the kernel's, not the call's: another host thread may be between its
  // own two calls here, so it is always set to the most that any call wants
  cudaError_t e = cudaFuncSetAttribute(chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem_bytes(kChunkMaxSeqs));
  if (e != cudaSuccess) return e;
  e = launch_pdl(chunk_kernel, dim3(a.num_sms), dim3(kThreads), smem_bytes(a.num_seqs), stream, q_map, k_map, v_map, p);
  if (e != cudaSuccess || a.num_sms < 2) return e;
  // tiles of one step have no boundary inside
  if (tiles == 1 && a.max_context_len <= kKeys) return cudaSuccess;
  const int rows = static_cast<int>(std::min<int64_t>(kRows, static_cast<int64_t>(a.max_seqlen_q) << p.gqa_log2));
  return launch_pdl(chunk_join_kernel, dim3(a.num_sms - 1, (rows + kJoinRows - 1) / kJoinRows),
                    dim3(kJoinWarps * 32), 0, stream, p);
}

cudaError_t chunk_error_word(uint32_t **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_chunk_errors);
}

}  // namespace pkv
