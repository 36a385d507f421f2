/*
 * pkv.h -- paged-KV-cache attention for GB300 (sm_103a): the C ABI of libpkv.so.
 *
 * The pages describe a nano-vLLM style serving engine whose scheduler asks a
 * KV block manager for cache blocks ("How lunaryes/nano-vllm works",
 * Connections: "Scheduler -> KV Block Manager: allocates cached blocks") and
 * whose model runner sets an execution context before running the Qwen3
 * layers (same page, Connections: "Model Runner -> Execution Context"). This
 * library is the data-parallel hot path inside those layers: writing each
 * step's new K/V rows into the paged cache (the "paged KV cache" of the
 * nano-vllm-rs README, "GGUF Models"), q=1 decode attention (the q=1 decode
 * kernel of the nano-vllm-sansho README, "Sansho Serving Roofline Anchors") and
 * varlen causal prefill attention that also serves prompts whose leading blocks
 * are already cached (prefix caching: nano-vllm-sansho README, "Key Features").
 * Its arguments are that execution context: slot mapping, block tables,
 * context lengths, cumulative sequence lengths.
 *
 * Conventions shared by every call
 * --------------------------------
 * Layout. bf16 everywhere for tensors; row-major, contiguous.
 *   new K/V rows   k, v        [T, H_kv, D]
 *   cache          k_cache     [num_blocks, block_size, H_kv, D]  (same for v_cache)
 *   queries        q           [T_q, H_q, D] (prefill) or [S, H_q, D] (decode)
 *   outputs        out         like q; lse float32 [rows, H_q]
 *   block tables   int32       [S, max_blocks_per_seq]; entry -1 = no block
 * Slot of token at position p of sequence s:
 *   block_tables[s][p / block_size] * block_size + p % block_size.
 * Query head h reads KV head h / (H_q / H_kv).
 * D must be 128, block_size a multiple of 16, H_q / H_kv in {1, 2, 4}.
 *
 * Memory and ownership. Every pointer is caller-owned device memory (except
 * the host pointer flags_out); the library allocates and frees nothing, keeps
 * no per-call state, and returns before the kernels finish. Device buffers
 * must be 16-byte aligned. What a call writes (outputs, workspace) must not
 * overlap its inputs or itself, except where the call says that it may.
 *
 * Streams. `stream` is a cudaStream_t passed as void* (NULL = the legacy
 * default stream). Every call only enqueues work on that stream and never
 * synchronises, so it may be captured into a CUDA graph, except
 * pkv_check_device_errors, which synchronises the stream.
 *
 * Errors. Arguments the host can see are checked before anything is enqueued:
 * PKV_ERR_INVALID_ARG (null pointer, negative size, inconsistent shape),
 * PKV_ERR_UNSUPPORTED (a shape this library has no kernel for),
 * PKV_ERR_WORKSPACE_TOO_SMALL. A failing CUDA call gives PKV_ERR_CUDA and
 * pkv_last_cuda_error() names it (thread-local). Values that live on the device
 * (slots, table entries, lengths) are checked by the kernels: an invalid one
 * skips the access it would have made and raises a bit of the device error
 * word (PKV_DEVERR_*), read with pkv_check_device_errors (which blocks) or
 * pkv_read_device_errors_async (which does not). Outputs that depend on an
 * invalid value are undefined; nothing outside the given buffers is touched.
 *
 * Timeouts are sticky. Every wait inside a kernel is bounded; a kernel that
 * gives up raises PKV_DEVERR_TIMEOUT. From then on every later call on that
 * device that runs the kernel that gave up - bf16 decode (fused store, sinks and
 * accumulated weights included), prefill, or chunks - returns PKV_OK but
 * skips all its work, leaving its outputs (and, for the fused call, the cache)
 * untouched, until the word is cleared by pkv_check_device_errors. (The bit
 * raised by pkv_raise_device_errors stops all of them.) An engine
 * that runs these calls inside CUDA graphs and never synchronises should
 * append pkv_read_device_errors_async to its step and act on the bit.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1,
  PKV_ERR_UNSUPPORTED = 2,
  PKV_ERR_WORKSPACE_TOO_SMALL = 3,
  PKV_ERR_CUDA = 4,
  PKV_ERR_OUT_OF_BLOCKS = 5 /* the block manager has too few free blocks (pkv_blocks.h) */
} pkv_status;

/* Bits of the device error word. */
#define PKV_DEVERR_SLOT 0x1u      /* a slot outside [-1, num_blocks * block_size)      */
#define PKV_DEVERR_BLOCK 0x2u     /* a needed block-table entry outside [0, num_blocks) */
#define PKV_DEVERR_CONTEXT 0x4u   /* context_len <= 0, above max_context_len or above
                                     max_blocks_per_seq * block_size                  */
#define PKV_DEVERR_SEQLENS 0x8u   /* cu_seqlens inconsistent with the host-side maxima  */
#define PKV_DEVERR_TIMEOUT 0x10u  /* a kernel gave up waiting on one of its barriers    */

/*
 * Launch mode, process-wide: with enabled != 0 (the default) every kernel is
 * launched with programmatic stream serialization (programmatic dependent
 * launch), so it may start while the previous kernel on the stream finishes;
 * each kernel still waits for that kernel's completion before it reads or
 * writes global memory, so results and ordering are unchanged. 0 launches
 * them the classic way.
 */
void pkv_set_programmatic_launch(int32_t enabled);

/* Name of a status code (static string). */
const char *pkv_status_string(pkv_status status);

/* The CUDA error string of this thread's last PKV_ERR_CUDA, or "" if none. */
const char *pkv_last_cuda_error(void);

/*
 * KV store: the slot-mapping scatter of the new tokens' K/V rows into the
 * paged cache (the engine's KV block manager hands out the cache slots: "How
 * lunaryes/nano-vllm works", Components: KV Block Manager, and Connections:
 * "Scheduler -> KV Block Manager: allocates cached blocks"; the cache is the
 * paged KV cache of the nano-vllm-rs README, "GGUF Models").
 * k_cache[slot_mapping[t]] = k[t] and v_cache[slot_mapping[t]] = v[t]
 * for every t with slot_mapping[t] >= 0 (all H_kv * D values of the row, bit
 * for bit); -1 skips the token (the block manager gave it no slot, as for
 * tokens of a cached prefix). Two tokens with the same non-negative slot in one
 * call race. A slot below -1 or at/above num_blocks * block_size is skipped
 * and raises PKV_DEVERR_SLOT.
 *   k, v           device bf16 [num_tokens, num_kv_heads, head_dim]
 *   k_cache,v_cache device bf16 [num_blocks, block_size, num_kv_heads, head_dim]
 *   slot_mapping   device int32 [num_tokens]
 * num_tokens == 0 is a no-op. Here head_dim may be any value with
 * num_kv_heads * head_dim * 2 a multiple of 16 bytes.
 */
pkv_status pkv_kv_store(const void *k, const void *v, void *k_cache, void *v_cache,
                        const int32_t *slot_mapping, int32_t num_tokens,
                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                        int64_t num_blocks, void *stream);

/*
 * Bytes of device workspace that pkv_paged_decode_attn needs for these sizes on
 * the current device (0 on invalid sizes or without a device). The workspace
 * holds the partial results of the (sequence, KV head) pairs whose keys are
 * split between CTAs; its size depends on the heads and on the device's SM
 * count, not on context length or on the number of sequences. The caller
 * allocates it once and may reuse it for every call with sizes no larger than
 * these; it needs no initialisation. Calls that share a workspace must be
 * ordered (same stream).
 */
size_t pkv_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim, int32_t max_context_len);

/*
 * Paged decode attention, one query token per sequence (q=1 decode).
 * For sequence s, query head h and KV head g = h / (H_q / H_kv):
 *   z_p   = scale * <q[s,h], k_cache[slot(s, p), g]>   for p < context_lens[s]
 *   out   = sum_p exp(z_p - M) v_cache[slot(s,p), g] / sum_p exp(z_p - M)
 *   lse   = M + ln sum_p exp(z_p - M),   M = max_p z_p      (natural log)
 * The query's own K/V must already be in the cache (store first, then attend,
 * on the same stream). Split-K over the context ("flash decoding"): partial
 * results go to the workspace and a second kernel merges them.
 *   q              device bf16 [num_seqs, num_q_heads, head_dim]
 *   block_tables   device int32 [num_seqs, max_blocks_per_seq]
 *   context_lens   device int32 [num_seqs], each in [1, max_context_len]
 *   max_context_len host int: an upper bound of context_lens (sizes the grid)
 *   scale          the logit scale (usually 1/sqrt(head_dim))
 *   sliding_window 0: every key; W > 0: only the last W keys up to the
 *                  query's own, p >= context_lens[s] - W (sliding-window
 *                  attention: the SWA-256 serving target of the
 *                  nano-vllm-sansho README, "Sansho Fork"); blocks wholly
 *                  before the window are not read. Negative: PKV_ERR_INVALID_ARG.
 *   out            device bf16 [num_seqs, num_q_heads, head_dim]
 *   lse            device float32 [num_seqs, num_q_heads], or NULL
 *   workspace      device, >= pkv_decode_workspace_size(...) bytes, 16-byte aligned
 * num_seqs is at most 1024.
 * Rows whose context_len is invalid raise PKV_DEVERR_CONTEXT and are not written.
 */
pkv_status pkv_paged_decode_attn(const void *q, const void *k_cache, const void *v_cache,
                                 const int32_t *block_tables, int32_t max_blocks_per_seq,
                                 const int32_t *context_lens, int32_t max_context_len,
                                 int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                 float scale, int32_t sliding_window, void *out, float *lse,
                                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * Fused decode step: the KV store of each sequence's new token and paged decode
 * attention in one kernel (the engine's per-layer decode work, one launch).
 * Equivalent to pkv_kv_store(k_new, v_new, k_cache, v_cache, slot_mapping,
 * num_seqs, ...) followed by pkv_paged_decode_attn(...) on the same stream:
 * the new token of sequence s is the one at logical position
 * context_lens[s] - 1, its K/V rows k_new[s], v_new[s] are written to
 * slot_mapping[s] (-1: not written) and used as that key by the attention.
 *   k_new, v_new   device bf16 [num_seqs, num_kv_heads, head_dim]
 *   slot_mapping   device int32 [num_seqs]
 * Other arguments, the workspace and the error behaviour are those of
 * pkv_paged_decode_attn; an invalid slot raises PKV_DEVERR_SLOT (not written;
 * the attention still uses the new rows).
 *   flags          0, or PKV_DECODE_STABLE_INPUTS: the caller guarantees that
 *                  k_cache and v_cache (except the rows this call stores),
 *                  block_tables and context_lens are written neither by the
 *                  kernel enqueued just before this call nor by any earlier one
 *                  that may still be running (with programmatic dependent
 *                  launch a kernel of this library lets the next one start
 *                  before it ends). The call then reads them, and starts
 *                  streaming K/V, while the previous kernel finishes; q,
 *                  k_new, v_new and slot_mapping are still read only after it
 *                  has completed. This holds in a decode step whose tables and
 *                  lengths are set before the step and whose layers each have
 *                  their own caches.
 */
#define PKV_DECODE_STABLE_INPUTS 0x1u
pkv_status pkv_paged_decode_attn_store(const void *k_new, const void *v_new,
                                       const int32_t *slot_mapping, const void *q,
                                       void *k_cache, void *v_cache,
                                       const int32_t *block_tables, int32_t max_blocks_per_seq,
                                       const int32_t *context_lens, int32_t max_context_len,
                                       int32_t num_seqs, int32_t num_q_heads,
                                       int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                       int64_t num_blocks, float scale, int32_t sliding_window,
                                       void *out, float *lse, void *workspace,
                                       size_t workspace_bytes, uint32_t flags, void *stream);

/*
 * Tuning knob of the decode launch, process-wide (not thread-safe against
 * concurrent launches): ctas = number of persistent CTAs (0 = one per SM, the
 * default); variant = launch shape (0 = default: head groups of 8 KV heads and
 * three TMA stages per CTA when the KV heads split into groups of 8, else the
 * shape of variant 2; 1 = head groups of up to 8 KV heads, two stages; 2 =
 * head groups of up to 4 KV heads, two stages, two CTAs per SM). Results do
 * not depend on either, beyond rounding.
 * A non-default ctas changes pkv_decode_workspace_size.
 */
void pkv_decode_set_config(int32_t ctas, int32_t variant);

/*
 * Decode attention for callers that cannot allocate device memory.
 * (An addition of this library: the pages have no counterpart.)
 * Some callers of decode cannot call cudaMalloc where they run: a plugin inside
 * a host framework whose allocator owns the whole device pool, a deployment
 * that forbids dynamic allocation after start-up, a latency-critical loop where
 * an allocation may synchronise the device. This call computes exactly what
 * pkv_paged_decode_attn computes, with the same arguments except the
 * workspace: its scratch is a static device array of
 * PKV_DECODE_NOALLOC_SCRATCH_BYTES inside libpkv.so, present on every GPU that
 * loads the library until the process exits. It calls no cudaMalloc, cudaFree
 * or other allocator.
 *   - Sizes whose pkv_decode_workspace_size exceeds that limit are rejected with
 *     PKV_ERR_WORKSPACE_TOO_SMALL before anything is enqueued.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture. The address is kept for the life of the
 *     process: a cudaDeviceReset of that device afterwards is not supported.
 *   - Without a usable device the call returns PKV_ERR_CUDA (with
 *     pkv_last_cuda_error set); sizes that no decode call accepts return
 *     PKV_ERR_INVALID_ARG.
 *   - Every call on a device shares that device's one array, which keeps the
 *     last call's contents; nothing in it needs to start at zero. Calls that
 *     can overlap on the GPU (for example on two streams with no ordering
 *     between them) race on the array: the caller must order them.
 */
#define PKV_DECODE_NOALLOC_SCRATCH_BYTES (16u << 20)
pkv_status pkv_paged_decode_attn_noalloc(const void *q, const void *k_cache, const void *v_cache,
                                         const int32_t *block_tables,
                                         int32_t max_blocks_per_seq,
                                         const int32_t *context_lens, int32_t max_context_len,
                                         int32_t num_seqs, int32_t num_q_heads,
                                         int32_t num_kv_heads, int32_t head_dim,
                                         int32_t block_size, int64_t num_blocks, float scale,
                                         int32_t sliding_window, void *out, float *lse,
                                         void *stream);

/*
 * Decode attention under a sliding window with first tokens that stay visible
 * ("sinks"): pkv_paged_decode_attn, or with new rows pkv_paged_decode_attn_store,
 * where sequence s attends to the keys
 *   p < num_sinks  or  p >= context_lens[s] - sliding_window.
 * Streams longer than their window keep the statistics of their softmax this way.
 * Blocks that hold neither kind of key are not read: their table entries may be
 * -1, their memory another sequence's. Keys that are not attended to may hold
 * anything, NaN and infinities included.
 *   k_new, v_new, slot_mapping  as in pkv_paged_decode_attn_store, or all NULL: no store
 *   num_sinks  >= 0 (negative: PKV_ERR_INVALID_ARG); without a window every key is
 *              attended to, as in the two calls above
 *   flags      0, or with new rows PKV_DECODE_STABLE_INPUTS
 * Other arguments, the workspace and the errors are theirs.
 */
pkv_status pkv_paged_decode_attn_sinks(const void *k_new, const void *v_new,
                                       const int32_t *slot_mapping, const void *q, void *k_cache,
                                       void *v_cache, const int32_t *block_tables,
                                       int32_t max_blocks_per_seq, const int32_t *context_lens,
                                       int32_t max_context_len, int32_t num_seqs,
                                       int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                       int32_t block_size, int64_t num_blocks, float scale,
                                       int32_t sliding_window, int32_t num_sinks, void *out,
                                       float *lse, void *workspace, size_t workspace_bytes,
                                       uint32_t flags, void *stream);

/*
 * Bytes of device workspace that pkv_paged_prefill_attn needs (currently 0 for
 * every size: the prefill kernel keeps all its state on chip).
 */
size_t pkv_prefill_workspace_size(int32_t num_seqs, int32_t max_seqlen_q);

/*
 * Varlen causal prefill attention over the paged cache, with prefix caching
 * (nano-vllm-sansho README, "Key Features": prefix caching; "How
 * lunaryes/nano-vllm works", Connections: the block manager allocates cached
 * blocks, which a later prompt with the same leading tokens reads instead of
 * recomputing them).
 * Segment s has Lq = cu_seqlens_q[s+1] - cu_seqlens_q[s] query tokens
 * (rows cu_seqlens_q[s] .. of q) and Lk = cu_seqlens_k[s+1] - cu_seqlens_k[s]
 * keys, read through block_tables[s]; the queries are the last Lq of the Lk
 * positions, so query i sees keys p <= Lk - Lq + i (bottom-right causal;
 * Lq == Lk is plain causal attention, Lq < Lk serves a prompt whose first
 * Lk - Lq tokens are cached). Keys are always read from the cache: store the
 * prompt's new K/V first, on the same stream. Lq == 0 writes nothing.
 * Output and lse as in decode, for every query row. With sliding_window
 * W > 0 query i sees only keys Lk - Lq + i - W < p <= Lk - Lq + i (the last W
 * positions up to its own); KV tiles wholly before a CTA's windows are not
 * read. Negative: PKV_ERR_INVALID_ARG.
 *   q              device bf16 [total_q, num_q_heads, head_dim]
 *   cu_seqlens_q/k device int32 [num_seqs + 1], non-decreasing, from 0
 *   max_seqlen_q/k host ints: upper bounds of Lq and Lk (size the grid)
 *   out            device bf16 [total_q, num_q_heads, head_dim]
 *   lse            device float32 [total_q, num_q_heads], or NULL
 *   workspace      may be NULL when pkv_prefill_workspace_size returns 0
 * Segments with Lq > Lk, Lq > max_seqlen_q, Lk > max_seqlen_k or Lk beyond
 * the table raise PKV_DEVERR_SEQLENS and are not written.
 */
pkv_status pkv_paged_prefill_attn(const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                  const int32_t *block_tables, int32_t max_blocks_per_seq,
                                  int32_t num_seqs, int32_t total_q, int32_t max_seqlen_q,
                                  int32_t max_seqlen_k, int32_t num_q_heads,
                                  int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                  int64_t num_blocks, float scale, int32_t sliding_window,
                                  void *out, float *lse, void *workspace, size_t workspace_bytes,
                                  void *stream);

/*
 * Attention of a chunk of new tokens of each sequence over the paged cache: the
 * next tokens of a prompt that is taken in pieces, drafted tokens to be checked, the
 * single tokens of sequences that decode beside them, in one call. Segment s has Lq =
 * cu_seqlens_q[s+1] - cu_seqlens_q[s] query tokens, the last Lq of the sequence's
 * context_lens[s] positions, whose rows are in the cache (store them first). Query i,
 * at position p_i = context_lens[s] - Lq + i, sees the keys
 *   p <= p_i,  and with a window  p > p_i - sliding_window  or  p < num_sinks.
 * Output and lse as in decode, for every query row, but for the weights: as in prefill
 * they are rounded to bf16 for the tensor cores, and the output is divided by the sum of
 * the rounded ones (the lse is not), which leaves it within 2^-7 of the weighted mean of
 * |v|. A batch of single tokens alone keeps fp32 weights in pkv_paged_decode_attn[_sinks].
 * A pkv_paged_prefill_attn with context lengths in place of cu_seqlens_k, whose keys are
 * shared out over all SMs and joined by a second kernel. Only a call without a window whose
 * total_q and max_seqlen_q say that its segments are long and about as long as each other
 * runs as prefill does, each 128 rows of two heads passing their keys on one SM. These host
 * values choose, not the lengths on the device: a graph captured with wide bounds and
 * replayed with a few tokens over long contexts stays there, at several times the chunk
 * kernel's time. Capture such replays on their own, with tight bounds.
 *   q, out       device bf16 [total_q, num_q_heads, head_dim]
 *   lse          device float32 [total_q, num_q_heads], or NULL
 *   cu_seqlens_q device int32 [num_seqs + 1], non-decreasing, from 0; rows of q and
 *                out past its last value are not touched
 *   context_lens device int32 [num_seqs]; not looked at where Lq == 0
 *   max_seqlen_q, max_context_len  host ints: upper bounds, the latter at most 2^30, the
 *                former at most the latter (else PKV_ERR_INVALID_ARG)
 *   workspace    device, >= pkv_chunk_workspace_size(...) bytes, 16-byte aligned; needs
 *                no initialisation; calls that share one must be ordered (same stream)
 * num_seqs is at most 1024. Blocks with no key that a query of the segment sees are not
 * read (their entries may be -1), and keys that none sees may hold anything; keys that
 * some query of a segment sees must be finite, or that segment's rows may all be
 * NaN. Segments with Lq < 0, Lq > max_seqlen_q, Lq > context_lens[s], rows past
 * total_q, or context_lens[s] above max_context_len or past the table raise
 * PKV_DEVERR_SEQLENS and are not written; an invalid table entry raises
 * PKV_DEVERR_BLOCK and makes its segment's rows undefined. After a PKV_DEVERR_TIMEOUT
 * of the kernel that it runs (see above) the call does nothing.
 */
size_t pkv_chunk_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                int32_t head_dim);
pkv_status pkv_paged_chunk_attn(const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *cu_seqlens_q, const int32_t *context_lens,
                                const int32_t *block_tables, int32_t max_blocks_per_seq,
                                int32_t num_seqs, int32_t total_q, int32_t max_seqlen_q,
                                int32_t max_context_len, int32_t num_q_heads,
                                int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                int64_t num_blocks, float scale, int32_t sliding_window,
                                int32_t num_sinks, void *out, float *lse, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * A cache held in 4 bits
 * ----------------------
 * The same paged cache with each K and V row quantised: codes of 4 bits and a
 * (scale, offset) pair for every group of group_size (32, 64 or 128) dims.
 *   k_codes, v_codes    uint8 [num_blocks, H_kv, block_size, 64]: byte j of a row
 *                       holds dim 2j in its low nibble and dim 2j + 1 in its high one
 *   k_params, v_params  bf16 [num_blocks, H_kv, block_size, 128 / group_size, 2]
 * A row takes 64 + 512 / group_size bytes (80, 72 or 68) instead of 256. All
 * four arrays are 16-byte aligned and contiguous. Within a block the rows of a
 * head are contiguous (not those of a token, as in the bf16 cache), which is how
 * the decode kernel reads them; slots and block tables mean the same.
 *
 * Values. Code n of a group with (scale, offset) stands for
 *   bf16(scale * (16 + n) + offset),  rounded once, to nearest even.
 * Attention over the cache is attention over exactly these bf16 values.
 * Quantisation of a group with smallest value lo and largest value hi, each
 * operation rounded to the type it is written with:
 *   scale  = bf16(fp32(hi - lo) * fp32(1/15)), or 0 if that product is below 2^-100
 *   offset = bf16(lo - 16 scale)
 *   n      = clamp(floor(fp32(x - offset) / scale + 1/2) - 16, 0, 15), or 0 if scale = 0
 * A value comes back within half a scale, plus the roundings of the parameters
 * and of the result. A group that holds a NaN or an infinity, or whose range
 * makes the offset overflow, gets scale 0 and offset NaN: it reads back as NaN.
 */

/*
 * Quantise the new tokens' K/V rows into their slots: pkv_kv_store for a 4-bit
 * cache, with the same slot_mapping semantics and errors (-1 skips the token;
 * another value outside the pool is skipped and raises PKV_DEVERR_SLOT; two
 * tokens with the same slot race). num_tokens * num_kv_heads must be below 2^31.
 *   k, v  device bf16 [num_tokens, num_kv_heads, 128]
 */
pkv_status pkv_kv_store_q4(const void *k, const void *v, void *k_codes, void *k_params,
                           void *v_codes, void *v_params, const int32_t *slot_mapping,
                           int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                           int32_t group_size, int32_t block_size, int64_t num_blocks,
                           void *stream);

/*
 * Read rows back as bf16: k[t], v[t] = the values that the rows at slots[t]
 * stand for. A slot may appear any number of times; the rows of slot -1, and of
 * a slot outside the pool (which raises PKV_DEVERR_SLOT), become zeros.
 *   slots device int32 [num_tokens]
 *   k, v  device bf16 [num_tokens, num_kv_heads, 128], written
 */
pkv_status pkv_kv_load_q4(const void *k_codes, const void *k_params, const void *v_codes,
                          const void *v_params, const int32_t *slots, void *k, void *v,
                          int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                          int32_t group_size, int32_t block_size, int64_t num_blocks,
                          void *stream);

/*
 * Bytes of device workspace of pkv_paged_decode_attn_q4 (0 on invalid sizes or
 * without a device). with_scores != 0: for calls with key_scores, which keep the
 * logits of the call there (4 bytes per key and query head). A workspace serves
 * every call with these head counts whose num_seqs and max_context_len are no
 * larger; it needs no initialisation; calls that share one must be ordered (same
 * stream, or graphs that never overlap).
 */
size_t pkv_decode_q4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                    int32_t head_dim, int32_t max_context_len,
                                    int32_t with_scores);

/*
 * pkv_paged_decode_attn over a 4-bit cache. Arguments, result, sliding window
 * and device errors are that call's, except:
 *   - H_q / H_kv may be 1, 2, 4 or 8, num_seqs is at most 65535 and
 *     max_context_len at most 2^30 (PKV_ERR_UNSUPPORTED);
 *   - an invalid table entry raises PKV_DEVERR_BLOCK and its keys are left out;
 *   - no wait inside the kernels can run out, so the call takes no notice of
 *     PKV_DEVERR_TIMEOUT (like pkv_kv_store);
 *   - key_scores, if not NULL, accumulates the attention weights:
 *       key_scores[s * score_stride + p] += sum over query heads h of
 *                                           exp(z_hp - lse[s, h])
 *     for every key p that sequence s attended to (those in its window, if
 *     any); other entries keep their values. float32, score_stride >=
 *     max_context_len. The caller sets a sequence's row to zero when it admits
 *     the sequence. The heads are summed in order: the same call (sizes and
 *     inputs) on the same device gives the same bits.
 */
pkv_status pkv_paged_decode_attn_q4(const void *q, const void *k_codes, const void *k_params,
                                    const void *v_codes, const void *v_params,
                                    const int32_t *block_tables, int32_t max_blocks_per_seq,
                                    const int32_t *context_lens, int32_t max_context_len,
                                    int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                    int32_t head_dim, int32_t group_size, int32_t block_size,
                                    int64_t num_blocks, float scale, int32_t sliding_window,
                                    void *out, float *lse, float *key_scores,
                                    int64_t score_stride, void *workspace,
                                    size_t workspace_bytes, void *stream);

/*
 * Bytes of device workspace of pkv_paged_prefill_attn_q4 (0 on invalid sizes or
 * without a device): the call may widen the batch's keys to bf16 there, 512 *
 * num_kv_heads bytes per key and up to 128 keys more per sequence. A workspace
 * serves every call with sizes no larger than these; else conditions as above.
 */
size_t pkv_prefill_q4_workspace_size(int32_t num_seqs, int32_t total_k, int32_t max_seqlen_k,
                                     int32_t num_kv_heads, int32_t head_dim);

/*
 * pkv_paged_prefill_attn over a 4-bit cache: the new tokens attend to the
 * quantised values of the cached prefix and of themselves (store them first).
 * Arguments, result, sliding window, errors and the skip after a timeout are
 * that call's, except:
 *   total_k    host int: an upper bound of cu_seqlens_k[num_seqs]; a segment
 *              that ends past it raises PKV_DEVERR_SEQLENS and is not written
 *   workspace  device, >= pkv_prefill_q4_workspace_size(...) bytes
 * An invalid table entry that a segment's queries see raises PKV_DEVERR_BLOCK; that
 * segment's rows are then undefined (which of the two ways below the call takes
 * decides what stands for the missing keys), the other segments' are not touched
 * by it.
 * num_seqs is at most 65535. With few query tokens over many keys the call runs
 * each row through the decode kernels instead of widening the keys (the same
 * sums in another order); it then takes no notice of PKV_DEVERR_TIMEOUT.
 */
pkv_status pkv_paged_prefill_attn_q4(const void *q, const void *k_codes, const void *k_params,
                                     const void *v_codes, const void *v_params,
                                     const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                     const int32_t *block_tables, int32_t max_blocks_per_seq,
                                     int32_t num_seqs, int32_t total_q, int32_t total_k,
                                     int32_t max_seqlen_q, int32_t max_seqlen_k,
                                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                     int32_t group_size, int32_t block_size, int64_t num_blocks,
                                     float scale, int32_t sliding_window, void *out, float *lse,
                                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * Eviction by accumulated attention weight
 * ----------------------------------------
 * A sequence whose cache has grown past a budget keeps its most recent tokens
 * and, of the older ones, those that have received most attention: decode calls
 * accumulate each key's weight (pkv_paged_decode_attn_scores, or key_scores of
 * pkv_paged_decode_attn_q4), pkv_evict_select chooses the positions, and
 * pkv_evict_compact moves their rows together in order. Afterwards the sequence
 * has new_lens[s] keys, at positions 0 .. new_lens[s] - 1 of the destination
 * table (keys carry their rotary position in their values).
 */

/*
 * pkv_paged_decode_attn that also accumulates the attention weights:
 *   key_scores[s * score_stride + p] += sum over query heads h of exp(z_hp - lse[s, h])
 * for every key p that sequence s attended to; other entries keep their values.
 * The heads are summed in order: the same call (sizes and inputs) on the same
 * device gives the same bits. An invalid table entry raises PKV_DEVERR_BLOCK and its
 * keys are left out, of the attention and of the weights.
 *   key_scores   device float32 [num_seqs, score_stride], not NULL; the caller
 *                sets a sequence's row to zero when it admits the sequence
 *   score_stride >= max_context_len, which is at most 2^30 (PKV_ERR_UNSUPPORTED)
 *   workspace    device, >= pkv_decode_scores_workspace_size(...) bytes: the
 *                decode workspace and the call's logits (4 bytes per key and
 *                query head). Conditions as for the decode workspace, but its
 *                size follows num_seqs and max_context_len.
 * After a timeout (see above) nothing is added.
 */
size_t pkv_decode_scores_workspace_size(int32_t num_seqs, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t max_context_len);
pkv_status pkv_paged_decode_attn_scores(const void *q, const void *k_cache, const void *v_cache,
                                        const int32_t *block_tables, int32_t max_blocks_per_seq,
                                        const int32_t *context_lens, int32_t max_context_len,
                                        int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                        int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                        float scale, int32_t sliding_window, void *out, float *lse,
                                        float *key_scores, int64_t score_stride, void *workspace,
                                        size_t workspace_bytes, void *stream);

/*
 * The positions that stay: of a sequence with ctx = context_lens[s] keys, all if
 * ctx <= budget; else the last `recent` and, of the others, the budget - recent
 * with the highest scores (equal scores: the lowest positions; a NaN counts as
 * lower than any number).
 *   key_scores   device float32 [num_seqs, score_stride], score_stride >= max_context_len
 *   context_lens device int32 [num_seqs], each in [0, max_context_len]
 *   budget       in [1, 2^29] here and below;  recent in [0, budget]
 *   keep         device int32 [num_seqs, budget]: the kept positions in
 *                ascending order, then -1
 *   new_lens     device int32 [num_seqs]: min(ctx, budget)
 * A sequence whose length is invalid raises PKV_DEVERR_CONTEXT and its rows of
 * keep and new_lens are not written: a compaction enqueued behind the call acts on
 * what they held. Set them to -1 beforehand, or use pkv_evict_select_new.
 */
pkv_status pkv_evict_select(const float *key_scores, int64_t score_stride,
                            const int32_t *context_lens, int32_t max_context_len, int32_t num_seqs,
                            int32_t budget, int32_t recent, int32_t *keep, int32_t *new_lens,
                            void *stream);

/*
 * The same into arrays that hold nothing yet: a sequence whose length is invalid
 * raises PKV_DEVERR_CONTEXT and gets -1 in new_lens and in its whole row of keep, a
 * length that pkv_evict_compact refuses.
 */
pkv_status pkv_evict_select_new(const float *key_scores, int64_t score_stride,
                                const int32_t *context_lens, int32_t max_context_len,
                                int32_t num_seqs, int32_t budget, int32_t recent, int32_t *keep,
                                int32_t *new_lens, void *stream);

/*
 * Move the kept rows together: for i < new_lens[s], the K and V rows at position
 * i of dst_tables[s] become those at position keep[s][i] of src_tables[s], in
 * every head. keep must be strictly ascending, as pkv_evict_select writes it.
 *   src_tables  device int32 [num_seqs, src_max_blocks]
 *   dst_tables  device int32 [num_seqs, dst_max_blocks]. Each entry used is
 *               either the source's entry at the same index, if no other
 *               sequence of the call reads that block (compaction in place), or
 *               a block that no source table of the call names. Equal tables
 *               compact every sequence in place; sequences that share blocks
 *               with others need fresh ones (pkv_bm_evict_sequences makes
 *               such rows). Nothing else is written.
 *   key_scores  device float32 [num_seqs, score_stride], or NULL (both):
 *   dst_key_scores  dst_key_scores[s * dst_score_stride + i] =
 *               key_scores[s * score_stride + keep[s][i]], and the entries from
 *               new_lens[s] to dst_score_stride - 1 become 0, so that tokens
 *               appended next start from zero. May be the same array (then with
 *               the same stride), or must not overlap.
 * A new_lens[s] outside [0, budget], past dst_tables or past dst_score_stride
 * raises PKV_DEVERR_CONTEXT and nothing of that sequence moves; a position
 * outside a table raises PKV_DEVERR_CONTEXT and an invalid table entry
 * PKV_DEVERR_BLOCK, and that row does not move. num_seqs is at most 65535;
 * head_dim 128; block_size any positive number. Here and in the selections
 * num_seqs == 0 is a no-op.
 */
pkv_status pkv_evict_compact(void *k_cache, void *v_cache, const int32_t *src_tables,
                             int32_t src_max_blocks, const int32_t *dst_tables,
                             int32_t dst_max_blocks, const int32_t *keep, int32_t budget,
                             const int32_t *new_lens, int32_t num_seqs, int32_t num_kv_heads,
                             int32_t head_dim, int32_t block_size, int64_t num_blocks,
                             const float *key_scores, int64_t score_stride, float *dst_key_scores,
                             int64_t dst_score_stride, void *stream);

/* The same for a 4-bit cache: codes and parameters move, bit for bit. */
pkv_status pkv_evict_compact_q4(void *k_codes, void *k_params, void *v_codes, void *v_params,
                                const int32_t *src_tables, int32_t src_max_blocks,
                                const int32_t *dst_tables, int32_t dst_max_blocks,
                                const int32_t *keep, int32_t budget, const int32_t *new_lens,
                                int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim,
                                int32_t group_size, int32_t block_size, int64_t num_blocks,
                                const float *key_scores, int64_t score_stride,
                                float *dst_key_scores, int64_t dst_score_stride, void *stream);

/*
 * Queries and keys on their way to attention
 * ------------------------------------------
 * The step of a layer between its projections and its attention: each head's
 * row x of 128 values is normed and rotated by its token's position,
 *   y = w x / sqrt(mean(x^2) + eps),
 *   (y_a, y_b) -> magnitude (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
 * for the pairs (a, b) of the first rotary_dim dims and the angle t = position
 * * frequency of the pair; the other dims stay y. Computed in fp32 and rounded
 * once, to bf16. (Sums of squares are fp32 too: values beyond some 2^60 overflow
 * them, and their row comes out as zeros.) The angle is off by some 2^-26 of a turn,
 * as fp32 holds it modulo a turn, whatever the position, and by |position| * frequency
 * * 2^-54 of a turn, as 64 bits hold the frequency.
 */

/*
 * A rotation, in host memory: filled by one of the two calls below, then passed
 * to any number of calls, which copy it. rotary_dim is 0 (none) to 128, a
 * multiple of 8. The pairs are (i, i + rotary_dim / 2), or with interleaved != 0
 * (2 i, 2 i + 1).
 */
typedef struct {
  int32_t rotary_dim, interleaved;
  float magnitude;
  int32_t reserved;
  uint64_t turns[64]; /* of each pair: frequency / (2 pi), times 2^64, modulo 2^64 */
} pkv_rope;

/*
 * frequency_i = base^(-2 i / rotary_dim), base > 1, for i < rotary_dim / 2, then
 *   PKV_ROPE_PLAIN   as it is
 *   PKV_ROPE_LINEAR  divided by factor
 *   PKV_ROPE_NTK     with base * factor^(rotary_dim / (rotary_dim - 2)) for base
 *   PKV_ROPE_YARN    f (1 - r) + r f / factor with the ramp r = clamp((i - lo) /
 *                    max(hi - lo, 0.001), 0, 1), lo = max(floor(d(beta_fast)), 0),
 *                    hi = min(ceil(d(beta_slow)), rotary_dim - 1), d(b) = rotary_dim
 *                    ln(original_positions / (2 pi b)) / (2 ln base); and magnitude
 *                    0.1 ln(factor) + 1 (otherwise 1; factor >= 1 here)
 * factor > 0 (not read by PKV_ROPE_PLAIN); original_positions > 0 and beta_fast >=
 * beta_slow > 0 are read by PKV_ROPE_YARN only. Frequencies that no 64-bit number
 * holds, and other values outside these ranges, are PKV_ERR_INVALID_ARG; a rotary_dim
 * outside them is PKV_ERR_UNSUPPORTED. Nothing is written then.
 */
#define PKV_ROPE_PLAIN 0
#define PKV_ROPE_LINEAR 1
#define PKV_ROPE_NTK 2
#define PKV_ROPE_YARN 3
pkv_status pkv_rope_init(pkv_rope *rope, int32_t rotary_dim, int32_t interleaved, double base,
                         int32_t scaling, double factor, int32_t original_positions,
                         double beta_fast, double beta_slow);

/* The same from the frequencies themselves (radians a position, host [rotary_dim / 2]). */
pkv_status pkv_rope_init_frequencies(pkv_rope *rope, int32_t rotary_dim, int32_t interleaved,
                                     const double *frequencies, float magnitude);

/*
 * Norm and rotate the rows of q and k, in one pass over them.
 *   q, k       device bf16: head h of token t is the 128 values at element
 *              t * stride + h * 128, so that both may be parts of one packed
 *              projection [num_tokens, (H_q + 2 H_kv) * 128]. Strides count elements
 *              and are multiples of 8; 0 heads: NULL, and nothing is done for it
 *   q_weight, k_weight  device bf16 [128], or NULL: that tensor is not normed
 *   eps        finite, >= 0
 *   rope       host, or NULL: no rotation
 *   positions  device int32 [num_tokens], any values; may be NULL without a rotation
 *   q_out, k_out  device bf16, written; strides as above, with rows that do not
 *              overlap (stride >= heads * 128). May be q and k themselves with
 *              their strides (in place); otherwise must not overlap an input.
 * num_tokens == 0 is a no-op; num_tokens * (H_q + H_kv) must be below 2^31, and neither
 * head count above 65535.
 */
pkv_status pkv_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                            const void *q_weight, const void *k_weight, float eps,
                            const pkv_rope *rope, const int32_t *positions, int32_t num_tokens,
                            int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                            void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                            void *stream);

/*
 * The same on the way into the paged cache: q's rows go to q_out, k's, normed and
 * rotated, to their slots in k_cache, and v's, as they are, to theirs in v_cache.
 * Equivalent to pkv_qk_norm_rope, then pkv_kv_store of its keys and v; one pass.
 * A token whose slot is -1 is left out of the caches, not of q_out; another slot
 * outside the pool also raises PKV_DEVERR_SLOT. Two tokens with the same slot race.
 *   v          device bf16, as k
 *   slot_mapping  device int32 [num_tokens]
 *   k_cache, v_cache  device bf16 [num_blocks, block_size, H_kv, 128]; must not
 *              overlap the inputs or q_out
 * num_q_heads may be 0 (q and q_out are then not read); num_kv_heads may not. For a
 * 4-bit cache use pkv_qk_norm_rope, then pkv_kv_store_q4.
 * num_tokens * (H_q + 2 H_kv) must be below 2^31.
 */
pkv_status pkv_kv_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, const void *q_weight,
                         const void *k_weight, float eps, const pkv_rope *rope,
                         const int32_t *positions, const int32_t *slot_mapping,
                         int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                         int32_t head_dim, int32_t block_size, int64_t num_blocks, void *q_out,
                         int64_t q_out_stride, void *k_cache, void *v_cache, void *stream);

/*
 * Synchronise `stream`, then return in *flags_out the OR of the device error
 * words of every kernel of this library on the current device, and clear
 * them. It blocks the host; it is also the only way to clear the words, and
 * so to end the skip that a PKV_DEVERR_TIMEOUT starts.
 */
pkv_status pkv_check_device_errors(void *stream, uint32_t *flags_out);

/*
 * Non-blocking readout of the device error words: enqueues on `stream` a
 * one-thread kernel that writes the OR of the error words of every kernel of
 * this library on the current device into *host_flags, in stream order after
 * the work enqueued before it. The words are not cleared. host_flags must be
 * page-locked host memory (cudaHostAlloc, cudaMallocHost or cudaHostRegister)
 * that the device can write; other memory gives PKV_ERR_INVALID_ARG. The value
 * is there once that kernel has completed (for example after an event
 * recorded behind it). Capturable; make the first call on a device (which
 * looks up the words' addresses) before any stream capture.
 */
pkv_status pkv_read_device_errors_async(uint32_t *host_flags, void *stream);

/*
 * Raise bits of the device error words from the host, in stream order, as a
 * kernel that met the condition would. For tests of an engine's error
 * handling, for instance of the skip that follows PKV_DEVERR_TIMEOUT, without
 * making any kernel wait or fault. Bits outside PKV_DEVERR_* give
 * PKV_ERR_INVALID_ARG.
 */
pkv_status pkv_raise_device_errors(uint32_t flags, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
