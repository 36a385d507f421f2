"""Paged-KV-cache attention for GB300 (sm_103a): Python binding of libpkv.so.

The functions here have the names of the C entry points in ``include/pkv.h``
and do argument marshalling only: they check dtypes and shapes of torch
tensors, pass their device pointers and the current CUDA stream to the C ABI,
and allocate outputs the caller did not supply. (For 4-bit caches, eviction, queries
and keys before attention, sinks and chunks the checks are compiled, in the module
``_marshal`` beside the library, which only those calls load; they also want every
tensor on the current device.) Every step of the computation
runs in the library's CUDA kernels. There is no fallback: if libpkv.so has not
been built, or a call fails, an exception is raised.

Tensors (all CUDA, contiguous):
    k, v           bf16 [T, H_kv, 128]       new K/V rows
    k_cache,v_cache bf16 [num_blocks, block_size, H_kv, 128]
    slot_mapping   int32 [T]
    q              bf16 [S, H_q, 128] (decode) or [T_q, H_q, 128] (prefill)
    block_tables   int32 [S, max_blocks_per_seq], -1 padded
    context_lens   int32 [S]
    cu_seqlens_q/k int32 [S + 1]
"""
import contextlib
import ctypes
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libpkv.so")
MARSHAL_PATH = os.path.join(_HERE, "_marshal.so")

PKV_OK = 0
PKV_ERR_INVALID_ARG = 1
PKV_ERR_UNSUPPORTED = 2
PKV_ERR_WORKSPACE_TOO_SMALL = 3
PKV_ERR_CUDA = 4
PKV_ERR_OUT_OF_BLOCKS = 5

DECODE_STABLE_INPUTS = 0x1  # flag of paged_decode_attn_store (PKV_DECODE_STABLE_INPUTS)

DEVERR_SLOT = 0x1
DEVERR_BLOCK = 0x2
DEVERR_CONTEXT = 0x4
DEVERR_SEQLENS = 0x8
DEVERR_TIMEOUT = 0x10

_lib = None
_m = None  # the _marshal module (see _calls)


class PkvError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        name = status_string(status)
        detail = lib().pkv_last_cuda_error().decode() if status == PKV_ERR_CUDA else ""
        super().__init__(f"{what}: {name}" + (f" ({detail})" if detail else ""))


def _require(path):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with "
            "`python -m paged_kv_attention_22_gb300.build` (nvcc, sm_103a)")


def lib():
    """The loaded libpkv.so (ctypes), with argument types declared."""
    global _lib
    if _lib is not None:
        return _lib
    _require(LIBRARY_PATH)
    L = ctypes.CDLL(LIBRARY_PATH)
    P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_size_t)
    L.pkv_status_string.argtypes = [ctypes.c_int]
    L.pkv_status_string.restype = ctypes.c_char_p
    L.pkv_last_cuda_error.argtypes = []
    L.pkv_last_cuda_error.restype = ctypes.c_char_p
    L.pkv_kv_store.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i64, P]
    L.pkv_kv_store.restype = ctypes.c_int
    L.pkv_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.pkv_decode_workspace_size.restype = sz
    L.pkv_paged_decode_attn.argtypes = [P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i64,
                                        f32, i32, P, P, P, sz, P]
    L.pkv_paged_decode_attn.restype = ctypes.c_int
    L.pkv_paged_decode_attn_store.argtypes = [P, P, P, P, P, P, P, i32, P, i32, i32, i32, i32,
                                              i32, i32, i64, f32, i32, P, P, P, sz,
                                              ctypes.c_uint32, P]
    L.pkv_paged_decode_attn_store.restype = ctypes.c_int
    L.pkv_paged_decode_attn_noalloc.argtypes = [P, P, P, P, i32, P, i32, i32, i32, i32, i32,
                                                i32, i64, f32, i32, P, P, P]
    L.pkv_paged_decode_attn_noalloc.restype = ctypes.c_int
    L.pkv_set_programmatic_launch.argtypes = [i32]
    L.pkv_set_programmatic_launch.restype = None
    L.pkv_decode_set_config.argtypes = [i32, i32]
    L.pkv_decode_set_config.restype = None
    L.pkv_prefill_workspace_size.argtypes = [i32, i32]
    L.pkv_prefill_workspace_size.restype = sz
    L.pkv_paged_prefill_attn.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32,
                                         i32, i32, i64, f32, i32, P, P, P, sz, P]
    L.pkv_paged_prefill_attn.restype = ctypes.c_int
    q4 = [P, P, P, P]  # k_codes, k_params, v_codes, v_params
    L.pkv_kv_store_q4.argtypes = [P, P] + q4 + [P, i32, i32, i32, i32, i32, i64, P]
    L.pkv_kv_store_q4.restype = ctypes.c_int
    L.pkv_kv_load_q4.argtypes = q4 + [P, P, P, i32, i32, i32, i32, i32, i64, P]
    L.pkv_kv_load_q4.restype = ctypes.c_int
    L.pkv_decode_q4_workspace_size.argtypes = [i32] * 6
    L.pkv_decode_q4_workspace_size.restype = sz
    L.pkv_paged_decode_attn_q4.argtypes = [P] + q4 + [P, i32, P, i32, i32, i32, i32, i32, i32, i32,
                                                      i64, f32, i32, P, P, P, i64, P, sz, P]
    L.pkv_paged_decode_attn_q4.restype = ctypes.c_int
    L.pkv_prefill_q4_workspace_size.argtypes = [i32] * 5
    L.pkv_prefill_q4_workspace_size.restype = sz
    L.pkv_paged_prefill_attn_q4.argtypes = [P] + q4 + [P, P, P, i32, i32, i32, i32, i32, i32, i32,
                                                       i32, i32, i32, i32, i64, f32, i32, P, P, P,
                                                       sz, P]
    L.pkv_paged_prefill_attn_q4.restype = ctypes.c_int
    L.pkv_decode_scores_workspace_size.argtypes = [i32] * 5
    L.pkv_decode_scores_workspace_size.restype = sz
    L.pkv_paged_decode_attn_scores.argtypes = [P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32,
                                               i64, f32, i32, P, P, P, i64, P, sz, P]
    L.pkv_paged_decode_attn_scores.restype = ctypes.c_int
    L.pkv_evict_select.argtypes = [P, i64, P, i32, i32, i32, i32, P, P, P]
    L.pkv_evict_select.restype = ctypes.c_int
    L.pkv_evict_select_new.argtypes = L.pkv_evict_select.argtypes
    L.pkv_evict_select_new.restype = ctypes.c_int
    rows = [P, i32, P, i32, P, i32, P, i32]  # source and destination tables, keep, new_lens, num_seqs
    L.pkv_evict_compact.argtypes = [P, P] + rows + [i32, i32, i32, i64, P, i64, P, i64, P]
    L.pkv_evict_compact.restype = ctypes.c_int
    L.pkv_evict_compact_q4.argtypes = q4 + rows + [i32, i32, i32, i32, i64, P, i64, P, i64, P]
    L.pkv_evict_compact_q4.restype = ctypes.c_int
    L.pkv_paged_decode_attn_sinks.argtypes = [P, P, P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i64,
                                              f32, i32, i32, P, P, P, sz, ctypes.c_uint32, P]
    L.pkv_paged_decode_attn_sinks.restype = ctypes.c_int
    L.pkv_chunk_workspace_size.argtypes = [i32] * 4
    L.pkv_chunk_workspace_size.restype = sz
    L.pkv_paged_chunk_attn.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32, i32, i64, f32,
                                       i32, i32, P, P, P, sz, P]
    L.pkv_paged_chunk_attn.restype = ctypes.c_int
    L.pkv_rope_init.argtypes = [P, i32, i32, ctypes.c_double, i32, ctypes.c_double, i32, ctypes.c_double,
                                ctypes.c_double]
    L.pkv_rope_init.restype = ctypes.c_int
    L.pkv_rope_init_frequencies.argtypes = [P, i32, i32, P, f32]
    L.pkv_rope_init_frequencies.restype = ctypes.c_int
    L.pkv_qk_norm_rope.argtypes = [P, i64, P, i64, P, P, f32, P, P, i32, i32, i32, i32, P, i64, P, i64, P]
    L.pkv_qk_norm_rope.restype = ctypes.c_int
    L.pkv_kv_append.argtypes = [P, i64, P, i64, P, i64, P, P, f32, P, P, P, i32, i32, i32, i32, i32, i64,
                                P, i64, P, P, P]
    L.pkv_kv_append.restype = ctypes.c_int
    L.pkv_check_device_errors.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    L.pkv_check_device_errors.restype = ctypes.c_int
    L.pkv_read_device_errors_async.argtypes = [P, P]
    L.pkv_read_device_errors_async.restype = ctypes.c_int
    L.pkv_raise_device_errors.argtypes = [ctypes.c_uint32, P]
    L.pkv_raise_device_errors.restype = ctypes.c_int
    pi32 = ctypes.POINTER(ctypes.c_int32)
    L.pkv_bm_create.argtypes = [i32, i32]
    L.pkv_bm_create.restype = P
    L.pkv_bm_destroy.argtypes = [P]
    L.pkv_bm_destroy.restype = None
    L.pkv_bm_num_free_blocks.argtypes = [P]
    L.pkv_bm_num_free_blocks.restype = i32
    L.pkv_bm_ref_count.argtypes = [P, i32]
    L.pkv_bm_ref_count.restype = i32
    L.pkv_bm_add_sequence.argtypes = [P, i64, P, i32, pi32]
    L.pkv_bm_add_sequence.restype = ctypes.c_int
    L.pkv_bm_append_token.argtypes = [P, i64, i32]
    L.pkv_bm_append_token.restype = ctypes.c_int
    L.pkv_bm_evict_sequences.argtypes = [P, P, P, i32]
    L.pkv_bm_evict_sequences.restype = ctypes.c_int
    L.pkv_bm_free_sequence.argtypes = [P, i64]
    L.pkv_bm_free_sequence.restype = ctypes.c_int
    L.pkv_bm_num_tokens.argtypes = [P, i64, pi32]
    L.pkv_bm_num_tokens.restype = ctypes.c_int
    L.pkv_bm_block_table.argtypes = [P, i64, P, i32, pi32]
    L.pkv_bm_block_table.restype = ctypes.c_int
    L.pkv_bm_slots.argtypes = [P, i64, i32, i32, P]
    L.pkv_bm_slots.restype = ctypes.c_int
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().pkv_status_string(int(status)).decode()


def _check(status, what):
    if status != PKV_OK:
        raise PkvError(status, what)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, name, dtype, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def kv_store(k, v, k_cache, v_cache, slot_mapping, stream=None):
    """Scatter k, v [T, H_kv, D] into the caches at slot_mapping (-1: skip)."""
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    NB, bs, H_kv, D = k_cache.shape
    if v_cache.shape != k_cache.shape or k.shape != v.shape or k.shape[1:] != (H_kv, D) \
            or slot_mapping.shape[0] != k.shape[0]:
        raise ValueError("inconsistent shapes")
    _check(lib().pkv_kv_store(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
                              k.shape[0], H_kv, D, bs, NB, _stream(stream)), "pkv_kv_store")


def decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len) -> int:
    """Workspace bytes of paged_decode_attn on the current device (0: invalid sizes)."""
    return int(lib().pkv_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                               max_context_len))


DECODE_NUM_VARIANTS = 3


def new_decode_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                         device="cuda"):
    """A decode workspace for these sizes on the current device."""
    need = decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len)
    if need == 0:
        raise PkvError(PKV_ERR_CUDA, "pkv_decode_workspace_size")
    return torch.zeros(need, dtype=torch.uint8, device=device)


def set_programmatic_launch(enabled: bool) -> None:
    """Launch kernels with programmatic dependent launch (the default) or not."""
    lib().pkv_set_programmatic_launch(1 if enabled else 0)


def decode_set_config(ctas: int = 0, variant: int = 0) -> None:
    """Tuning knob of the decode launch: persistent CTAs (0 = one per SM) and
    launch-shape variant (0 = default). Process-wide."""
    lib().pkv_decode_set_config(int(ctas), int(variant))


def paged_decode_attn(q, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
                      out=None, lse=None, workspace=None, stream=None, with_lse=True,
                      sliding_window=0):
    """q=1 decode attention through block tables (sliding_window > 0: each query
    sees only the last sliding_window keys up to its own). Returns (out, lse)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    S, H_q, D = q.shape
    NB, bs, H_kv, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3)
    if lse is None and with_lse:
        lse = torch.empty((S, H_q), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    if workspace is None:
        workspace = new_decode_workspace(S, H_q, H_kv, D, int(max_context_len), q.device)
    _need(workspace, "workspace", torch.uint8, 1)
    _check(lib().pkv_paged_decode_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), int(max_context_len), S, H_q, H_kv, D, bs, NB, float(scale),
        int(sliding_window), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
        _stream(stream)), "pkv_paged_decode_attn")
    return out, lse


def paged_decode_attn_store(k_new, v_new, slot_mapping, q, k_cache, v_cache, block_tables,
                            context_lens, max_context_len, scale, out=None, lse=None,
                            workspace=None, stream=None, with_lse=True, sliding_window=0,
                            stable_inputs=False):
    """Fused decode step: store each sequence's new K/V row (position
    context_lens[s] - 1, slot slot_mapping[s]) and attend. Returns (out, lse).
    stable_inputs: the caches (but the new rows), block_tables and context_lens
    are not written by the kernels still in flight on the stream, so the call
    may read them before the previous kernel ends (PKV_DECODE_STABLE_INPUTS)."""
    _need(k_new, "k_new", torch.bfloat16, 3)
    _need(v_new, "v_new", torch.bfloat16, 3)
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    S, H_q, D = q.shape
    NB, bs, H_kv, _ = k_cache.shape
    if k_new.shape != (S, H_kv, D) or v_new.shape != k_new.shape or slot_mapping.shape[0] != S:
        raise ValueError("inconsistent shapes")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3)
    if lse is None and with_lse:
        lse = torch.empty((S, H_q), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    if workspace is None:
        workspace = new_decode_workspace(S, H_q, H_kv, D, int(max_context_len), q.device)
    _need(workspace, "workspace", torch.uint8, 1)
    _check(lib().pkv_paged_decode_attn_store(
        _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(q), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), int(max_context_len), S,
        H_q, H_kv, D, bs, NB, float(scale), int(sliding_window), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel(), DECODE_STABLE_INPUTS if stable_inputs else 0,
        _stream(stream)), "pkv_paged_decode_attn_store")
    return out, lse


# Static scratch of paged_decode_attn_noalloc (PKV_DECODE_NOALLOC_SCRATCH_BYTES).
DECODE_NOALLOC_SCRATCH_BYTES = 16 << 20


def paged_decode_attn_noalloc(q, k_cache, v_cache, block_tables, context_lens, max_context_len,
                              scale, out, lse=None, stream=None, sliding_window=0):
    """Decode attention for callers that cannot allocate device memory: same
    result as paged_decode_attn, with the library's static scratch in place of a
    workspace. `out` (and `lse`, if wanted) must be supplied; nothing is
    allocated here either. Calls overlapping on one GPU race on the scratch."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    S, H_q, D = q.shape
    NB, bs, H_kv, _ = k_cache.shape
    _check(lib().pkv_paged_decode_attn_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), int(max_context_len), S, H_q, H_kv, D, bs, NB, float(scale),
        int(sliding_window), _ptr(out), _ptr(lse), _stream(stream)),
        "pkv_paged_decode_attn_noalloc")
    return out, lse


def prefill_workspace_size(num_seqs, max_seqlen_q) -> int:
    return int(lib().pkv_prefill_workspace_size(num_seqs, max_seqlen_q))


def paged_prefill_attn(q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_tables,
                       max_seqlen_q, max_seqlen_k, scale, out=None, lse=None, workspace=None,
                       stream=None, with_lse=True, sliding_window=0):
    """Varlen causal prefill over the paged cache (bottom-right aligned;
    sliding_window > 0: each query sees only the last sliding_window keys up to
    its own). Returns (out, lse)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    _need(block_tables, "block_tables", torch.int32, 2)
    T, H_q, D = q.shape
    NB, bs, H_kv, _ = k_cache.shape
    S = cu_seqlens_q.shape[0] - 1
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3)
    if lse is None and with_lse:
        lse = torch.empty((T, H_q), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    need = prefill_workspace_size(S, int(max_seqlen_q))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(lib().pkv_paged_prefill_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
        _ptr(block_tables), block_tables.shape[1], S, T, int(max_seqlen_q), int(max_seqlen_k),
        H_q, H_kv, D, bs, NB, float(scale), int(sliding_window), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel() if workspace is not None else 0, _stream(stream)),
        "pkv_paged_prefill_attn")
    return out, lse


class Q4Cache(NamedTuple):
    """K or V of a paged cache held in 4 bits (pkv.h, "A cache held in 4 bits").
    The calls also take a plain (codes, params) pair."""
    codes: torch.Tensor   # uint8 [num_blocks, H_kv, block_size, 64]
    params: torch.Tensor  # bf16 [num_blocks, H_kv, block_size, 128 / group_size, 2]


def new_q4_cache(num_blocks, block_size, num_kv_heads, group_size=32, device="cuda") -> Q4Cache:
    """A 4-bit K or V cache whose rows read back as zeros."""
    if group_size not in (32, 64, 128):
        raise ValueError("group_size must be 32, 64 or 128")
    head = (num_blocks, num_kv_heads, block_size)
    return Q4Cache(torch.zeros(*head, 64, dtype=torch.uint8, device=device),
                   torch.zeros(*head, 128 // group_size, 2, dtype=torch.bfloat16, device=device))


def _calls():
    """The _marshal module, which checks arguments and calls the C entries."""
    global _m
    if _m is None:
        lib()
        _require(MARSHAL_PATH)
        from . import _marshal
        _m = _marshal
    return _m


_CURRENT = contextlib.nullcontext()


def _on(stream):
    """Allocate for work on `stream` (None: the current one): memory that is freed
    when a call returns is then reused in that stream's order only."""
    return torch.cuda.stream(stream) if stream is not None else _CURRENT


def kv_store_q4(k, v, k_cache, v_cache, slot_mapping, stream=None):
    """Quantise k, v [T, H_kv, 128] into the 4-bit caches at slot_mapping (-1: skip)."""
    st = _calls().kv_store_q4(k, v, k_cache, v_cache, slot_mapping, stream)
    if st:
        raise PkvError(st, "pkv_kv_store_q4")


def kv_load_q4(k_cache, v_cache, slots, k=None, v=None, stream=None):
    """The rows at slots [T] as bf16 (k, v) [T, H_kv, 128]; zeros for slot -1."""
    if stream is None:
        st, k, v = _calls().kv_load_q4(k_cache, v_cache, slots, k, v, None)
    else:  # what the call allocates belongs to its stream
        with torch.cuda.stream(stream):
            st, k, v = _calls().kv_load_q4(k_cache, v_cache, slots, k, v, stream)
    if st:
        raise PkvError(st, "pkv_kv_load_q4")
    return k, v


def q4_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, max_context_len,
                             with_scores=False) -> int:
    """Workspace bytes of paged_decode_attn_q4 on the current device (0: invalid sizes)."""
    return int(lib().pkv_decode_q4_workspace_size(num_seqs, num_q_heads, num_kv_heads, 128,
                                                  max_context_len, 1 if with_scores else 0))


def new_q4_decode_workspace(num_seqs, num_q_heads, num_kv_heads, max_context_len, with_scores=False,
                            device="cuda"):
    """A workspace of paged_decode_attn_q4 for these sizes on the current device."""
    need = q4_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, max_context_len, with_scores)
    if need == 0:
        raise PkvError(PKV_ERR_CUDA, "pkv_decode_q4_workspace_size")
    return torch.empty(need, dtype=torch.uint8, device=device)


def _decode_outputs(q, out, lse, with_lse):
    """Allocate the outputs of a decode call that the caller did not supply."""
    if out is None:
        out = torch.empty_like(q)
    if lse is None and with_lse:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    return out, lse


def paged_decode_attn_q4(q, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
                         out=None, lse=None, workspace=None, stream=None, with_lse=True,
                         sliding_window=0, key_scores=None):
    """q=1 decode attention over a 4-bit cache. key_scores [S, >= max_context_len]
    (fp32), if given, gains each key's attention weight, summed over the query
    heads. Returns (out, lse)."""
    if out is None or workspace is None or (lse is None and with_lse):
        with _on(stream):
            out, lse = _decode_outputs(q, out, lse, with_lse)
            if workspace is None:
                workspace = new_q4_decode_workspace(q.shape[0], q.shape[1], k_cache[0].shape[1],
                                                    int(max_context_len), key_scores is not None,
                                                    q.device)
    st = _calls().paged_decode_attn_q4(k_cache, v_cache, q, block_tables, context_lens,
                                         max_context_len, scale, out, lse, key_scores, workspace,
                                         sliding_window, stream)
    if st:
        raise PkvError(st, "pkv_paged_decode_attn_q4")
    return out, lse


def q4_prefill_workspace_size(num_seqs, total_k, max_seqlen_k, num_kv_heads) -> int:
    """Workspace bytes of paged_prefill_attn_q4 on the current device (0: invalid sizes)."""
    return int(lib().pkv_prefill_q4_workspace_size(num_seqs, total_k, max_seqlen_k, num_kv_heads, 128))


def new_q4_prefill_workspace(num_seqs, total_k, max_seqlen_k, num_kv_heads, device="cuda"):
    """A workspace of paged_prefill_attn_q4 for these sizes on the current device."""
    need = q4_prefill_workspace_size(num_seqs, total_k, max_seqlen_k, num_kv_heads)
    if need == 0:
        raise PkvError(PKV_ERR_CUDA, "pkv_prefill_q4_workspace_size")
    return torch.empty(need, dtype=torch.uint8, device=device)


def paged_prefill_attn_q4(q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_tables,
                          max_seqlen_q, max_seqlen_k, total_k, scale, out=None, lse=None,
                          workspace=None, stream=None, with_lse=True, sliding_window=0):
    """Varlen causal prefill over a 4-bit cache (arguments as paged_prefill_attn;
    total_k: an upper bound of cu_seqlens_k[-1]). Returns (out, lse)."""
    if out is None or workspace is None or (lse is None and with_lse):
        with _on(stream):
            out, lse = _decode_outputs(q, out, lse, with_lse)
            S = cu_seqlens_q.shape[0] - 1
            if workspace is None and S > 0 and q.shape[0] > 0:
                workspace = new_q4_prefill_workspace(S, int(total_k), int(max_seqlen_k),
                                                     k_cache[0].shape[1], q.device)
    st = _calls().paged_prefill_attn_q4(k_cache, v_cache, q, cu_seqlens_q, cu_seqlens_k,
                                          block_tables, max_seqlen_q, max_seqlen_k, total_k, scale,
                                          out, lse, workspace, sliding_window, stream)
    if st:
        raise PkvError(st, "pkv_paged_prefill_attn_q4")
    return out, lse


def decode_scores_workspace_size(num_seqs, num_q_heads, num_kv_heads, max_context_len) -> int:
    """Workspace bytes of paged_decode_attn_scores on the current device (0: invalid sizes)."""
    return int(lib().pkv_decode_scores_workspace_size(num_seqs, num_q_heads, num_kv_heads, 128,
                                                      max_context_len))


def new_decode_scores_workspace(num_seqs, num_q_heads, num_kv_heads, max_context_len,
                                device="cuda"):
    """A workspace of paged_decode_attn_scores for these sizes on the current device."""
    need = decode_scores_workspace_size(num_seqs, num_q_heads, num_kv_heads, max_context_len)
    if need == 0:
        raise PkvError(PKV_ERR_CUDA, "pkv_decode_scores_workspace_size")
    return torch.empty(need, dtype=torch.uint8, device=device)


def paged_decode_attn_scores(q, k_cache, v_cache, block_tables, context_lens, max_context_len,
                             scale, key_scores, out=None, lse=None, workspace=None, stream=None,
                             with_lse=True, sliding_window=0):
    """paged_decode_attn that also adds each key's attention weight, summed over
    the query heads, to key_scores [S, >= max_context_len] (fp32). Returns (out, lse)."""
    if out is None or workspace is None or (lse is None and with_lse):
        with _on(stream):
            out, lse = _decode_outputs(q, out, lse, with_lse)
            if workspace is None:
                workspace = new_decode_scores_workspace(q.shape[0], q.shape[1], k_cache.shape[2],
                                                        int(max_context_len), q.device)
    st = _calls().paged_decode_attn_scores(k_cache, v_cache, q, block_tables, context_lens,
                                             max_context_len, scale, out, lse, key_scores,
                                             workspace, sliding_window, stream)
    if st:
        raise PkvError(st, "pkv_paged_decode_attn_scores")
    return out, lse


def evict_select(key_scores, context_lens, budget, recent, keep=None, new_lens=None, stream=None):
    """Positions that stay: the last `recent` and the highest-scoring others, budget
    in all, ascending. Returns (keep int32 [S, budget], -1 padded, new_lens int32 [S]).
    A sequence of invalid length gets -1 in both, which a compaction refuses, unless
    keep and new_lens are both given: its rows are then left as they were."""
    if stream is None:
        st, keep, new_lens = _calls().evict_select(key_scores, context_lens, budget, recent, keep,
                                                   new_lens, None)
    else:  # what the call allocates belongs to its stream
        with torch.cuda.stream(stream):
            st, keep, new_lens = _calls().evict_select(key_scores, context_lens, budget, recent,
                                                       keep, new_lens, stream)
    if st:
        raise PkvError(st, "pkv_evict_select")
    return keep, new_lens


def evict_compact(k_cache, v_cache, src_tables, dst_tables, keep, new_lens, key_scores=None,
                  dst_key_scores=None, stream=None):
    """Move each sequence's kept rows (evict_select) to positions 0 .. new_lens - 1 of
    dst_tables; equal tables compact in place. The scores move along, with zeros
    behind them (pass the same tensor twice for in place)."""
    st = _calls().evict_compact(k_cache, v_cache, src_tables, dst_tables, keep, new_lens,
                                  key_scores, dst_key_scores, stream)
    if st:
        raise PkvError(st, "pkv_evict_compact")


def evict_compact_q4(k_cache, v_cache, src_tables, dst_tables, keep, new_lens, key_scores=None,
                     dst_key_scores=None, stream=None):
    """evict_compact for a 4-bit cache."""
    st = _calls().evict_compact_q4(k_cache, v_cache, src_tables, dst_tables, keep, new_lens,
                                     key_scores, dst_key_scores, stream)
    if st:
        raise PkvError(st, "pkv_evict_compact_q4")


def paged_decode_attn_sinks(q, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
                            sliding_window, num_sinks, out=None, lse=None, workspace=None, stream=None,
                            with_lse=True, k_new=None, v_new=None, slot_mapping=None, stable_inputs=False):
    """q=1 decode attention where each sequence sees its first num_sinks keys and its last
    sliding_window ones. With k_new, v_new [S, H_kv, 128] and slot_mapping the new token's rows are
    stored by the call, as in paged_decode_attn_store. The workspace is new_decode_workspace's.
    Returns (out, lse)."""
    if out is None or workspace is None or (lse is None and with_lse):
        with _on(stream):
            out, lse = _decode_outputs(q, out, lse, with_lse)
            if workspace is None:
                workspace = new_decode_workspace(q.shape[0], q.shape[1], k_cache.shape[2], 128,
                                                 int(max_context_len), q.device)
    st = _calls().paged_decode_attn_sinks(k_cache, v_cache, q, block_tables, context_lens, max_context_len,
                                          scale, out, lse, None, workspace, sliding_window, num_sinks, k_new,
                                          v_new, slot_mapping, DECODE_STABLE_INPUTS if stable_inputs else 0,
                                          stream)
    if st:
        raise PkvError(st, "pkv_paged_decode_attn_sinks")
    return out, lse


def chunk_workspace_size(num_seqs, num_q_heads, num_kv_heads) -> int:
    """Workspace bytes of paged_chunk_attn on the current device (0: invalid sizes)."""
    return int(lib().pkv_chunk_workspace_size(num_seqs, num_q_heads, num_kv_heads, 128))


def new_chunk_workspace(num_seqs, num_q_heads, num_kv_heads, device="cuda"):
    """A workspace of paged_chunk_attn for these sizes on the current device."""
    need = chunk_workspace_size(num_seqs, num_q_heads, num_kv_heads)
    if need == 0:
        raise PkvError(PKV_ERR_CUDA, "pkv_chunk_workspace_size")
    return torch.empty(need, dtype=torch.uint8, device=device)


def paged_chunk_attn(q, k_cache, v_cache, cu_seqlens_q, context_lens, block_tables, max_seqlen_q,
                     max_context_len, scale, sliding_window=0, num_sinks=0, out=None, lse=None, workspace=None,
                     stream=None, with_lse=True):
    """Attention of each sequence's last cu_seqlens_q[s + 1] - cu_seqlens_q[s] positions (their rows
    stored before) over its context_lens[s] keys in the paged cache, causal; with a window each query sees
    the last sliding_window keys up to its own and the first num_sinks. Weights are rounded to bf16, as in
    prefill (decode keeps them in fp32). The bounds choose between two kernels: pkv.h says how, and why a
    graph that is replayed for short segments wants tight ones. Returns (out, lse)."""
    if out is None or workspace is None or (lse is None and with_lse):
        with _on(stream):
            out, lse = _decode_outputs(q, out, lse, with_lse)
            S = cu_seqlens_q.shape[0] - 1
            if workspace is None and S > 0 and q.shape[0] > 0:
                workspace = new_chunk_workspace(S, q.shape[1], k_cache.shape[2], q.device)
    st = _calls().paged_chunk_attn(k_cache, v_cache, q, cu_seqlens_q, context_lens, block_tables, max_seqlen_q,
                                   max_context_len, scale, out, lse, workspace, sliding_window, num_sinks, stream)
    if st:
        raise PkvError(st, "pkv_paged_chunk_attn")
    return out, lse


class _RopeStruct(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("turns", ctypes.c_uint64 * 64)]


class Rope(NamedTuple):
    """A rotation by position (pkv_rope), made by rope() once for a model."""
    data: bytes        # the C structure
    rotary_dim: int
    interleaved: bool
    magnitude: float


_ROPE_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}


def rope(rotary_dim=128, base=10000.0, interleaved=False, scaling=None, factor=1.0,
         original_positions=0, beta_fast=32.0, beta_slow=1.0, frequencies=None, magnitude=1.0) -> Rope:
    """The rotation of the first rotary_dim dims of a head, in pairs (i, i + rotary_dim / 2) or,
    interleaved, (2 i, 2 i + 1). scaling: None, "linear", "ntk" or "yarn" (pkv.h has the formulas).
    frequencies: radians a position of each pair, in place of base and scaling, with a magnitude."""
    made = _RopeStruct()
    if frequencies is not None:
        values = [float(f) for f in frequencies]
        if len(values) * 2 != rotary_dim:
            raise ValueError("frequencies must have rotary_dim / 2 values")
        if scaling is not None:
            raise ValueError("frequencies take no scaling")
        _check(lib().pkv_rope_init_frequencies(ctypes.byref(made), int(rotary_dim), int(bool(interleaved)),
                                               (ctypes.c_double * max(1, len(values)))(*values),
                                               float(magnitude)), "pkv_rope_init_frequencies")
    else:
        if scaling not in _ROPE_SCALINGS:
            raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
        if magnitude != 1.0:
            raise ValueError("a magnitude goes with frequencies")
        _check(lib().pkv_rope_init(ctypes.byref(made), int(rotary_dim), int(bool(interleaved)), float(base),
                                   _ROPE_SCALINGS[scaling], float(factor), int(original_positions),
                                   float(beta_fast), float(beta_slow)), "pkv_rope_init")
    return Rope(bytes(made), made.rotary_dim, bool(made.interleaved), made.magnitude)


def qk_norm_rope(q, k, rope, positions, q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None,
                 stream=None):
    """Norm each head's row of q [T, H_q, 128] and k [T, H_kv, 128] (with weights [128]; None: not
    normed) and rotate it by its token's position. q and k may be parts of a packed projection
    (heads contiguous, any distance between tokens), q_out and k_out the same tensors. Either of q
    and k may be None; rope None: no rotation. Returns (q_out, k_out)."""
    if (q_out is None and q is not None) or (k_out is None and k is not None):
        with _on(stream):
            if q_out is None and q is not None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if k_out is None and k is not None:
                k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    st = _calls().qk_norm_rope(q, k, q_weight, k_weight, positions, eps, rope.data if rope is not None else None,
                               q_out, k_out, stream)
    if st:
        raise PkvError(st, "pkv_qk_norm_rope")
    return q_out, k_out


def kv_append(q, k, v, rope, positions, k_cache, v_cache, slot_mapping, q_weight=None, k_weight=None, eps=1e-6,
              q_out=None, stream=None):
    """qk_norm_rope on the way into the paged cache: k's rows, normed and rotated, and v's, as they
    are, go to slot_mapping (-1: skip), q's to q_out. q may be None. Returns q_out."""
    if q_out is None and q is not None:
        with _on(stream):
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    st = _calls().kv_append(q, k, v, q_weight, k_weight, positions, eps, rope.data if rope is not None else None,
                            k_cache, v_cache, slot_mapping, q_out, stream)
    if st:
        raise PkvError(st, "pkv_kv_append")
    return q_out


def check_device_errors(stream=None) -> int:
    """Synchronise, then return and clear the OR of the kernels' device error words."""
    flags = ctypes.c_uint32(0)
    _check(lib().pkv_check_device_errors(_stream(stream), ctypes.byref(flags)),
           "pkv_check_device_errors")
    return int(flags.value)


def read_device_errors_async(host_flags, stream=None) -> None:
    """Enqueue a non-blocking readout of the OR of the kernels' device error
    words into host_flags, a pinned (page-locked) CPU int32/uint32 tensor of
    at least one element; its first element holds the value once the work
    enqueued before this call on the stream has completed. Nothing is cleared."""
    if not isinstance(host_flags, torch.Tensor) or host_flags.is_cuda \
            or host_flags.dtype not in (torch.int32,) or host_flags.numel() < 1:
        raise TypeError("host_flags must be a CPU int32 tensor")
    _check(lib().pkv_read_device_errors_async(_ptr(host_flags), _stream(stream)),
           "pkv_read_device_errors_async")


def raise_device_errors(flags: int, stream=None) -> None:
    """Raise bits of the device error words from the host, in stream order (for
    tests of error handling)."""
    _check(lib().pkv_raise_device_errors(int(flags), _stream(stream)), "pkv_raise_device_errors")


class BlockManager:
    """The host-side KV block manager of libpkv.so (pkv_blocks.h): reference-
    counted cache blocks with prefix sharing of full blocks; it emits block-table
    rows and the slots of the tokens to store."""

    def __init__(self, num_blocks: int, block_size: int):
        import numpy as np  # noqa: F401  (used by the methods)
        self._L = lib()
        self._h = self._L.pkv_bm_create(int(num_blocks), int(block_size))
        if not self._h:
            raise PkvError(PKV_ERR_INVALID_ARG, "pkv_bm_create")
        self.num_blocks = int(num_blocks)
        self.block_size = int(block_size)

    def close(self):
        if getattr(self, "_h", None):
            self._L.pkv_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()

    @property
    def num_free_blocks(self) -> int:
        return int(self._L.pkv_bm_num_free_blocks(self._h))

    def ref_count(self, block: int) -> int:
        return int(self._L.pkv_bm_ref_count(self._h, int(block)))

    def add_sequence(self, seq_id: int, token_ids) -> int:
        """Admit a prompt; returns how many leading tokens are already cached."""
        import numpy as np
        tok = np.ascontiguousarray(token_ids, dtype=np.int32)
        cached = ctypes.c_int32(0)
        _check(self._L.pkv_bm_add_sequence(self._h, int(seq_id), tok.ctypes.data, tok.shape[0],
                                           ctypes.byref(cached)), "pkv_bm_add_sequence")
        return int(cached.value)

    def append_token(self, seq_id: int, token_id: int) -> None:
        _check(self._L.pkv_bm_append_token(self._h, int(seq_id), int(token_id)),
               "pkv_bm_append_token")

    def evict_sequences(self, seq_ids, num_kept) -> None:
        """Keep num_kept[k] tokens of seq_ids[k]; block_table() then gives the
        destination rows of one compaction of these sequences."""
        import numpy as np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        kept = np.ascontiguousarray(num_kept, dtype=np.int32)
        if ids.ndim != 1 or ids.shape != kept.shape:
            raise ValueError("seq_ids and num_kept must be lists of the same length")
        _check(self._L.pkv_bm_evict_sequences(self._h, ids.ctypes.data, kept.ctypes.data,
                                              ids.shape[0]), "pkv_bm_evict_sequences")

    def free_sequence(self, seq_id: int) -> None:
        _check(self._L.pkv_bm_free_sequence(self._h, int(seq_id)), "pkv_bm_free_sequence")

    def num_tokens(self, seq_id: int) -> int:
        n = ctypes.c_int32(0)
        _check(self._L.pkv_bm_num_tokens(self._h, int(seq_id), ctypes.byref(n)),
               "pkv_bm_num_tokens")
        return int(n.value)

    def block_table(self, seq_id: int, max_blocks: int = None):
        """The sequence's block ids, padded with -1 to max_blocks (default: none)."""
        import numpy as np
        n = ctypes.c_int32(0)
        self._L.pkv_bm_block_table(self._h, int(seq_id), None, 0, ctypes.byref(n))
        width = int(n.value) if max_blocks is None else int(max_blocks)
        row = np.empty(width, np.int32)
        _check(self._L.pkv_bm_block_table(self._h, int(seq_id), row.ctypes.data, width,
                                          ctypes.byref(n)), "pkv_bm_block_table")
        return row

    def block_tables(self, seq_ids, max_blocks: int):
        """Block-table rows of several sequences [len(seq_ids), max_blocks]."""
        import numpy as np
        return np.stack([self.block_table(s, max_blocks) for s in seq_ids]).astype(np.int32)

    def slots(self, seq_id: int, first: int, count: int):
        """Cache slots of positions first .. first + count - 1."""
        import numpy as np
        out = np.empty(int(count), np.int32)
        _check(self._L.pkv_bm_slots(self._h, int(seq_id), int(first), int(count),
                                    out.ctypes.data), "pkv_bm_slots")
        return out
