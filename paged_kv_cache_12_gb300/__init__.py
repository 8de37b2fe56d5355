"""Paged KV cache decode path for GB300 (sm_103a).

A thin ctypes binding over libpa.so, the C-ABI library declared in
``include/pa.h``.  The functions keep the C names and only marshal arguments:
tensors are passed as raw pointers, the stream is the caller's (default: the
current torch stream), and every step of the computation runs in the
library's CUDA kernels.  There is no fallback: if libpa.so is missing or a
call fails, a ``PAError`` is raised.

Device tensors are torch CUDA tensors (torch is used for device memory and
streams only):
  caches    fp16 [num_blocks, num_kv_heads, block_size, head_dim]
  query/out fp16 [num_seqs, num_heads, head_dim]
  key/value fp16 [num_tokens, num_kv_heads, head_dim]
Latent caches (the pa_latent_* calls) hold one row per token for all heads:
  16-bit    [num_blocks, block_size, 576] = 512 latent elements, 64 rotary ones
  FP8       uint8 [num_blocks, block_size, 656] = 512 E4M3 codes, 64 bf16
            rotary elements, 4 float scales
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

PA_OK = 0
PA_ERR_INVALID_ARG = -1
PA_ERR_OUT_OF_BLOCKS = -2
PA_ERR_STATE = -3
PA_ERR_WORKSPACE = -4
PA_ERR_CUDA = -5
PA_ERR_UNSUPPORTED = -6
PA_ERR_TIMEOUT = -7

# every symbol include/pa.h declares
EXPORTS = (
    "pa_status_string", "pa_version", "pa_kv_write", "pa_block_copy", "pa_decode_workspace_size", "pa_decode",
    "pa_workspace_status", "pa_alloc_create", "pa_alloc_destroy", "pa_alloc_add_seq", "pa_alloc_append",
    "pa_alloc_fork", "pa_alloc_free_seq", "pa_alloc_seq_len", "pa_alloc_block_tables", "pa_alloc_refcount",
    "pa_alloc_stats", "pa_decode_static_ws", "pa_alloc_free_queue", "pa_alloc_enable_prefix_cache",
    "pa_alloc_match_prefix", "pa_alloc_append_ids", "pa_alloc_block_hash", "pa_alloc_prefix_stats", "pa_sha256",
    "pa_decode_shared_prefix_workspace_size", "pa_decode_shared_prefix", "pa_selftest_wait_timeout",
    "pa_attention_causal_workspace_size", "pa_attention_causal", "pa_kv_write_fp8", "pa_block_copy_typed",
    "pa_decode_typed", "pa_attention_causal_typed", "pa_decode_static_ws_status", "pa_latent_write",
    "pa_latent_block_copy", "pa_latent_read", "pa_latent_attention_workspace_size", "pa_latent_attention",
    "pa_latent_attention_expanded_workspace_size", "pa_latent_attention_expanded", "pa_verify_drafts",
    "pa_kv_write_rope", "pa_attention_tree_workspace_size", "pa_attention_tree", "pa_verify_tree", "pa_kv_move_path",
)

# cache element types (PA_KV_* in pa.h)
PA_KV_F16, PA_KV_BF16, PA_KV_FP8_E4M3 = 0, 1, 2

# a latent cache's row (PA_LATENT_* in pa.h): latent and rotary elements, bytes when quantised
PA_LATENT_DIM, PA_LATENT_ROPE_DIM, PA_LATENT_ROW, PA_LATENT_ROW_FP8_BYTES = 512, 64, 576, 656

# element types of probability rows (PA_PROBS_* in pa.h)
PA_PROBS_F32, PA_PROBS_F16, PA_PROBS_BF16 = 0, 1, 2

# axes of a token's position and nodes of a tree, at most (PA_ROPE_MAX_AXES, PA_TREE_MAX_NODES in pa.h)
PA_ROPE_MAX_AXES, PA_TREE_MAX_NODES = 4, 256

# bytes of the library's built-in scratch array used by pa_decode_static_ws
PA_DECODE_STATIC_WS_BYTES = 64 << 20

_lib = None


class PAError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {status_text(code)} ({code})")
        self.code = code


class AllocStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("num_blocks", "free_blocks", "used_blocks", "shared_blocks", "num_seqs", "logical_tokens")]


def lib():
    """The loaded libpa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m paged_kv_cache_12_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        sig = {
            "pa_status_string": ([i32], ctypes.c_char_p),
            "pa_version": ([], i32),
            "pa_kv_write": ([vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, vp], i32),
            "pa_block_copy": ([vp, vp, vp, i32, i32, i32, i32, i64, vp], i32),
            "pa_decode_workspace_size": ([i32, i32, i32, i32, i32], sz),
            "pa_decode": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i64, i32, i32, ctypes.c_float, vp, sz, vp],
                          i32),
            "pa_workspace_status": ([vp, ctypes.POINTER(i32), vp], i32),
            "pa_alloc_create": ([i64, i32, vp, ctypes.POINTER(vp)], i32),
            "pa_alloc_destroy": ([vp], i32),
            "pa_alloc_add_seq": ([vp, i64], i32),
            "pa_alloc_append": ([vp, i32, vp, vp, vp, vp, i32, ctypes.POINTER(i32)], i32),
            "pa_alloc_fork": ([vp, i64, i64], i32),
            "pa_alloc_free_seq": ([vp, i64], i32),
            "pa_alloc_seq_len": ([vp, i64, ctypes.POINTER(i64)], i32),
            "pa_alloc_block_tables": ([vp, i32, vp, vp, i32, vp], i32),
            "pa_alloc_refcount": ([vp, i64, ctypes.POINTER(ctypes.c_int32)], i32),
            "pa_alloc_stats": ([vp, ctypes.POINTER(AllocStats)], i32),
            "pa_decode_static_ws": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i64, i32, i32,
                                     ctypes.c_float, vp], i32),
            "pa_decode_static_ws_status": ([ctypes.POINTER(i32), vp], i32),
            "pa_alloc_free_queue": ([vp, vp, i64, ctypes.POINTER(i64)], i32),
            "pa_alloc_enable_prefix_cache": ([vp], i32),
            "pa_alloc_match_prefix": ([vp, i64, vp, i32, ctypes.c_uint64, ctypes.POINTER(i32)], i32),
            "pa_alloc_append_ids": ([vp, i32, vp, vp, vp, vp, vp, i32, ctypes.POINTER(i32)], i32),
            "pa_alloc_block_hash": ([vp, i64, vp, ctypes.POINTER(i32)], i32),
            "pa_alloc_prefix_stats": ([vp, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i64)], i32),
            "pa_sha256": ([vp, sz, vp], i32),
            "pa_decode_shared_prefix_workspace_size": ([i32, i32, i32, i32, i32], sz),
            "pa_selftest_wait_timeout": ([ctypes.c_longlong, vp, vp], i32),
            "pa_decode_shared_prefix": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i64, i32, i32,
                                         ctypes.c_float, vp, sz, vp], i32),
            "pa_attention_causal_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
            "pa_kv_write_fp8": ([vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, ctypes.c_float, ctypes.c_float, vp],
                                i32),
            "pa_block_copy_typed": ([vp, vp, vp, i32, i32, i32, i32, i64, i32, vp], i32),
            "pa_decode_typed": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i64, i32, i32, ctypes.c_float, i32,
                                 ctypes.c_float, ctypes.c_float, vp, sz, vp], i32),
            "pa_attention_causal_typed": ([vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i64, i32, i32,
                                           ctypes.c_float, i32, ctypes.c_float, ctypes.c_float, vp, sz, vp], i32),
            "pa_attention_causal": ([vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i64, i32, i32,
                                     ctypes.c_float, vp, sz, vp], i32),
            "pa_latent_write": ([vp, vp, vp, vp, i32, i64, i64, i32, i64, i32, vp], i32),
            "pa_latent_block_copy": ([vp, vp, i32, i32, i64, i32, vp], i32),
            "pa_latent_read": ([vp, vp, vp, vp, vp, i32, i32, i64, i32, i64, i32, i32, vp], i32),
            "pa_latent_attention_workspace_size": ([i32, i32, i32, i32], sz),
            "pa_latent_attention": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i32, i32, ctypes.c_float, i32,
                                     vp, sz, vp], i32),
            "pa_latent_attention_expanded_workspace_size": ([i32, i32, i32], sz),
            "pa_latent_attention_expanded": ([vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i64, i64, i64, i64,
                                              ctypes.c_float, i32, vp, sz, vp], i32),
            "pa_verify_drafts": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i64, i32, vp], i32),
            "pa_kv_write_rope": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i64, i64,
                                  i64, i64, i32, i64, i32, ctypes.c_float, ctypes.c_float, vp], i32),
            "pa_attention_tree_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
            "pa_attention_tree": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i64, i32, i32,
                                   ctypes.c_float, i32, ctypes.c_float, ctypes.c_float, vp, sz, vp], i32),
            "pa_verify_tree": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i32, vp], i32),
            "pa_kv_move_path": ([vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i64, i32, i32, vp], i32),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def status_text(code: int) -> str:
    try:
        return lib().pa_status_string(int(code)).decode()
    except Exception:  # the library itself may be what failed to load
        return "status"


def pa_version() -> int:
    return lib().pa_version()


def pa_status_string(code: int) -> str:
    return lib().pa_status_string(int(code)).decode()


def _check(rc: int, where: str):
    if rc != PA_OK:
        raise PAError(rc, where)


# ---------------------------------------------------------------- device calls

def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t, dtype, ndim, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor with {ndim} dims")


def pa_kv_write(key, value, slot_mapping, k_cache, v_cache, stream=None):
    """Store key[t], value[t] at slot slot_mapping[t] of the caches (slot < 0:
    skipped); fp16 rows into fp16 caches or bf16 rows into bf16 caches (a copy
    of 16-bit elements either way)."""
    import torch
    dt = torch.bfloat16 if k_cache.dtype == torch.bfloat16 else torch.float16
    _need(k_cache, dt, 4, "k_cache")
    _need(v_cache, dt, 4, "v_cache")
    _need(key, dt, 3, "key")
    _need(value, dt, 3, "value")
    _need(slot_mapping, torch.int64, 1, "slot_mapping")
    nb, hkv, bs, d = k_cache.shape
    if v_cache.shape != k_cache.shape or key.shape != value.shape or key.shape[1:] != (hkv, d) \
            or slot_mapping.shape[0] != key.shape[0]:
        raise ValueError("pa_kv_write: shape mismatch")
    _check(lib().pa_kv_write(key.data_ptr(), value.data_ptr(), slot_mapping.data_ptr(), k_cache.data_ptr(),
                             v_cache.data_ptr(), key.shape[0], hkv, d, bs, nb, _stream(stream)), "pa_kv_write")


def kv_dtype_of(cache) -> int:
    """PA_KV_* of a cache tensor: float16, bfloat16, or one-byte E4M3 codes
    (uint8 or torch.float8_e4m3fn)."""
    import torch
    if cache.dtype == torch.float16:
        return PA_KV_F16
    if cache.dtype == torch.bfloat16:
        return PA_KV_BF16
    if cache.dtype == torch.uint8 or cache.dtype == getattr(torch, "float8_e4m3fn", None):
        return PA_KV_FP8_E4M3
    raise ValueError(f"unsupported cache dtype {cache.dtype}")


def _need_cache(t, name, kv):
    import torch
    want = {PA_KV_F16: (torch.float16,), PA_KV_BF16: (torch.bfloat16,),
            PA_KV_FP8_E4M3: (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))}[kv]
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in want or t.dim() != 4 \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous 4-d CUDA cache tensor of {want[0]}")


def pa_block_copy(k_cache, v_cache, pairs, stream=None):
    """Copy every (src, dst) block pair of int64 ``pairs`` [n, 2], K and V
    (caches of fp16, bf16 or fp8 codes)."""
    import torch
    kv = kv_dtype_of(k_cache)
    _need_cache(k_cache, "k_cache", kv)
    _need_cache(v_cache, "v_cache", kv)
    _need(pairs, torch.int64, 2, "pairs")
    nb, hkv, bs, d = k_cache.shape
    if v_cache.shape != k_cache.shape or pairs.shape[1] != 2:
        raise ValueError("pa_block_copy: shape mismatch")
    if kv == PA_KV_F16:
        _check(lib().pa_block_copy(k_cache.data_ptr(), v_cache.data_ptr(), pairs.data_ptr(), pairs.shape[0], hkv, d,
                                   bs, nb, _stream(stream)), "pa_block_copy")
    else:
        _check(lib().pa_block_copy_typed(k_cache.data_ptr(), v_cache.data_ptr(), pairs.data_ptr(), pairs.shape[0],
                                         hkv, d, bs, nb, kv, _stream(stream)), "pa_block_copy_typed")


def pa_kv_write_fp8(key, value, slot_mapping, k_cache, v_cache, k_scale, v_scale, stream=None):
    """Quantise fp16 key/value rows into caches of FP8 E4M3 codes (uint8 or
    float8_e4m3fn tensors): code = E4M3(fl32(x * fl32(1 / scale))), nearest
    value, ties to even, saturating at 448."""
    import torch
    _need_cache(k_cache, "k_cache", PA_KV_FP8_E4M3)
    _need_cache(v_cache, "v_cache", PA_KV_FP8_E4M3)
    _need(key, torch.float16, 3, "key")
    _need(value, torch.float16, 3, "value")
    _need(slot_mapping, torch.int64, 1, "slot_mapping")
    nb, hkv, bs, d = k_cache.shape
    if v_cache.shape != k_cache.shape or key.shape != value.shape or key.shape[1:] != (hkv, d) \
            or slot_mapping.shape[0] != key.shape[0]:
        raise ValueError("pa_kv_write_fp8: shape mismatch")
    _check(lib().pa_kv_write_fp8(key.data_ptr(), value.data_ptr(), slot_mapping.data_ptr(), k_cache.data_ptr(),
                                 v_cache.data_ptr(), key.shape[0], hkv, d, bs, nb, float(k_scale), float(v_scale),
                                 _stream(stream)), "pa_kv_write_fp8")


def pa_decode_typed(out, query, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, workspace,
                    k_scale=1.0, v_scale=1.0, stream=None):
    """pa_decode over a cache of fp16, bf16 (bf16 query/out) or fp8 E4M3 codes
    (fp16 query/out; a code stands for its value times k_scale or v_scale).
    Workspace: pa_decode_workspace_size."""
    import torch
    kv = kv_dtype_of(k_cache)
    qdt = torch.bfloat16 if kv == PA_KV_BF16 else torch.float16
    _need_cache(k_cache, "k_cache", kv)
    _need_cache(v_cache, "v_cache", kv)
    for t, dt, nd, nm in ((out, qdt, 3, "out"), (query, qdt, 3, "query"),
                          (block_tables, torch.int32, 2, "block_tables"), (context_lens, torch.int32, 1, "context_lens"),
                          (workspace, torch.uint8, 1, "workspace")):
        _need(t, dt, nd, nm)
    nb, hkv, bs, d = k_cache.shape
    B, hq, d2 = query.shape
    if out.shape != query.shape or d2 != d or v_cache.shape != k_cache.shape or block_tables.shape[0] != B \
            or context_lens.shape[0] != B:
        raise ValueError("pa_decode_typed: shape mismatch")
    _check(lib().pa_decode_typed(out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                 block_tables.data_ptr(), context_lens.data_ptr(), B, hq, hkv, d, bs, nb,
                                 block_tables.shape[1], int(max_context_len), float(scale), kv, float(k_scale),
                                 float(v_scale), workspace.data_ptr(), workspace.numel(), _stream(stream)),
           "pa_decode_typed")


def pa_attention_causal_typed(out, query, k_cache, v_cache, block_tables, context_lens, query_start, scale,
                              max_context_len, workspace, k_scale=1.0, v_scale=1.0, stream=None):
    """pa_attention_causal over a cache of fp16, bf16 or fp8 E4M3 codes (as
    pa_decode_typed).  Workspace: pa_attention_causal_workspace_size."""
    import torch
    kv = kv_dtype_of(k_cache)
    qdt = torch.bfloat16 if kv == PA_KV_BF16 else torch.float16
    _need_cache(k_cache, "k_cache", kv)
    _need_cache(v_cache, "v_cache", kv)
    for t, dt, nd, nm in ((out, qdt, 3, "out"), (query, qdt, 3, "query"),
                          (block_tables, torch.int32, 2, "block_tables"), (context_lens, torch.int32, 1, "context_lens"),
                          (query_start, torch.int32, 1, "query_start"), (workspace, torch.uint8, 1, "workspace")):
        _need(t, dt, nd, nm)
    nb, hkv, bs, d = k_cache.shape
    nq, hq, d2 = query.shape
    B = context_lens.shape[0]
    if out.shape != query.shape or d2 != d or v_cache.shape != k_cache.shape or block_tables.shape[0] != B \
            or query_start.shape[0] != B + 1:
        raise ValueError("pa_attention_causal_typed: shape mismatch")
    _check(lib().pa_attention_causal_typed(out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                           block_tables.data_ptr(), context_lens.data_ptr(), query_start.data_ptr(),
                                           B, nq, hq, hkv, d, bs, nb, block_tables.shape[1], int(max_context_len),
                                           float(scale), kv, float(k_scale), float(v_scale), workspace.data_ptr(),
                                           workspace.numel(), _stream(stream)), "pa_attention_causal_typed")


def pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len) -> int:
    n = lib().pa_decode_workspace_size(int(num_seqs), int(num_heads), int(num_kv_heads), int(head_dim),
                                       int(max_context_len))
    if n == 0 and num_seqs >= 0:
        raise PAError(PA_ERR_INVALID_ARG, "pa_decode_workspace_size")
    return n


def pa_decode(out, query, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, workspace,
              stream=None):
    """Paged decode attention: out[i][h] = softmax(scale q K^T) V over sequence i's blocks."""
    import torch
    for t, dt, nd, nm in ((out, torch.float16, 3, "out"), (query, torch.float16, 3, "query"),
                          (k_cache, torch.float16, 4, "k_cache"), (v_cache, torch.float16, 4, "v_cache"),
                          (block_tables, torch.int32, 2, "block_tables"), (context_lens, torch.int32, 1, "context_lens"),
                          (workspace, torch.uint8, 1, "workspace")):
        _need(t, dt, nd, nm)
    nb, hkv, bs, d = k_cache.shape
    B, hq, d2 = query.shape
    if out.shape != query.shape or d2 != d or v_cache.shape != k_cache.shape or block_tables.shape[0] != B \
            or context_lens.shape[0] != B:
        raise ValueError("pa_decode: shape mismatch")
    _check(lib().pa_decode(out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                           block_tables.data_ptr(), context_lens.data_ptr(), B, hq, hkv, d, bs, nb,
                           block_tables.shape[1], int(max_context_len), float(scale), workspace.data_ptr(),
                           workspace.numel(), _stream(stream)), "pa_decode")


def pa_decode_static_ws(out, query, k_cache, v_cache, block_tables, context_lens, scale, max_context_len,
                        stream=None):
    """pa_decode without a workspace argument, for callers that cannot allocate
    device memory: the library's own fixed scratch array (64 MiB, shared by all
    calls on a device) stands in for it.  Calls that overlap on the GPU must not
    share it; sizes needing more scratch raise PAError(PA_ERR_WORKSPACE)."""
    import torch
    for t, dt, nd, nm in ((out, torch.float16, 3, "out"), (query, torch.float16, 3, "query"),
                          (k_cache, torch.float16, 4, "k_cache"), (v_cache, torch.float16, 4, "v_cache"),
                          (block_tables, torch.int32, 2, "block_tables"), (context_lens, torch.int32, 1, "context_lens")):
        _need(t, dt, nd, nm)
    nb, hkv, bs, d = k_cache.shape
    B, hq, d2 = query.shape
    if out.shape != query.shape or d2 != d or v_cache.shape != k_cache.shape or block_tables.shape[0] != B \
            or context_lens.shape[0] != B:
        raise ValueError("pa_decode_static_ws: shape mismatch")
    _check(lib().pa_decode_static_ws(out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                     block_tables.data_ptr(), context_lens.data_ptr(), B, hq, hkv, d, bs, nb,
                                     block_tables.shape[1], int(max_context_len), float(scale), _stream(stream)),
           "pa_decode_static_ws")


def pa_decode_static_ws_status(stream=None) -> int:
    """The error word the last pa_decode_static_ws call on the current device
    left in the library's scratch array (PA_OK or PA_ERR_TIMEOUT); synchronises
    the stream."""
    st = ctypes.c_int(0)
    _check(lib().pa_decode_static_ws_status(ctypes.byref(st), _stream(stream)), "pa_decode_static_ws_status")
    return st.value


def pa_decode_shared_prefix_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len) -> int:
    n = lib().pa_decode_shared_prefix_workspace_size(int(num_seqs), int(num_heads), int(num_kv_heads),
                                                     int(head_dim), int(max_context_len))
    if n == 0:
        raise PAError(PA_ERR_INVALID_ARG, "pa_decode_shared_prefix_workspace_size")
    return n


def pa_decode_shared_prefix(out, query, k_cache, v_cache, block_tables, context_lens, group_leader, shared_len,
                            scale, max_context_len, workspace, stream=None):
    """pa_decode where runs of sequences share the blocks of a common prefix:
    group_leader[i] = first sequence of i's group, shared_len[leader] = tokens
    shared (int32 device tensors of num_seqs)."""
    import torch
    for t, dt, nd, nm in ((out, torch.float16, 3, "out"), (query, torch.float16, 3, "query"),
                          (k_cache, torch.float16, 4, "k_cache"), (v_cache, torch.float16, 4, "v_cache"),
                          (block_tables, torch.int32, 2, "block_tables"), (context_lens, torch.int32, 1, "context_lens"),
                          (group_leader, torch.int32, 1, "group_leader"), (shared_len, torch.int32, 1, "shared_len"),
                          (workspace, torch.uint8, 1, "workspace")):
        _need(t, dt, nd, nm)
    nb, hkv, bs, d = k_cache.shape
    B, hq, d2 = query.shape
    if out.shape != query.shape or d2 != d or v_cache.shape != k_cache.shape or block_tables.shape[0] != B \
            or context_lens.shape[0] != B or group_leader.shape[0] != B or shared_len.shape[0] != B:
        raise ValueError("pa_decode_shared_prefix: shape mismatch")
    _check(lib().pa_decode_shared_prefix(out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                         block_tables.data_ptr(), context_lens.data_ptr(), group_leader.data_ptr(),
                                         shared_len.data_ptr(), B, hq, hkv, d, bs, nb, block_tables.shape[1],
                                         int(max_context_len), float(scale), workspace.data_ptr(), workspace.numel(),
                                         _stream(stream)), "pa_decode_shared_prefix")


def pa_attention_causal_workspace_size(num_seqs, num_query_tokens, num_heads, num_kv_heads, head_dim,
                                       max_context_len) -> int:
    n = lib().pa_attention_causal_workspace_size(int(num_seqs), int(num_query_tokens), int(num_heads),
                                                 int(num_kv_heads), int(head_dim), int(max_context_len))
    if n == 0:
        raise PAError(PA_ERR_INVALID_ARG, "pa_attention_causal_workspace_size")
    return n


def pa_attention_causal(out, query, k_cache, v_cache, block_tables, context_lens, query_start, scale,
                        max_context_len, workspace, stream=None):
    """Several new tokens per sequence (chunked prefill, speculative tokens):
    query rows query_start[i] .. query_start[i+1]-1 are sequence i's last new
    tokens, each attending to the positions up to its own."""
    import torch
    for t, dt, nd, nm in ((out, torch.float16, 3, "out"), (query, torch.float16, 3, "query"),
                          (k_cache, torch.float16, 4, "k_cache"), (v_cache, torch.float16, 4, "v_cache"),
                          (block_tables, torch.int32, 2, "block_tables"), (context_lens, torch.int32, 1, "context_lens"),
                          (query_start, torch.int32, 1, "query_start"), (workspace, torch.uint8, 1, "workspace")):
        _need(t, dt, nd, nm)
    nb, hkv, bs, d = k_cache.shape
    nq, hq, d2 = query.shape
    B = context_lens.shape[0]
    if out.shape != query.shape or d2 != d or v_cache.shape != k_cache.shape or block_tables.shape[0] != B \
            or query_start.shape[0] != B + 1:
        raise ValueError("pa_attention_causal: shape mismatch")
    _check(lib().pa_attention_causal(out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                     block_tables.data_ptr(), context_lens.data_ptr(), query_start.data_ptr(), B, nq,
                                     hq, hkv, d, bs, nb, block_tables.shape[1], int(max_context_len), float(scale),
                                     workspace.data_ptr(), workspace.numel(), _stream(stream)), "pa_attention_causal")


def pa_selftest_wait_timeout(limit_cycles: int, status, stream=None):
    """Run the bounded-wait self-test; `status` is an int32 CUDA tensor of one element."""
    import torch
    _need(status, torch.int32, 1, "status")
    _check(lib().pa_selftest_wait_timeout(int(limit_cycles), status.data_ptr(), _stream(stream)),
           "pa_selftest_wait_timeout")


def pa_workspace_status(workspace, stream=None) -> int:
    st = ctypes.c_int(0)
    _check(lib().pa_workspace_status(workspace.data_ptr(), ctypes.byref(st), _stream(stream)), "pa_workspace_status")
    return st.value


# ---------------------------------------------------------------- latent cache

def _refuse(where, dev, t, name, dtype, ndim, how):
    raise ValueError(f"{where}: {name}: expected a {ndim}-d {dtype} tensor on CUDA device {dev}, {how}; got {t.dim()}-d "
                     f"{t.dtype} on {t.device}, strides {t.stride()}")


def _need_on(where, dev, t, name, dtype, ndim):
    """Check one tensor: on CUDA device `dev` (an index), of the type and number
    of dimensions, contiguous.  Decode steps make these calls per layer and each
    question to a tensor takes 50 to 200 ns, so they are asked once and the message
    is made only when it fails."""
    if t.get_device() != dev or dev < 0 or t.dtype is not dtype or t.dim() != ndim or not t.is_contiguous():
        _refuse(where, dev, t, name, dtype, ndim, "contiguous")


def _need_rows(where, dev, t, name, dtype, ndim):
    """The same for a tensor that needs unit stride in its last dimension only;
    gives its strides."""
    st = t.stride()
    if t.get_device() != dev or dev < 0 or t.dtype is not dtype or t.dim() != ndim or \
            (st[-1] != 1 and t.shape[-1] > 1 and t.numel() > 0):
        _refuse(where, dev, t, name, dtype, ndim, "contiguous in its last dimension")
    return st


_raw_stream = _current_device = None


def _run(where, dev, stream, *args):
    """Call the library on device `dev` (an index) and the given stream (default:
    that device's current torch stream)."""
    global _raw_stream, _current_device
    if _raw_stream is None:
        import torch
        # the handle alone, without a Stream object around it, where torch offers it
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda d: torch.cuda.current_stream(d).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if stream is None:
        h = _raw_stream(dev)
    else:
        h = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    f = getattr(_lib or lib(), where)
    if dev == _current_device():
        rc = f(*args, h)
    else:
        import torch
        with torch.cuda.device(dev):
            rc = f(*args, h)
    if rc != PA_OK:
        raise PAError(rc, where)


def _latent_cache(torch, where, cache):
    """(PA_KV_*, torch dtype of the rows that go in and come out, device index,
    blocks, block size) of a latent cache tensor."""
    dt = cache.dtype
    if cache.dim() == 3 and cache.is_contiguous() and cache.is_cuda:
        nb, bs, w = cache.shape
        if dt is torch.uint8 and w == PA_LATENT_ROW_FP8_BYTES:
            return PA_KV_FP8_E4M3, torch.bfloat16, cache.get_device(), nb, bs
        if w == PA_LATENT_ROW and (dt is torch.bfloat16 or dt is torch.float16):
            return (PA_KV_BF16 if dt is torch.bfloat16 else PA_KV_F16), dt, cache.get_device(), nb, bs
    raise ValueError(f"{where}: a latent cache is a contiguous CUDA tensor [num_blocks, block_size, {PA_LATENT_ROW}] "
                     f"float16 or bfloat16, or [num_blocks, block_size, {PA_LATENT_ROW_FP8_BYTES}] uint8")


def pa_latent_write(latent, rope, slot_mapping, cache, stream=None):
    """Write latent[t] ([num_tokens, 512]) and rope[t] ([num_tokens, 64]) to
    slot slot_mapping[t] of a latent cache (slot < 0: skipped); bf16 rows are
    quantised as they go into an FP8 cache.  latent and rope may be slices of
    wider rows (unit stride in the last dimension)."""
    import torch
    where = "pa_latent_write"
    kv, dt, dev, nb, bs = _latent_cache(torch, where, cache)
    sl = _need_rows(where, dev, latent, "latent", dt, 2)[0]
    sr = _need_rows(where, dev, rope, "rope", dt, 2)[0]
    _need_on(where, dev, slot_mapping, "slot_mapping", torch.int64, 1)
    n, w = latent.shape
    if w != PA_LATENT_DIM or rope.shape != (n, PA_LATENT_ROPE_DIM) or slot_mapping.shape[0] != n:
        raise ValueError("pa_latent_write: shape mismatch")
    if n <= 1:   # one row (or none) has no stride of its own
        sl, sr = PA_LATENT_DIM, PA_LATENT_ROPE_DIM
    _run(where, dev, stream, latent.data_ptr(), rope.data_ptr(), slot_mapping.data_ptr(), cache.data_ptr(), n, sl, sr,
         bs, nb, kv)


def pa_latent_block_copy(cache, pairs, stream=None):
    """Copy every (src, dst) block pair of int64 ``pairs`` [n, 2] of a latent cache."""
    import torch
    where = "pa_latent_block_copy"
    kv, _, dev, nb, bs = _latent_cache(torch, where, cache)
    _need_on(where, dev, pairs, "pairs", torch.int64, 2)
    if pairs.shape[1] != 2:
        raise ValueError("pa_latent_block_copy: shape mismatch")
    _run(where, dev, stream, cache.data_ptr(), pairs.data_ptr(), pairs.shape[0], bs, nb, kv)


def pa_latent_read(out, cache, block_tables, row_start, first_token=None, stream=None):
    """Read cached rows back: out[row_start[i] + j] ([num_rows, 576], rows may
    be strided) = token first_token[i] + j (0 + j without first_token) of
    sequence i; rows from row_start[-1] on are left as they are."""
    import torch
    where, i32 = "pa_latent_read", torch.int32
    kv, dt, dev, nb, bs = _latent_cache(torch, where, cache)
    so = _need_rows(where, dev, out, "out", dt, 2)[0]
    _need_on(where, dev, block_tables, "block_tables", i32, 2)
    _need_on(where, dev, row_start, "row_start", i32, 1)
    if first_token is not None:
        _need_on(where, dev, first_token, "first_token", i32, 1)
    n, w = out.shape
    b, mb = block_tables.shape
    if w != PA_LATENT_ROW or row_start.shape[0] != b + 1 or (first_token is not None and first_token.shape[0] != b):
        raise ValueError("pa_latent_read: shape mismatch")
    _run(where, dev, stream, out.data_ptr(), cache.data_ptr(), block_tables.data_ptr(), row_start.data_ptr(),
         None if first_token is None else first_token.data_ptr(), b, n, so if n > 1 else PA_LATENT_ROW, bs,
         nb, mb, kv)


def pa_latent_attention_workspace_size(num_seqs, num_query_tokens, num_heads, max_context_len) -> int:
    n = lib().pa_latent_attention_workspace_size(int(num_seqs), int(num_query_tokens), int(num_heads),
                                                 int(max_context_len))
    if n == 0:
        raise PAError(PA_ERR_INVALID_ARG, "pa_latent_attention_workspace_size")
    return n


def pa_latent_attention(out, query, cache, block_tables, context_lens, scale, max_context_len, workspace,
                        query_start=None, stream=None):
    """Attention over a latent cache, queries multiplied into the latent space:
    out[row][h] ([n, heads, 512]) = softmax(scale q C^T) C[:, :512] over the
    rows C of the sequence, q = query[row][h] ([n, heads, 576]).  Without
    query_start one row per sequence (decode); with it rows query_start[i] ..
    query_start[i + 1] - 1 are sequence i's last new tokens, causal."""
    import torch
    where, i32 = "pa_latent_attention", torch.int32
    kv, dt, dev, nb, bs = _latent_cache(torch, where, cache)
    _need_on(where, dev, out, "out", dt, 3)
    _need_on(where, dev, query, "query", dt, 3)
    _need_on(where, dev, block_tables, "block_tables", i32, 2)
    _need_on(where, dev, context_lens, "context_lens", i32, 1)
    _need_on(where, dev, workspace, "workspace", torch.uint8, 1)
    if query_start is not None:
        _need_on(where, dev, query_start, "query_start", i32, 1)
    nq, h, w = query.shape
    b, mb = block_tables.shape
    if w != PA_LATENT_ROW or out.shape != (nq, h, PA_LATENT_DIM) or context_lens.shape[0] != b or \
            (nq != b if query_start is None else query_start.shape[0] != b + 1):
        raise ValueError("pa_latent_attention: shape mismatch")
    _run(where, dev, stream, out.data_ptr(), query.data_ptr(), cache.data_ptr(), block_tables.data_ptr(),
         context_lens.data_ptr(), None if query_start is None else query_start.data_ptr(), b, nq, h, bs, nb, mb,
         int(max_context_len), float(scale), kv, workspace.data_ptr(), workspace.shape[0])


def pa_latent_attention_expanded_workspace_size(num_seqs, num_query_tokens, num_heads) -> int:
    n = lib().pa_latent_attention_expanded_workspace_size(int(num_seqs), int(num_query_tokens), int(num_heads))
    if n == 0:
        raise PAError(PA_ERR_INVALID_ARG, "pa_latent_attention_expanded_workspace_size")
    return n


def pa_latent_attention_expanded(out, query, k_nope, k_rope, value, query_start, kv_start, scale, workspace,
                                 stream=None):
    """Causal attention over keys and values expanded per head from latents:
    query [nq, heads, 192], k_nope and value [nk, heads, 128] (token and head
    strides free: slices of one product), k_rope [nk, 64] shared by the heads,
    out [nq, heads, 128]; sequence i has rows kv_start[i] .. kv_start[i + 1] - 1
    of the keys, its last new tokens rows query_start[i] .. of the queries."""
    import torch
    where, i32 = "pa_latent_attention_expanded", torch.int32
    dt, dev = query.dtype, query.get_device()
    if dt is not torch.float16 and dt is not torch.bfloat16:
        raise ValueError(f"{where}: query must be float16 or bfloat16")
    _need_on(where, dev, query, "query", dt, 3)
    _need_on(where, dev, out, "out", dt, 3)
    ks = _need_rows(where, dev, k_nope, "k_nope", dt, 3)
    vs = _need_rows(where, dev, value, "value", dt, 3)
    rs = _need_rows(where, dev, k_rope, "k_rope", dt, 2)
    _need_on(where, dev, query_start, "query_start", i32, 1)
    _need_on(where, dev, kv_start, "kv_start", i32, 1)
    _need_on(where, dev, workspace, "workspace", torch.uint8, 1)
    nq, h, w = query.shape
    nk = k_nope.shape[0]
    if w != 192 or out.shape != (nq, h, 128) or k_nope.shape != (nk, h, 128) or value.shape != (nk, h, 128) or \
            k_rope.shape != (nk, 64) or query_start.shape != kv_start.shape or query_start.shape[0] < 1:
        raise ValueError(f"{where}: shape mismatch")

    # a dimension of size one has no stride of its own
    kh, vh = (ks[1], vs[1]) if h > 1 else (128, 128)
    kt, vt = (ks[0], vs[0]) if nk > 1 else (h * kh, h * vh)
    _run(where, dev, stream, out.data_ptr(), query.data_ptr(), k_nope.data_ptr(), k_rope.data_ptr(), value.data_ptr(),
         query_start.data_ptr(), kv_start.data_ptr(), query_start.shape[0] - 1, nq, nk, h, kt, kh,
         rs[0] if nk > 1 else 64, vt, vh, float(scale), PA_KV_F16 if dt is torch.float16 else PA_KV_BF16,
         workspace.data_ptr(), workspace.shape[0])


# ---------------------------------------------------------------- speculative steps

def pa_verify_drafts(accepted, tokens, target_probs, draft_probs, draft_tokens, draft_start, uniform, sample_uniform,
                     stream=None):
    """How many drafted tokens of each sequence stand (accepted [num_seqs]) and
    the tokens that follow (tokens [num_seqs, max_drafts + 1]: those drafts, one
    token drawn from max(p - q, 0) or p, then -1).  target_probs [num_drafts +
    num_seqs, vocab] and draft_probs [num_drafts, vocab] (or None: drafts of
    probability one) are float32, float16 or bfloat16 rows; sequence i's drafts
    are draft_start[i] .. draft_start[i + 1] - 1."""
    import torch
    where, i32, f32 = "pa_verify_drafts", torch.int32, torch.float32
    dt, dev = target_probs.dtype, target_probs.get_device()
    kind = PA_PROBS_F32 if dt is f32 else PA_PROBS_F16 if dt is torch.float16 else \
        PA_PROBS_BF16 if dt is torch.bfloat16 else -1
    if kind < 0:
        raise ValueError(f"{where}: target_probs must be float32, float16 or bfloat16")
    st = _need_rows(where, dev, target_probs, "target_probs", dt, 2)[0]
    _need_on(where, dev, accepted, "accepted", i32, 1)
    _need_on(where, dev, tokens, "tokens", i32, 2)
    _need_on(where, dev, draft_tokens, "draft_tokens", i32, 1)
    _need_on(where, dev, draft_start, "draft_start", i32, 1)
    _need_on(where, dev, uniform, "uniform", f32, 1)
    _need_on(where, dev, sample_uniform, "sample_uniform", f32, 1)
    sd = 0 if draft_probs is None else _need_rows(where, dev, draft_probs, "draft_probs", dt, 2)[0]
    b, nd = accepted.shape[0], draft_tokens.shape[0]
    rows, v = target_probs.shape
    bt, most = tokens.shape
    most -= 1
    if rows != nd + b or bt != b or most < 0 or uniform.shape[0] != nd or \
            draft_start.shape[0] != b + 1 or sample_uniform.shape[0] != b or \
            (draft_probs is not None and draft_probs.shape != (nd, v)):
        raise ValueError(f"{where}: shape mismatch")
    _run(where, dev, stream, accepted.data_ptr(), tokens.data_ptr(), target_probs.data_ptr(),
         None if draft_probs is None else draft_probs.data_ptr(), draft_tokens.data_ptr(), draft_start.data_ptr(),
         uniform.data_ptr(), sample_uniform.data_ptr(), b, nd, most, v, st if rows > 1 else v,
         sd if draft_probs is not None and nd > 1 else v, kind)


# ---------------------------------------------------------------- rotary positions, trees of drafted tokens

# These calls run once a layer and step, and each question to a tensor takes 50 to
# 120 ns: a call asks them in one expression, and only when that fails asks again, one
# by one, for the message.

def _kv_cache_type(torch, where, cache):
    """(PA_KV_*, torch dtype of queries, keys and values) of a K or V cache tensor."""
    dt = cache.dtype
    if dt is torch.bfloat16:
        return PA_KV_BF16, dt
    if dt is torch.float16:
        return PA_KV_F16, dt
    if dt is torch.uint8 or dt is getattr(torch, "float8_e4m3fn", None):
        return PA_KV_FP8_E4M3, torch.float16
    raise ValueError(f"{where}: unsupported cache dtype {dt}")


def _mismatch(where, dev, *tensors):
    """Raise for the first of (tensor, name, dtype, dimensions) that is not a
    contiguous tensor of that kind on the device, else for their shapes."""
    for t, name, dtype, ndim in tensors:
        _need_on(where, dev, t, name, dtype, ndim)
    raise ValueError(f"{where}: shape mismatch")


def _token_stride(where, dev, t, name, dtype, shape):
    """The token stride of [tokens, heads, head_dim] rows whose heads lie side by side (slices of one projection's
    rows, for instance); the tensor must have the shape."""
    n, heads, d = shape
    st = t.stride()
    if t.dtype is not dtype or t.get_device() != dev or dev < 0 or len(st) != 3 or \
            ((st[2] != 1 or st[1] != d) and t.numel() > 0 and ((st[2] != 1 and d > 1) or (st[1] != d and heads > 1))):
        _refuse(where, dev, t, name, dtype, 3, "each token's heads contiguous")
    if t.shape != shape:
        raise ValueError(f"{where}: shape mismatch")
    return st[0] if n > 1 else heads * d


def pa_kv_write_rope(key, value, positions, inv_freq, slot_mapping, k_cache, v_cache, query=None, query_out=None,
                     pair_axis=None, interleaved=False, k_scale=1.0, v_scale=1.0, stream=None):
    """Turn keys and queries to their positions and write keys and values to
    their slots (slot < 0: nothing of the token is written).  key, value
    [tokens, kv_heads, head_dim], query [tokens, heads, head_dim] (token strides
    free), positions int32 [tokens] or [axes, tokens], inv_freq float32
    [rope_dim / 2], pair_axis int32 [rope_dim / 2] (the axis of each pair).  Turned
    queries go to query_out, or to query itself without one."""
    import torch
    where, i32 = "pa_kv_write_rope", torch.int32
    kv, dt = _kv_cache_type(torch, where, k_cache)
    dev, held = k_cache.get_device(), k_cache.shape
    pos, n, pairs = positions.shape, key.shape[0], inv_freq.shape[0]
    if len(held) != 4 or v_cache.shape != held or v_cache.dtype is not k_cache.dtype or v_cache.get_device() != dev or \
            dev < 0 or not k_cache.is_contiguous() or not v_cache.is_contiguous() or \
            positions.dtype is not i32 or positions.get_device() != dev or not positions.is_contiguous() or \
            len(pos) not in (1, 2) or pos[-1] != n or \
            inv_freq.dtype is not torch.float32 or inv_freq.get_device() != dev or inv_freq.stride() != (1,) or \
            slot_mapping.dtype is not torch.int64 or slot_mapping.get_device() != dev or \
            not slot_mapping.is_contiguous() or slot_mapping.shape != (n,):
        _mismatch(where, dev, (k_cache, "k_cache", k_cache.dtype, 4), (v_cache, "v_cache", k_cache.dtype, 4),
                  (positions, "positions", i32, 1 if len(pos) == 1 else 2), (inv_freq, "inv_freq", torch.float32, 1),
                  (slot_mapping, "slot_mapping", torch.int64, 1))
    ax = None
    if pair_axis is not None:
        if pair_axis.dtype is not i32 or pair_axis.get_device() != dev or not pair_axis.is_contiguous() or \
                pair_axis.shape != (pairs,):
            _mismatch(where, dev, (pair_axis, "pair_axis", i32, 1))
        ax = pair_axis.data_ptr()
    nb, hk, bs, d = held
    rows, kst, vst = (n, hk, d), key.stride(), value.stride()
    if key.shape == rows and value.shape == rows and key.dtype is dt and value.dtype is dt and \
            key.get_device() == dev and value.get_device() == dev and kst[2] == 1 and kst[1] == d and vst[2] == 1 and \
            vst[1] == d and n > 1:
        sk, sv = kst[0], vst[0]
    else:
        sk = _token_stride(where, dev, key, "key", dt, rows)
        sv = _token_stride(where, dev, value, "value", dt, rows)
    hq = sq = so = 0
    qi = qo = None
    if query is not None:
        hq = query.shape[1]
        rows, kst = (n, hq, d), query.stride()
        if query.shape == rows and query.dtype is dt and query.get_device() == dev and kst[2] == 1 and kst[1] == d and n > 1:
            sq = so = kst[0]
        else:
            sq = so = _token_stride(where, dev, query, "query", dt, rows)
        qi = qo = query.data_ptr()
        if query_out is not None:
            kst = query_out.stride()
            if query_out.shape == rows and query_out.dtype is dt and query_out.get_device() == dev and kst[2] == 1 and \
                    kst[1] == d and n > 1:
                so = kst[0]
            else:
                so = _token_stride(where, dev, query_out, "query_out", dt, rows)
            qo = query_out.data_ptr()
    elif query_out is not None:
        raise ValueError(f"{where}: query_out without query")
    _run(where, dev, stream, qo, qi, key.data_ptr(), value.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), ax,
         slot_mapping.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), n, hq, hk, d, 2 * pairs,
         1 if len(pos) == 1 else pos[0], 1 if interleaved else 0, sq, so, sk, sv, bs, nb, kv,
         float(k_scale), float(v_scale))


def pa_attention_tree_workspace_size(num_seqs, num_query_tokens, num_heads, num_kv_heads, head_dim,
                                     max_context_len) -> int:
    n = lib().pa_attention_tree_workspace_size(int(num_seqs), int(num_query_tokens), int(num_heads),
                                               int(num_kv_heads), int(head_dim), int(max_context_len))
    if n == 0:
        raise PAError(PA_ERR_INVALID_ARG, "pa_attention_tree_workspace_size")
    return n


def pa_attention_tree(out, query, k_cache, v_cache, block_tables, context_lens, query_start, parents, scale,
                      max_context_len, workspace, k_scale=1.0, v_scale=1.0, stream=None):
    """Attention of trees of drafted tokens: query rows query_start[i] ..
    query_start[i + 1] - 1 are the nodes of sequence i's tree, its last
    positions; each sees the context before the tree, itself and its ancestors
    (parents [num_query_tokens] int32: a smaller node of the sequence, or -1).
    Caches of fp16, bf16 or fp8 E4M3 codes as in pa_attention_causal_typed."""
    import torch
    where, i32 = "pa_attention_tree", torch.int32
    kv, dt = _kv_cache_type(torch, where, k_cache)
    dev, held, rows, tab = k_cache.get_device(), k_cache.shape, query.shape, block_tables.shape
    if len(held) != 4 or v_cache.shape != held or v_cache.dtype is not k_cache.dtype or v_cache.get_device() != dev or \
            dev < 0 or not k_cache.is_contiguous() or not v_cache.is_contiguous() or \
            len(rows) != 3 or rows[2] != held[3] or query.dtype is not dt or query.get_device() != dev or \
            not query.is_contiguous() or \
            out.shape != rows or out.dtype is not dt or out.get_device() != dev or not out.is_contiguous() or \
            len(tab) != 2 or block_tables.dtype is not i32 or block_tables.get_device() != dev or \
            not block_tables.is_contiguous() or \
            context_lens.shape != (tab[0],) or context_lens.dtype is not i32 or context_lens.get_device() != dev or \
            not context_lens.is_contiguous() or \
            query_start.shape != (tab[0] + 1,) or query_start.dtype is not i32 or query_start.get_device() != dev or \
            not query_start.is_contiguous() or \
            parents.shape != (rows[0],) or parents.dtype is not i32 or parents.get_device() != dev or \
            not parents.is_contiguous() or \
            workspace.dtype is not torch.uint8 or workspace.get_device() != dev or workspace.dim() != 1 or \
            not workspace.is_contiguous():
        _mismatch(where, dev, (k_cache, "k_cache", k_cache.dtype, 4), (v_cache, "v_cache", k_cache.dtype, 4),
                  (query, "query", dt, 3), (out, "out", dt, 3), (block_tables, "block_tables", i32, 2),
                  (context_lens, "context_lens", i32, 1), (query_start, "query_start", i32, 1),
                  (parents, "parents", i32, 1), (workspace, "workspace", torch.uint8, 1))
    nb, hk, bs, d = held
    _run(where, dev, stream, out.data_ptr(), query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
         block_tables.data_ptr(), context_lens.data_ptr(), query_start.data_ptr(), parents.data_ptr(), tab[0], rows[0],
         rows[1], hk, d, bs, nb, tab[1], int(max_context_len), float(scale), kv, float(k_scale), float(v_scale),
         workspace.data_ptr(), workspace.shape[0])


def pa_verify_tree(accepted, tokens, path, target_probs, node_tokens, parents, tree_start, uniform, stream=None):
    """The path of each sequence's tree that stands: from node 0 on a token is
    drawn from the node's row of target_probs ([num_nodes, vocab] float32, float16
    or bfloat16) with its `uniform`, and the child with that token follows.
    accepted [num_seqs], tokens and path [num_seqs, max_depth + 1] int32: the
    drafts that stand and the token after them; node 0 and the nodes that stand;
    then -1.  Sequence i's nodes are tree_start[i] .. tree_start[i + 1] - 1."""
    import torch
    where, i32, f32 = "pa_verify_tree", torch.int32, torch.float32
    dt, dev = target_probs.dtype, target_probs.get_device()
    kind = PA_PROBS_F32 if dt is f32 else PA_PROBS_F16 if dt is torch.float16 else \
        PA_PROBS_BF16 if dt is torch.bfloat16 else -1
    if kind < 0:
        raise ValueError(f"{where}: target_probs must be float32, float16 or bfloat16")
    st = _need_rows(where, dev, target_probs, "target_probs", dt, 2)[0]
    n, v = target_probs.shape
    out = tokens.shape
    if len(out) != 2 or out[1] < 1 or tokens.dtype is not i32 or tokens.get_device() != dev or \
            not tokens.is_contiguous() or \
            path.shape != out or path.dtype is not i32 or path.get_device() != dev or not path.is_contiguous() or \
            accepted.shape != (out[0],) or accepted.dtype is not i32 or accepted.get_device() != dev or \
            not accepted.is_contiguous() or \
            node_tokens.shape != (n,) or node_tokens.dtype is not i32 or node_tokens.get_device() != dev or \
            not node_tokens.is_contiguous() or \
            parents.shape != (n,) or parents.dtype is not i32 or parents.get_device() != dev or \
            not parents.is_contiguous() or \
            tree_start.shape != (out[0] + 1,) or tree_start.dtype is not i32 or tree_start.get_device() != dev or \
            not tree_start.is_contiguous() or \
            uniform.shape != (n,) or uniform.dtype is not f32 or uniform.get_device() != dev or \
            not uniform.is_contiguous():
        _mismatch(where, dev, (accepted, "accepted", i32, 1), (tokens, "tokens", i32, 2), (path, "path", i32, 2),
                  (node_tokens, "node_tokens", i32, 1), (parents, "parents", i32, 1), (tree_start, "tree_start", i32, 1),
                  (uniform, "uniform", f32, 1))
    _run(where, dev, stream, accepted.data_ptr(), tokens.data_ptr(), path.data_ptr(), target_probs.data_ptr(),
         node_tokens.data_ptr(), parents.data_ptr(), tree_start.data_ptr(), uniform.data_ptr(), out[0], n, out[1] - 1, v,
         st if n > 1 else v, kind)


def pa_kv_move_path(k_cache, v_cache, block_tables, context_lens, query_start, path, accepted, stream=None):
    """Move K and V of the nodes path[i][0 .. accepted[i]] of each sequence's tree
    (its last query_start[i + 1] - query_start[i] positions) to the positions that
    follow the context before the tree.  Caches of one layer [num_blocks,
    kv_heads, block_size, head_dim] or of several [num_layers, ...]; path
    [num_seqs, max_depth + 1] and accepted as pa_verify_tree wrote them."""
    import torch
    where, i32 = "pa_kv_move_path", torch.int32
    kv, _ = _kv_cache_type(torch, where, k_cache)
    dev, held, tab, ways = k_cache.get_device(), k_cache.shape, block_tables.shape, path.shape
    if len(held) not in (4, 5) or v_cache.shape != held or v_cache.dtype is not k_cache.dtype or \
            v_cache.get_device() != dev or dev < 0 or not k_cache.is_contiguous() or not v_cache.is_contiguous() or \
            len(tab) != 2 or block_tables.dtype is not i32 or block_tables.get_device() != dev or \
            not block_tables.is_contiguous() or \
            context_lens.shape != (tab[0],) or context_lens.dtype is not i32 or context_lens.get_device() != dev or \
            not context_lens.is_contiguous() or \
            query_start.shape != (tab[0] + 1,) or query_start.dtype is not i32 or query_start.get_device() != dev or \
            not query_start.is_contiguous() or \
            len(ways) != 2 or ways[0] != tab[0] or ways[1] < 1 or path.dtype is not i32 or path.get_device() != dev or \
            not path.is_contiguous() or \
            accepted.shape != (tab[0],) or accepted.dtype is not i32 or accepted.get_device() != dev or \
            not accepted.is_contiguous():
        _mismatch(where, dev, (k_cache, "k_cache", k_cache.dtype, 5 if len(held) == 5 else 4),
                  (v_cache, "v_cache", k_cache.dtype, 5 if len(held) == 5 else 4),
                  (block_tables, "block_tables", i32, 2), (context_lens, "context_lens", i32, 1),
                  (query_start, "query_start", i32, 1), (path, "path", i32, 2), (accepted, "accepted", i32, 1))
    nb, hk, bs, d = held[-4:]
    _run(where, dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
         query_start.data_ptr(), path.data_ptr(), accepted.data_ptr(), tab[0], ways[1] - 1,
         held[0] if len(held) == 5 else 1, hk, d, bs, nb, tab[1], kv)


# ---------------------------------------------------------------- allocator

def _i64(a):
    return np.ascontiguousarray(a, dtype=np.int64)


def pa_sha256(data: bytes) -> bytes:
    """SHA-256 of a byte string, as the prefix cache computes it."""
    out = (ctypes.c_uint8 * 32)()
    buf = bytes(data)
    _check(lib().pa_sha256(buf, len(buf), out), "pa_sha256")
    return bytes(out)


class Allocator:
    """Host block allocator (pa_alloc_* calls)."""

    def __init__(self, num_blocks: int, block_size: int, free_order=None, prefix_cache: bool = False):
        self._h = ctypes.c_void_p()
        self.num_blocks, self.block_size = int(num_blocks), int(block_size)
        order = None if free_order is None else np.ascontiguousarray(free_order, dtype=np.int32)
        _check(lib().pa_alloc_create(self.num_blocks, self.block_size,
                                     None if order is None else order.ctypes.data, ctypes.byref(self._h)),
               "pa_alloc_create")
        if prefix_cache:
            _check(lib().pa_alloc_enable_prefix_cache(self._h), "pa_alloc_enable_prefix_cache")

    def close(self):
        if self._h:
            lib().pa_alloc_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_seq(self, seq_id: int):
        _check(lib().pa_alloc_add_seq(self._h, int(seq_id)), "pa_alloc_add_seq")

    def append(self, seq_ids, counts):
        """Reserve slots; returns (slots int64 [sum(counts)], pairs int64 [n, 2])."""
        ids = _i64(seq_ids)
        cnt = np.ascontiguousarray(counts, dtype=np.int32)
        slots = np.empty(max(0, int(cnt[cnt > 0].sum())), dtype=np.int64)
        pairs = np.empty((max(1, len(ids)), 2), dtype=np.int64)
        n = ctypes.c_int(0)
        _check(lib().pa_alloc_append(self._h, len(ids), ids.ctypes.data, cnt.ctypes.data, slots.ctypes.data,
                                     pairs.ctypes.data, pairs.shape[0], ctypes.byref(n)), "pa_alloc_append")
        return slots, pairs[: n.value].copy()

    def append_ids(self, seq_ids, counts, token_ids):
        """append() with the appended tokens' ids (concatenated in sequence order)."""
        ids = _i64(seq_ids)
        cnt = np.ascontiguousarray(counts, dtype=np.int32)
        toks = np.ascontiguousarray(token_ids, dtype=np.int32)
        slots = np.empty(max(0, int(cnt[cnt > 0].sum())), dtype=np.int64)
        pairs = np.empty((max(1, len(ids)), 2), dtype=np.int64)
        n = ctypes.c_int(0)
        _check(lib().pa_alloc_append_ids(self._h, len(ids), ids.ctypes.data, cnt.ctypes.data, toks.ctypes.data,
                                         slots.ctypes.data, pairs.ctypes.data, pairs.shape[0], ctypes.byref(n)),
               "pa_alloc_append_ids")
        return slots, pairs[: n.value].copy()

    def match_prefix(self, seq_id: int, tokens, extra_key: int = 0) -> int:
        """Start seq_id on a prompt, reusing cached full blocks; returns the tokens covered."""
        toks = np.ascontiguousarray(tokens, dtype=np.int32)
        got = ctypes.c_int(0)
        _check(lib().pa_alloc_match_prefix(self._h, int(seq_id), toks.ctypes.data, len(toks),
                                           ctypes.c_uint64(int(extra_key) & (2 ** 64 - 1)), ctypes.byref(got)),
               "pa_alloc_match_prefix")
        return got.value

    def free_queue(self):
        n = ctypes.c_int64(0)
        lib().pa_alloc_free_queue(self._h, None, 0, ctypes.byref(n))
        out = np.empty(n.value, dtype=np.int32)
        _check(lib().pa_alloc_free_queue(self._h, out.ctypes.data, len(out), ctypes.byref(n)), "pa_alloc_free_queue")
        return out.tolist()

    def block_hash(self, block: int):
        h = (ctypes.c_uint8 * 32)()
        c = ctypes.c_int(0)
        _check(lib().pa_alloc_block_hash(self._h, int(block), h, ctypes.byref(c)), "pa_alloc_block_hash")
        return bytes(h), bool(c.value)

    def prefix_stats(self) -> dict:
        c, q, h = ctypes.c_int64(0), ctypes.c_int64(0), ctypes.c_int64(0)
        _check(lib().pa_alloc_prefix_stats(self._h, ctypes.byref(c), ctypes.byref(q), ctypes.byref(h)),
               "pa_alloc_prefix_stats")
        return {"cached_blocks": c.value, "queries": q.value, "hits": h.value}

    def fork(self, parent: int, child: int):
        _check(lib().pa_alloc_fork(self._h, int(parent), int(child)), "pa_alloc_fork")

    def free_seq(self, seq_id: int):
        _check(lib().pa_alloc_free_seq(self._h, int(seq_id)), "pa_alloc_free_seq")

    def seq_len(self, seq_id: int) -> int:
        n = ctypes.c_int64(0)
        _check(lib().pa_alloc_seq_len(self._h, int(seq_id), ctypes.byref(n)), "pa_alloc_seq_len")
        return n.value

    def block_tables(self, seq_ids, max_blocks: int):
        """int32 [n, max_blocks] tables (unused -1) and int32 [n] lengths."""
        ids = _i64(seq_ids)
        tab = np.empty((len(ids), int(max_blocks)), dtype=np.int32)
        lens = np.empty(len(ids), dtype=np.int32)
        _check(lib().pa_alloc_block_tables(self._h, len(ids), ids.ctypes.data, tab.ctypes.data, int(max_blocks),
                                           lens.ctypes.data), "pa_alloc_block_tables")
        return tab, lens

    def refcount(self, block: int) -> int:
        c = ctypes.c_int32(0)
        _check(lib().pa_alloc_refcount(self._h, int(block), ctypes.byref(c)), "pa_alloc_refcount")
        return c.value

    def stats(self) -> dict:
        s = AllocStats()
        _check(lib().pa_alloc_stats(self._h, ctypes.byref(s)), "pa_alloc_stats")
        return {n: getattr(s, n) for n, _ in AllocStats._fields_}
