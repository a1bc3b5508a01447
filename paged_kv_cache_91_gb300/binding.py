"""ctypes binding of libpaged_kv.so (C ABI: include/paged_kv.h).

Argument marshalling only: tensors become device pointers and sizes, the
current torch stream becomes the call's stream, and a non-zero status becomes
a PagedKVError. Every step of the computation runs in the library's kernels;
there is no fallback of any kind, so a missing library raises on first use.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpaged_kv.so")

PKV_F16, PKV_BF16, PKV_FP8_E4M3 = 0, 1, 2
_DTYPE = {torch.float16: PKV_F16, torch.bfloat16: PKV_BF16}
_FP8_DTYPES = (torch.uint8, torch.float8_e4m3fn)  # an FP8 cache: E4M3 codes
DEVERR_BITS = {1: "BLOCK_ID", 2: "CONTEXT", 4: "SLOT", 8: "TIMEOUT", 16: "QUERY", 32: "LAYOUT"}

_lib = None


class PagedKVError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        super().__init__(message)


def load():
    """Load the library (once). Raises PagedKVError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise PagedKVError(None, f"{LIB_PATH} is missing: build it with "
                                 "`python -m paged_kv_cache_91_gb300.build` (or __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.paged_kv_write.restype = i32
    lib.paged_kv_write.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, i32, P]
    lib.paged_attention_workspace_size.restype = sz
    lib.paged_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.paged_attention_decode.restype = i32
    lib.paged_attention_decode.argtypes = [P, P, P, P, P, i32, P, i32, i32, f32, i32, i32, i32, i32, i32, i32,
                                           i32, P, sz, P]
    lib.paged_kv_device_errors.restype = i32
    lib.paged_kv_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
    lib.pkv_status_string.restype = ctypes.c_char_p
    lib.pkv_status_string.argtypes = [i32]
    lib.pkv_last_error_message.restype = ctypes.c_char_p
    lib.pkv_last_error_message.argtypes = []
    lib.paged_kv_copy_blocks.restype = i32
    lib.paged_kv_copy_blocks.argtypes = [P, P, P, i32, i32, i32, i32, i32, i32, P]
    lib.pkv_selftest_wait_timeout.restype = i32
    lib.pkv_selftest_wait_timeout.argtypes = [i64, P]
    lib.paged_kv_write_fp8.restype = i32
    lib.paged_kv_write_fp8.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, i32, f32, f32, P]
    lib.paged_attention_workspace_size_fp8.restype = sz
    lib.paged_attention_workspace_size_fp8.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.paged_attention_multi_query_workspace_size.restype = sz
    lib.paged_attention_multi_query_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.pkv_set_multi_query_tile.restype = i32
    lib.pkv_set_multi_query_tile.argtypes = [i32]
    lib.paged_attention_shared_prefix_workspace_size.restype = sz
    lib.paged_attention_shared_prefix_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.paged_attention_decode_shared_prefix.restype = i32
    lib.paged_attention_decode_shared_prefix.argtypes = [P, P, P, P, P, i32, P, i32, P, i32, i32, f32, i32, i32, i32,
                                                         i32, i32, i32, P, sz, P]
    lib.paged_attention_decode_shared_prefix_fp8.restype = i32
    lib.paged_attention_decode_shared_prefix_fp8.argtypes = [P, P, P, P, P, i32, P, i32, P, i32, i32, f32, i32, i32,
                                                             i32, i32, i32, i32, f32, f32, P, sz, P]
    lib.paged_attention_multi_query.restype = i32
    lib.paged_attention_multi_query.argtypes = [P, P, P, P, P, i32, P, P, i32, i32, i32, i32, f32, i32, i32, i32,
                                                i32, i32, i32, i32, P, sz, P]
    lib.paged_attention_multi_query_fp8.restype = i32
    lib.paged_attention_multi_query_fp8.argtypes = [P, P, P, P, P, i32, P, P, i32, i32, i32, i32, f32, i32, i32,
                                                    i32, i32, i32, i32, f32, f32, i32, P, sz, P]
    lib.paged_attention_decode_fp8.restype = i32
    lib.paged_attention_decode_fp8.argtypes = [P, P, P, P, P, i32, P, i32, i32, f32, i32, i32, i32, i32, i32, i32,
                                               f32, f32, i32, P, sz, P]
    lib.paged_attention_scored_workspace_size.restype = sz
    lib.paged_attention_scored_workspace_size.argtypes = [i32] * 9
    scored = [P, P, P, P, P, i32, P]          # out, query, caches, tables, table width, contexts
    rules = [f32, f32, P, i32, P]             # scale, softcap, slopes, window, key_begin
    shape = [i32, i32, i32, i32, i32, i32]    # block size, heads, kv heads, head dim, blocks, dtype
    work = [i32, P, sz, P]                    # partition, workspace, its bytes, stream
    for name, own in (("decode", [i32, i32] + rules), ("multi_query", [P, i32, i32, i32, i32] + rules + [P])):
        for fp8 in ("", "_fp8"):
            fn = getattr(lib, f"paged_attention_{name}_scored{fp8}")
            fn.restype = i32
            fn.argtypes = scored + own + shape + ([f32, f32] if fp8 else []) + work
    lib.paged_kv_reserve_slots.restype = i32
    lib.paged_kv_reserve_slots.argtypes = [P, i32, P, P, P, i32, P, P, i32, P, P, P, P, i32, i32, i32, P]
    lib.paged_kv_release_blocks.restype = i32
    lib.paged_kv_release_blocks.argtypes = [P, i32, P, P, P, i32, P, P, P, i32, i32, i32, P]
    lib.paged_kv_trim_blocks.restype = i32
    lib.paged_kv_trim_blocks.argtypes = lib.paged_kv_release_blocks.argtypes
    lib.paged_kv_tree_layout.restype = i32
    lib.paged_kv_tree_layout.argtypes = [P, P, P, i32, i32, i32, P, i32, P, P]
    lib.paged_kv_compact_accepted.restype = i32
    lib.paged_kv_compact_accepted.argtypes = [P, P, i32, P, i32, P, P, i32, P, i32, P, i32, i32, i32, i32, i32, P]
    lib.paged_attention_tree_workspace_size.restype = sz
    lib.paged_attention_tree_workspace_size.argtypes = [i32] * 8
    rope = [P] * 9 + [i32, i32, i32, P, P, f32, i32, i64, i64, i64, i32, i32, i32, i32, i32, i32]
    tree = scored + [P, i32, i32, i32, i32, P, i32, f32, f32, P] + shape
    for fp8 in ("", "_fp8"):
        scales = [f32, f32] if fp8 else []
        for name, args in ((f"paged_kv_write_rope{fp8}", rope + scales + [P]),
                           (f"paged_attention_tree{fp8}", tree + scales + work)):
            fn = getattr(lib, name)
            fn.restype = i32
            fn.argtypes = args
    _lib = lib
    return lib


def _check(lib, status: int) -> None:
    if status != 0:
        name = lib.pkv_status_string(status).decode()
        msg = lib.pkv_last_error_message().decode()
        raise PagedKVError(status, f"{name}: {msg}")


def _ptr(t: Optional[torch.Tensor]):
    # the argtypes are c_void_p: a Python int (or None) converts without a wrapper object
    return t.data_ptr() if t is not None else None


# The current stream's handle as an int, without building a torch Stream object (about 2 us per call);
# torch.cuda.current_stream where that accessor is missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor, stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(t.get_device())
        stream = torch.cuda.current_stream(t.device)
    return stream.cuda_stream


def _longest_query(query_start_loc: torch.Tensor, stream) -> int:
    """The longest query, read (and waited for) behind the work that is queued on the call's stream: the offsets may be
    made there."""
    with torch.cuda.stream(_torch_stream(stream, query_start_loc)):
        return int((query_start_loc[1:] - query_start_loc[:-1]).max().item())


def _torch_stream(stream, like: torch.Tensor):
    """The call's stream (None: the current one) as torch's: another library's is known by its handle."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream) and hasattr(stream, "cuda_stream"):
        return torch.cuda.ExternalStream(stream.cuda_stream, device=like.device)
    return stream


def _new_workspace(nbytes: int, like: torch.Tensor, stream) -> torch.Tensor:
    """A workspace for one call on `stream` (None: the current one), from the memory that the allocator keeps for that
    stream: memory freed on another one may still be in use by work queued there, and is given out again only in the
    order of its own stream."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    with torch.cuda.stream(_torch_stream(stream, like)):
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


def _cuda16(name: str, t: torch.Tensor) -> int:
    dt = _DTYPE.get(t.dtype)
    if dt is None or not t.is_cuda or not t.is_contiguous():
        if not t.is_cuda:
            raise PagedKVError(-1, f"{name} must be a CUDA tensor")
        if dt is None:
            raise PagedKVError(-1, f"{name} must be float16 or bfloat16, got {t.dtype}")
        raise PagedKVError(-1, f"{name} must be contiguous")
    return dt


def _cuda_i32(name: str, t: torch.Tensor) -> None:
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise PagedKVError(-1, f"{name} must be a contiguous CUDA int32 tensor")


def _cuda_fp8(name: str, t: torch.Tensor) -> None:
    if not t.is_cuda or t.dtype not in _FP8_DTYPES or not t.is_contiguous():
        raise PagedKVError(-1, f"{name} must be a contiguous CUDA uint8 or float8_e4m3fn tensor (E4M3 codes)")


def _cache_dtype(name: str, t: torch.Tensor) -> int:
    if t.dtype in _FP8_DTYPES:
        _cuda_fp8(name, t)
        return PKV_FP8_E4M3
    return _cuda16(name, t)


def paged_kv_write(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                   slot_mapping: torch.Tensor, stream=None) -> None:
    """Scatter key/value [T][Hkv][D] into the pool [NB][Hkv][B][D] at slot_mapping [T] (int64)."""
    lib = load()
    dt = _cuda16("key_cache", key_cache)
    for n, t in (("key", key), ("value", value), ("value_cache", value_cache)):
        if _cuda16(n, t) != dt:
            raise PagedKVError(-1, f"{n} dtype differs from key_cache")
    if slot_mapping.dtype != torch.int64 or not slot_mapping.is_cuda or not slot_mapping.is_contiguous():
        raise PagedKVError(-1, "slot_mapping must be a contiguous CUDA int64 tensor")
    NB, Hkv, B, D = key_cache.shape
    T = slot_mapping.numel()
    if key.shape != (T, Hkv, D) or value.shape != (T, Hkv, D) or value_cache.shape != key_cache.shape:
        raise PagedKVError(-1, "shape mismatch between key/value, caches and slot_mapping")
    _check(lib, lib.paged_kv_write(_ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache), _ptr(slot_mapping),
                                   T, Hkv, D, B, NB, dt, _stream(key_cache, stream)))


def paged_kv_copy_blocks(key_cache: torch.Tensor, value_cache: torch.Tensor, block_mapping: torch.Tensor,
                         stream=None) -> None:
    """Copy whole physical blocks: block_mapping [num_pairs][2] int64 (src, dst) on the device."""
    lib = load()
    dt = _cache_dtype("key_cache", key_cache)
    if _cache_dtype("value_cache", value_cache) != dt or value_cache.shape != key_cache.shape:
        raise PagedKVError(-1, "value_cache must match key_cache")
    if block_mapping.dtype != torch.int64 or not block_mapping.is_cuda or not block_mapping.is_contiguous():
        raise PagedKVError(-1, "block_mapping must be a contiguous CUDA int64 tensor")
    if block_mapping.numel() % 2:
        raise PagedKVError(-1, "block_mapping must hold (src, dst) pairs")
    NB, Hkv, B, D = key_cache.shape
    _check(lib, lib.paged_kv_copy_blocks(_ptr(key_cache), _ptr(value_cache), _ptr(block_mapping),
                                         block_mapping.numel() // 2, Hkv, D, B, NB, dt, _stream(key_cache, stream)))


def paged_attention_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                   block_size: int, max_context_len: int, partition_size: int = 0) -> int:
    return int(load().paged_attention_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                     max_context_len, partition_size))


def paged_attention_decode(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                           value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                           scale: float, block_size: Optional[int] = None, num_kv_heads: Optional[int] = None,
                           max_context_len: Optional[int] = None, partition_size: int = 0,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode attention: out[s][h] = softmax(scale q.K^T) V over the first context_lens[s] tokens.

    ``max_context_len`` bounds every context length on the host; when omitted it
    is max_blocks_per_seq * block_size (always safe, possibly more partitions).
    ``workspace`` (uint8, >= paged_attention_workspace_size bytes) is allocated
    here through torch when omitted and a split is needed.
    """
    lib = load()
    dt = _cuda16("query", query)
    for n, t in (("out", out), ("key_cache", key_cache), ("value_cache", value_cache)):
        if _cuda16(n, t) != dt:
            raise PagedKVError(-1, f"{n} dtype differs from query")
    _cuda_i32("block_tables", block_tables)
    _cuda_i32("context_lens", context_lens)
    NB, Hkv, B, D = key_cache.shape
    if block_size is not None and block_size != B:
        raise PagedKVError(-1, f"block_size {block_size} != key_cache.shape[2] {B}")
    if num_kv_heads is not None and num_kv_heads != Hkv:
        raise PagedKVError(-1, f"num_kv_heads {num_kv_heads} != key_cache.shape[1] {Hkv}")
    S, H, D2 = query.shape
    if D2 != D or out.shape != query.shape or value_cache.shape != key_cache.shape:
        raise PagedKVError(-1, "shape mismatch between query, out and caches")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise PagedKVError(-1, "block_tables must be [S][max_blocks] and context_lens [S]")
    maxb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = maxb * B
    if workspace is None:  # (a workspace passed in is checked against the size by the library)
        need = int(lib.paged_attention_workspace_size(S, H, Hkv, D, B, max_context_len, partition_size))
        if need:
            workspace = _new_workspace(need, query, stream)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib, lib.paged_attention_decode(
        _ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables), maxb,
        _ptr(context_lens), S, int(max_context_len), float(scale), B, H, Hkv, D, NB, dt, int(partition_size),
        _ptr(workspace), wbytes, _stream(query, stream)))
    return out


def paged_kv_write_fp8(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                       slot_mapping: torch.Tensor, k_scale: float, v_scale: float, stream=None) -> None:
    """Quantizing scatter: key/value [T][Hkv][D] (f16/bf16) into an E4M3 pool [NB][Hkv][B][D]
    (uint8 or float8_e4m3fn): code = E4M3(x / k_scale), likewise for values with v_scale."""
    lib = load()
    dt = _cuda16("key", key)
    if _cuda16("value", value) != dt:
        raise PagedKVError(-1, "value dtype differs from key")
    _cuda_fp8("key_cache", key_cache)
    _cuda_fp8("value_cache", value_cache)
    if slot_mapping.dtype != torch.int64 or not slot_mapping.is_cuda or not slot_mapping.is_contiguous():
        raise PagedKVError(-1, "slot_mapping must be a contiguous CUDA int64 tensor")
    NB, Hkv, B, D = key_cache.shape
    T = slot_mapping.numel()
    if key.shape != (T, Hkv, D) or value.shape != (T, Hkv, D) or value_cache.shape != key_cache.shape:
        raise PagedKVError(-1, "shape mismatch between key/value, caches and slot_mapping")
    _check(lib, lib.paged_kv_write_fp8(_ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache),
                                       _ptr(slot_mapping), T, Hkv, D, B, NB, dt, float(k_scale), float(v_scale),
                                       _stream(key_cache, stream)))


def paged_attention_workspace_size_fp8(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                       block_size: int, max_context_len: int, partition_size: int = 0) -> int:
    return int(load().paged_attention_workspace_size_fp8(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                         max_context_len, partition_size))


def paged_attention_decode_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                               value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                               scale: float, k_scale: float, v_scale: float, max_context_len: Optional[int] = None,
                               partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """paged_attention_decode over an E4M3 pool whose elements are code * k_scale (K) and code * v_scale (V)."""
    lib = load()
    dt = _cuda16("query", query)
    if _cuda16("out", out) != dt:
        raise PagedKVError(-1, "out dtype differs from query")
    _cuda_fp8("key_cache", key_cache)
    _cuda_fp8("value_cache", value_cache)
    _cuda_i32("block_tables", block_tables)
    _cuda_i32("context_lens", context_lens)
    NB, Hkv, B, D = key_cache.shape
    S, H, D2 = query.shape
    if D2 != D or out.shape != query.shape or value_cache.shape != key_cache.shape:
        raise PagedKVError(-1, "shape mismatch between query, out and caches")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise PagedKVError(-1, "block_tables must be [S][max_blocks] and context_lens [S]")
    maxb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = maxb * B
    if workspace is None:
        need = int(lib.paged_attention_workspace_size_fp8(S, H, Hkv, D, B, max_context_len, partition_size))
        if need:
            workspace = _new_workspace(need, query, stream)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib, lib.paged_attention_decode_fp8(
        _ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables), maxb,
        _ptr(context_lens), S, int(max_context_len), float(scale), B, H, Hkv, D, NB, dt, float(k_scale),
        float(v_scale), int(partition_size), _ptr(workspace), wbytes, _stream(query, stream)))
    return out


MQ_TILE_AUTO, MQ_TILE_COLUMNS, MQ_TILE_ROWS, MQ_TILE_TENSOR, MQ_TILE_PAIRS = 0, 1, 2, 3, 4


def set_multi_query_tile(tile: int) -> int:
    """Choose the multi-query tile for later calls (MQ_TILE_*); returns the previous choice."""
    prev = int(load().pkv_set_multi_query_tile(int(tile)))
    if prev < 0:
        raise PagedKVError(-1, f"unknown multi-query tile {tile}")
    return prev


def paged_attention_multi_query_workspace_size(num_query_tokens: int, num_heads: int, num_kv_heads: int,
                                               head_dim: int, block_size: int, max_context_len: int,
                                               partition_size: int = 0) -> int:
    return int(load().paged_attention_multi_query_workspace_size(num_query_tokens, num_heads, num_kv_heads,
                                                                 head_dim, block_size, max_context_len,
                                                                 partition_size))


def _multi_query(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, scale,
                 max_query_len, max_context_len, partition_size, workspace, stream, fp8, k_scale, v_scale):
    lib = load()
    dt = _cuda16("query", query)
    if _cuda16("out", out) != dt:
        raise PagedKVError(-1, "out dtype differs from query")
    for n, t in (("key_cache", key_cache), ("value_cache", value_cache)):
        if fp8:
            _cuda_fp8(n, t)
        elif _cuda16(n, t) != dt:
            raise PagedKVError(-1, f"{n} dtype differs from query")
    _cuda_i32("block_tables", block_tables)
    _cuda_i32("context_lens", context_lens)
    _cuda_i32("query_start_loc", query_start_loc)
    NB, Hkv, B, D = key_cache.shape
    T, H, D2 = query.shape
    S = context_lens.shape[0]
    if D2 != D or out.shape != query.shape or value_cache.shape != key_cache.shape:
        raise PagedKVError(-1, "shape mismatch between query, out and caches")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or query_start_loc.shape != (S + 1,):
        raise PagedKVError(-1, "block_tables must be [S][max_blocks] and query_start_loc [S + 1]")
    maxb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = maxb * B
    if max_query_len is None:
        max_query_len = _longest_query(query_start_loc, stream) if S else 0
    if workspace is None:
        need = int(lib.paged_attention_multi_query_workspace_size(T, H, Hkv, D, B, max_context_len,
                                                                  partition_size))
        if need:
            workspace = _new_workspace(need, query, stream)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    head = (_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables), maxb,
            _ptr(context_lens), _ptr(query_start_loc), S, T, int(max_query_len), int(max_context_len), float(scale),
            B, H, Hkv, D, NB, dt)
    tail = (int(partition_size), _ptr(workspace), wbytes, _stream(query, stream))
    if fp8:
        _check(lib, lib.paged_attention_multi_query_fp8(*head, float(k_scale), float(v_scale), *tail))
    else:
        _check(lib, lib.paged_attention_multi_query(*head, *tail))
    return out


def paged_attention_multi_query(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                                query_start_loc: torch.Tensor, scale: float, max_query_len: Optional[int] = None,
                                max_context_len: Optional[int] = None, partition_size: int = 0,
                                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention of several query tokens per sequence (query/out [T][H][D], packed by
    query_start_loc [S+1] int32): sequence s's q_len tokens are its last q_len context positions.

    ``max_query_len`` bounds every q_len on the host; when omitted it is read from
    query_start_loc, which synchronises the call's stream.
    """
    return _multi_query(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, scale,
                        max_query_len, max_context_len, partition_size, workspace, stream, False, 1.0, 1.0)


def paged_attention_multi_query_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                    value_cache: torch.Tensor, block_tables: torch.Tensor,
                                    context_lens: torch.Tensor, query_start_loc: torch.Tensor, scale: float,
                                    k_scale: float, v_scale: float, max_query_len: Optional[int] = None,
                                    max_context_len: Optional[int] = None, partition_size: int = 0,
                                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """paged_attention_multi_query over an E4M3 pool whose elements are code * k_scale (K) and
    code * v_scale (V); head_dim 128."""
    return _multi_query(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, scale,
                        max_query_len, max_context_len, partition_size, workspace, stream, True, k_scale, v_scale)


def paged_attention_shared_prefix_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                                 block_size: int, prefix_len: int, max_tail_len: int) -> int:
    return int(load().paged_attention_shared_prefix_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                                   block_size, prefix_len, max_tail_len))


def _shared_prefix(out, query, key_cache, value_cache, prefix_blocks, prefix_len, block_tables, tail_lens, scale,
                   max_tail_len, workspace, stream, fp8, k_scale, v_scale):
    lib = load()
    dt = _cuda16("query", query)
    if _cuda16("out", out) != dt:
        raise PagedKVError(-1, "out dtype differs from query")
    for n, t in (("key_cache", key_cache), ("value_cache", value_cache)):
        if fp8:
            _cuda_fp8(n, t)
        elif _cuda16(n, t) != dt:
            raise PagedKVError(-1, f"{n} dtype differs from query")
    _cuda_i32("prefix_blocks", prefix_blocks)
    _cuda_i32("block_tables", block_tables)
    _cuda_i32("tail_lens", tail_lens)
    NB, Hkv, B, D = key_cache.shape
    S, H, D2 = query.shape
    if D2 != D or out.shape != query.shape or value_cache.shape != key_cache.shape:
        raise PagedKVError(-1, "shape mismatch between query, out and caches")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or tail_lens.shape != (S,):
        raise PagedKVError(-1, "block_tables must be [S][max_blocks] and tail_lens [S]")
    maxb = block_tables.shape[1]
    if max_tail_len is None:
        max_tail_len = maxb * B
    if workspace is None:
        need = paged_attention_shared_prefix_workspace_size(S, H, Hkv, D, B, int(prefix_len), int(max_tail_len))
        workspace = _new_workspace(max(need, 16), query, stream)
    wbytes = workspace.numel() * workspace.element_size()
    head = (_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(prefix_blocks), int(prefix_len),
            _ptr(block_tables), maxb, _ptr(tail_lens), S, int(max_tail_len), float(scale), B, H, Hkv, D, NB, dt)
    tail = (_ptr(workspace), wbytes, _stream(query, stream))
    if fp8:
        _check(lib, lib.paged_attention_decode_shared_prefix_fp8(*head, float(k_scale), float(v_scale), *tail))
    else:
        _check(lib, lib.paged_attention_decode_shared_prefix(*head, *tail))
    return out


def paged_attention_decode_shared_prefix(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                         value_cache: torch.Tensor, prefix_blocks: torch.Tensor, prefix_len: int,
                                         block_tables: torch.Tensor, tail_lens: torch.Tensor, scale: float,
                                         max_tail_len: Optional[int] = None,
                                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode for sequences that share their first prefix_len tokens (prefix_blocks [prefix_len / B] int32);
    block_tables [S][max] and tail_lens [S] describe each sequence's tokens after the prefix. Same result as
    paged_attention_decode over prefix_blocks ++ block_tables[s], with the prefix read once."""
    return _shared_prefix(out, query, key_cache, value_cache, prefix_blocks, prefix_len, block_tables, tail_lens,
                          scale, max_tail_len, workspace, stream, False, 1.0, 1.0)


def paged_attention_decode_shared_prefix_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                             value_cache: torch.Tensor, prefix_blocks: torch.Tensor,
                                             prefix_len: int, block_tables: torch.Tensor, tail_lens: torch.Tensor,
                                             scale: float, k_scale: float, v_scale: float,
                                             max_tail_len: Optional[int] = None,
                                             workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """paged_attention_decode_shared_prefix over an E4M3 pool (elements code * k_scale, code * v_scale)."""
    return _shared_prefix(out, query, key_cache, value_cache, prefix_blocks, prefix_len, block_tables, tail_lens,
                          scale, max_tail_len, workspace, stream, True, k_scale, v_scale)


def paged_attention_scored_workspace_size(num_query_tokens: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                          block_size: int, max_query_len: int, max_context_len: int, window: int = 0,
                                          partition_size: int = 0) -> int:
    return int(load().paged_attention_scored_workspace_size(num_query_tokens, num_heads, num_kv_heads, head_dim,
                                                            block_size, max_query_len, max_context_len, window,
                                                            partition_size))


# The current device's index, without torch.cuda's lazy initialisation test (a CUDA tensor exists by then).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _expect(name: str, t: torch.Tensor, dtype: torch.dtype, dev: int) -> None:
    """t must be a contiguous tensor of this type on CUDA device dev."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        if not t.is_cuda:
            raise PagedKVError(-1, f"{name} must be a CUDA tensor")
        if t.get_device() != dev:
            raise PagedKVError(-1, f"{name} is on {t.device}, other tensors of the call on cuda:{dev}")
        if t.dtype is not dtype:
            raise PagedKVError(-1, f"{name} must be {dtype}, got {t.dtype}")
        raise PagedKVError(-1, f"{name} must be contiguous")


def _expect_all(dev: int, names: str, tensors, dtypes) -> None:
    """Each tensor (or None) must be contiguous, of its type and on CUDA device dev (names: theirs, for the message)."""
    for t, dtype in zip(tensors, dtypes):
        if t is not None and (t.dtype is not dtype or t.get_device() != dev or dev < 0 or not t.is_contiguous()):
            for name, x, d in zip(names.split(), tensors, dtypes):
                if x is None:
                    continue
                if not x.is_cuda:
                    raise PagedKVError(-1, f"{name} must be a CUDA tensor")
                _expect(name, x, d, dev)


def _pool_dtype(key_cache, value_cache, dtype, fp8):
    """The caches' type: the queries', or their own 8-bit one."""
    if not fp8:
        return dtype
    if key_cache.dtype not in _FP8_DTYPES or value_cache.dtype is not key_cache.dtype:
        _cuda_fp8("key_cache", key_cache)
        _cuda_fp8("value_cache", value_cache)
        raise PagedKVError(-1, f"value_cache is {value_cache.dtype}, key_cache {key_cache.dtype}")
    return key_cache.dtype


_I32 = (torch.int32,) * 5


def _run_on(dev: int, stream, fn, args) -> None:
    """fn(*args, stream handle) with device dev current (the library launches on the current device)."""
    if stream is not None:
        handle = stream.cuda_stream
    elif _raw_stream is not None:
        handle = _raw_stream(dev)
    else:
        handle = torch.cuda.current_stream(dev).cuda_stream
    if dev == _current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status:
        _check(_lib, status)


# These checks run on every call, and a small call is bound by them: each tensor's type, device and layout are
# tested in one expression, and the reasons are looked for only when one fails.
def _scored(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, scale, softcap,
            alibi_slopes, window, key_begin, key_end, max_query_len, max_context_len, partition_size, workspace,
            stream, fp8, k_scale, v_scale):
    lib = _lib or load()
    dtype = query.dtype
    dt = _DTYPE.get(dtype)
    dev = query.get_device()
    if dt is None or dev < 0 or not query.is_contiguous():
        _cuda16("query", query)
    if fp8:
        _expect("out", out, dtype, dev)
        for n, t in (("key_cache", key_cache), ("value_cache", value_cache)):
            _cuda_fp8(n, t)
            _expect(n, t, t.dtype, dev)
    else:
        for t in (out, key_cache, value_cache):
            if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
                for n, x in (("out", out), ("key_cache", key_cache), ("value_cache", value_cache)):
                    _expect(n, x, dtype, dev)
    _expect("block_tables", block_tables, torch.int32, dev)
    _expect("context_lens", context_lens, torch.int32, dev)
    shape, pool, tables = query.shape, key_cache.shape, block_tables.shape
    if len(pool) != 4 or len(shape) != 3 or len(tables) != 2:
        raise PagedKVError(-1, "key_cache must be [blocks][kv heads][block size][head dim], query [rows][heads][head "
                               "dim] and block_tables [S][max_blocks]")
    NB, Hkv, B, D = pool
    T, H, D2 = shape
    S, maxb = tables
    if D2 != D or out.shape != shape or value_cache.shape != pool:
        raise PagedKVError(-1, "shape mismatch between query, out and caches")
    if context_lens.shape != (S,):
        raise PagedKVError(-1, "block_tables must be [S][max_blocks] and context_lens [S]")
    if query_start_loc is None:
        if T != S:
            raise PagedKVError(-1, f"query has {T} rows for {S} sequences")
        max_query_len = 1
    else:
        _expect("query_start_loc", query_start_loc, torch.int32, dev)
        if query_start_loc.shape != (S + 1,):
            raise PagedKVError(-1, "query_start_loc must be [S + 1]")
        if max_query_len is None:
            max_query_len = _longest_query(query_start_loc, stream) if S else 0
    slopes = begin = end = ws = None
    if alibi_slopes is not None:
        _expect("alibi_slopes", alibi_slopes, torch.float32, dev)
        if alibi_slopes.shape != (H,):
            raise PagedKVError(-1, "alibi_slopes must have one entry per head")
        slopes = alibi_slopes.data_ptr()
    if key_begin is not None:
        _expect("key_begin", key_begin, torch.int32, dev)
        if key_begin.shape != (T,):
            raise PagedKVError(-1, "key_begin must have one entry per query row")
        begin = key_begin.data_ptr()
    if key_end is not None:
        _expect("key_end", key_end, torch.int32, dev)
        if key_end.shape != (T,):
            raise PagedKVError(-1, "key_end must have one entry per query row")
        end = key_end.data_ptr()
    if max_context_len is None:
        max_context_len = maxb * B
    wbytes = 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise PagedKVError(-1, "workspace must be a contiguous tensor on the query's device")
        wbytes = workspace.numel() * workspace.element_size()
    else:
        wbytes = lib.paged_attention_scored_workspace_size(T, H, Hkv, D, B, max_query_len, max_context_len, window,
                                                           partition_size)
        if wbytes:
            workspace = _new_workspace(wbytes, query, stream)
    if workspace is not None:
        ws = workspace.data_ptr()
    scales = (k_scale, v_scale) if fp8 else ()
    if query_start_loc is None:
        _run_on(dev, stream, lib.paged_attention_decode_scored_fp8 if fp8 else lib.paged_attention_decode_scored,
                (out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                 block_tables.data_ptr(), maxb, context_lens.data_ptr(), S, max_context_len, scale, softcap, slopes,
                 window, begin, B, H, Hkv, D, NB, dt, *scales, partition_size, ws, wbytes))
    else:
        _run_on(dev, stream,
                lib.paged_attention_multi_query_scored_fp8 if fp8 else lib.paged_attention_multi_query_scored,
                (out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                 block_tables.data_ptr(), maxb, context_lens.data_ptr(), query_start_loc.data_ptr(), S, T,
                 max_query_len, max_context_len, scale, softcap, slopes, window, begin, end, B, H, Hkv, D, NB, dt,
                 *scales, partition_size, ws, wbytes))
    return out


def paged_attention_decode_scored(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                  value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                                  scale: float, softcap: float = 0.0, alibi_slopes: Optional[torch.Tensor] = None,
                                  window: int = 0, key_begin: Optional[torch.Tensor] = None,
                                  max_context_len: Optional[int] = None, partition_size: int = 0,
                                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """paged_attention_decode with capped scores (``softcap`` > 0), a distance bias (``alibi_slopes`` [H] fp32), a
    sliding ``window`` (0: none) and a first visible key per sequence (``key_begin`` [S] int32)."""
    return _scored(out, query, key_cache, value_cache, block_tables, context_lens, None, scale, softcap,
                   alibi_slopes, window, key_begin, None, 1, max_context_len, partition_size, workspace, stream,
                   False, 1.0, 1.0)


def paged_attention_decode_scored_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                      value_cache: torch.Tensor, block_tables: torch.Tensor,
                                      context_lens: torch.Tensor, scale: float, k_scale: float, v_scale: float,
                                      softcap: float = 0.0, alibi_slopes: Optional[torch.Tensor] = None,
                                      window: int = 0, key_begin: Optional[torch.Tensor] = None,
                                      max_context_len: Optional[int] = None, partition_size: int = 0,
                                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """paged_attention_decode_scored over an E4M3 pool (elements code * k_scale, code * v_scale); head_dim 128."""
    return _scored(out, query, key_cache, value_cache, block_tables, context_lens, None, scale, softcap,
                   alibi_slopes, window, key_begin, None, 1, max_context_len, partition_size, workspace, stream,
                   True, k_scale, v_scale)


def paged_attention_multi_query_scored(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                       value_cache: torch.Tensor, block_tables: torch.Tensor,
                                       context_lens: torch.Tensor, query_start_loc: torch.Tensor, scale: float,
                                       softcap: float = 0.0, alibi_slopes: Optional[torch.Tensor] = None,
                                       window: int = 0, key_begin: Optional[torch.Tensor] = None,
                                       key_end: Optional[torch.Tensor] = None, max_query_len: Optional[int] = None,
                                       max_context_len: Optional[int] = None, partition_size: int = 0,
                                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """paged_attention_multi_query with the scores of paged_attention_decode_scored; query token t sees the keys
    [key_begin[t], key_end[t]) (int32 [T]; default: from 0, to its own position), cut by the window and the context.

    ``max_query_len`` bounds every query length on the host; when omitted it is read from query_start_loc, which
    synchronises the call's stream.
    """
    return _scored(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, scale, softcap,
                   alibi_slopes, window, key_begin, key_end, max_query_len, max_context_len, partition_size,
                   workspace, stream, False, 1.0, 1.0)


def paged_attention_multi_query_scored_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                           value_cache: torch.Tensor, block_tables: torch.Tensor,
                                           context_lens: torch.Tensor, query_start_loc: torch.Tensor, scale: float,
                                           k_scale: float, v_scale: float, softcap: float = 0.0,
                                           alibi_slopes: Optional[torch.Tensor] = None, window: int = 0,
                                           key_begin: Optional[torch.Tensor] = None,
                                           key_end: Optional[torch.Tensor] = None,
                                           max_query_len: Optional[int] = None,
                                           max_context_len: Optional[int] = None, partition_size: int = 0,
                                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """paged_attention_multi_query_scored over an E4M3 pool (elements code * k_scale, code * v_scale); head_dim 128."""
    return _scored(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, scale, softcap,
                   alibi_slopes, window, key_begin, key_end, max_query_len, max_context_len, partition_size,
                   workspace, stream, True, k_scale, v_scale)


def _pool_arrays(block_tables, context_lens, lens_name, lens, free_blocks, num_free, context_lens_out, num_free_out):
    """Check the arrays that the reserve and release calls share; returns (sequences, table width, device)."""
    dev = block_tables.get_device()
    i32 = torch.int32
    for t in (block_tables, context_lens, lens, free_blocks, num_free, context_lens_out, num_free_out):
        if t.dtype is not i32 or t.get_device() != dev or dev < 0 or not t.is_contiguous():
            for n, x in (("block_tables", block_tables), ("context_lens", context_lens), (lens_name, lens),
                         ("free_blocks", free_blocks), ("num_free", num_free),
                         ("context_lens_out", context_lens_out), ("num_free_out", num_free_out)):
                _cuda_i32(n, x)
                _expect(n, x, i32, dev)
    tables = block_tables.shape
    if len(tables) != 2:
        raise PagedKVError(-1, "block_tables must be [S][max_blocks]")
    S, maxb = tables
    if context_lens.shape != (S,) or lens.shape != (S,) or context_lens_out.shape != (S,):
        raise PagedKVError(-1, f"context_lens, {lens_name} and context_lens_out must be [S]")
    if free_blocks.dim() != 1 or num_free.numel() != 1 or num_free_out.numel() != 1:
        raise PagedKVError(-1, "free_blocks must be a vector, num_free and num_free_out one element")
    return S, maxb, dev


def paged_kv_reserve_slots(block_tables: torch.Tensor, context_lens: torch.Tensor, new_lens: torch.Tensor,
                           free_blocks: torch.Tensor, num_free: torch.Tensor, slot_mapping: torch.Tensor,
                           query_start_loc: torch.Tensor, context_lens_out: torch.Tensor,
                           num_free_out: torch.Tensor, granted: torch.Tensor, block_size: int, num_blocks: int,
                           stream=None) -> None:
    """Slots for new_lens[s] more tokens of each sequence, with blocks from the top of the free stack
    free_blocks[:num_free]: updates block_tables in place and writes slot_mapping [max_tokens] int64 (-1: padding,
    or a sequence that got nothing), query_start_loc [S + 1], context_lens_out [S], num_free_out [1] and granted [S].
    What is written must not overlap anything else of the call.

    A sequence that got nothing keeps its query tokens and its context. For the scored attention calls, pass the
    contexts context_lens + new_lens and a key_begin of 2**31 - 1 for the query tokens whose slot is -1: their rows
    are zeros, and granted need not be read on the host before the step's end."""
    lib = _lib or load()
    S, maxb, dev = _pool_arrays(block_tables, context_lens, "new_lens", new_lens, free_blocks, num_free,
                                context_lens_out, num_free_out)
    _expect("query_start_loc", query_start_loc, torch.int32, dev)
    _expect("granted", granted, torch.int32, dev)
    _expect("slot_mapping", slot_mapping, torch.int64, dev)
    if query_start_loc.shape != (S + 1,) or granted.shape != (S,):
        raise PagedKVError(-1, "query_start_loc must be [S + 1] and granted [S]")
    _run_on(dev, stream, lib.paged_kv_reserve_slots,
            (block_tables.data_ptr(), maxb, context_lens.data_ptr(), new_lens.data_ptr(), free_blocks.data_ptr(),
             free_blocks.numel(), num_free.data_ptr(), slot_mapping.data_ptr(), slot_mapping.numel(),
             query_start_loc.data_ptr(), context_lens_out.data_ptr(), num_free_out.data_ptr(), granted.data_ptr(), S,
             block_size, num_blocks))


def paged_kv_release_blocks(block_tables: torch.Tensor, context_lens: torch.Tensor, finished: torch.Tensor,
                            free_blocks: torch.Tensor, num_free: torch.Tensor, context_lens_out: torch.Tensor,
                            num_free_out: torch.Tensor, block_size: int, num_blocks: int, stream=None) -> None:
    """Push the blocks of the sequences with finished[s] != 0 on the free stack free_blocks (in place), and write
    context_lens_out [S] (0 for them) and num_free_out [1]. What is written must not overlap anything else of the call."""
    lib = _lib or load()
    S, maxb, dev = _pool_arrays(block_tables, context_lens, "finished", finished, free_blocks, num_free,
                                context_lens_out, num_free_out)
    _run_on(dev, stream, lib.paged_kv_release_blocks,
            (block_tables.data_ptr(), maxb, context_lens.data_ptr(), finished.data_ptr(), free_blocks.data_ptr(),
             free_blocks.numel(), num_free.data_ptr(), context_lens_out.data_ptr(), num_free_out.data_ptr(), S,
             block_size, num_blocks))


def _qkv_rows(name: str, t: torch.Tensor, dtype: torch.dtype, dev: int, tokens: int, heads: int, dim: int) -> int:
    """The elements between tokens of t [tokens][heads][dim], whose tokens' rows are contiguous."""
    if t.dtype is not dtype or t.get_device() != dev:
        if not t.is_cuda:
            raise PagedKVError(-1, f"{name} must be a CUDA tensor")
        if t.get_device() != dev:
            raise PagedKVError(-1, f"{name} is on {t.device}, other tensors of the call on cuda:{dev}")
        raise PagedKVError(-1, f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (tokens, heads, dim):
        raise PagedKVError(-1, f"{name} must be [{tokens}][{heads}][{dim}], got {list(t.shape)}")
    per_token, per_head, one = t.stride()
    if one != 1 or (per_head != dim and heads > 1):
        raise PagedKVError(-1, f"{name}: each token's heads must be contiguous")
    return per_token if tokens > 1 else heads * dim


def _write_rope(query_out, query, key, value, key_cache, value_cache, slot_mapping, positions, cos_sin, q_weight,
                k_weight, eps, interleaved, stream, fp8, scales):
    lib = _lib or load()
    dtype = query.dtype
    dt = _DTYPE.get(dtype)
    dev = query.get_device()
    if dt is None or dev < 0:
        _cuda16("query", query)
    stored, f32 = _pool_dtype(key_cache, value_cache, dtype, fp8), torch.float32
    _expect_all(dev, "key_cache value_cache query_out slot_mapping positions cos_sin q_weight k_weight",
                (key_cache, value_cache, query_out, slot_mapping, positions, cos_sin, q_weight, k_weight),
                (stored, stored, dtype, torch.int64, torch.int32, f32, f32, f32))
    pool, shape = key_cache.shape, query.shape
    if len(pool) != 4 or len(shape) != 3 or value_cache.shape != pool:
        raise PagedKVError(-1, "the caches must be [blocks][kv heads][block size][head dim], query [tokens][heads][head "
                               "dim]")
    NB, Hkv, B, D = pool
    T, H, D2 = shape
    if D2 != D:
        raise PagedKVError(-1, f"head dim {D2} of query, {D} of the caches")
    if query_out.shape != shape:
        raise PagedKVError(-1, "query_out must have query's shape")
    kv = (T, Hkv, D)
    qs, ks, vs = query.stride(), key.stride(), value.stride()
    if (T < 2 or H < 2 or Hkv < 2 or key.shape != kv or value.shape != kv or key.dtype is not dtype
            or value.dtype is not dtype or key.get_device() != dev or value.get_device() != dev
            or qs[1:] != (D, 1) or ks[1:] != (D, 1) or vs[1:] != (D, 1)):
        q_step, k_step, v_step = (_qkv_rows("query", query, dtype, dev, T, H, D),
                                  _qkv_rows("key", key, dtype, dev, T, Hkv, D),
                                  _qkv_rows("value", value, dtype, dev, T, Hkv, D))
    else:
        q_step, k_step, v_step = qs[0], ks[0], vs[0]
    if slot_mapping.shape != (T,):
        raise PagedKVError(-1, "slot_mapping must have one entry per token")
    at = angles = qw = kw = None
    rotary = most = 0
    if (positions is None) != (cos_sin is None):
        raise PagedKVError(-1, "positions and cos_sin go together")
    if cos_sin is not None:
        if positions.shape != (T,) or cos_sin.dim() != 2:
            raise PagedKVError(-1, "positions must have one entry per token, cos_sin be [max_position][rotary_dim]")
        most, rotary = cos_sin.shape
        at, angles = positions.data_ptr(), cos_sin.data_ptr()
    if q_weight is not None:
        if q_weight.shape != (D,):
            raise PagedKVError(-1, "q_weight must have one entry per dim of a head")
        qw = q_weight.data_ptr()
    if k_weight is not None:
        if k_weight.shape != (D,):
            raise PagedKVError(-1, "k_weight must have one entry per dim of a head")
        kw = k_weight.data_ptr()
    _run_on(dev, stream, lib.paged_kv_write_rope_fp8 if fp8 else lib.paged_kv_write_rope,
            (query_out.data_ptr(), query.data_ptr(), key.data_ptr(), value.data_ptr(), key_cache.data_ptr(),
             value_cache.data_ptr(), slot_mapping.data_ptr(), at, angles, most, rotary, 1 if interleaved else 0, qw, kw,
             eps, T, q_step, k_step, v_step, H, Hkv, D, B, NB, dt, *scales))
    return query_out


def paged_kv_write_rope(query_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                        key_cache: torch.Tensor, value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                        positions: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor],
                        q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                        eps: float = 1e-6, interleaved: bool = False, stream=None) -> torch.Tensor:
    """paged_kv_write of keys normed per head (``k_weight`` [D] fp32; None: not normed) and rotated by ``positions``
    [T] int32, and the same for the queries (into query_out, which may be query itself). ``cos_sin``
    [max_position][rotary_dim] fp32 holds a position's cosines, then its sines; both None: no rotation. query, key and
    value [T][heads][D] may be slices of one projection's output; pairs are (i, i + rotary_dim / 2), or (2i, 2i + 1)
    if ``interleaved``."""
    return _write_rope(query_out, query, key, value, key_cache, value_cache, slot_mapping, positions, cos_sin, q_weight,
                       k_weight, eps, interleaved, stream, False, ())


def paged_kv_write_rope_fp8(query_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                            key_cache: torch.Tensor, value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                            positions: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor], k_scale: float,
                            v_scale: float, q_weight: Optional[torch.Tensor] = None,
                            k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                            stream=None) -> torch.Tensor:
    """paged_kv_write_rope into an E4M3 pool: code = E4M3(x / k_scale) of the rotated keys, likewise for values with
    v_scale."""
    return _write_rope(query_out, query, key, value, key_cache, value_cache, slot_mapping, positions, cos_sin, q_weight,
                       k_weight, eps, interleaved, stream, True, (k_scale, v_scale))


def paged_kv_tree_layout(parents: torch.Tensor, query_start_loc: torch.Tensor, context_lens: torch.Tensor,
                         tree_mask: torch.Tensor, positions: torch.Tensor, max_query_len: Optional[int] = None,
                         stream=None) -> None:
    """Masks and positions of drafted trees: from each token's parent ([T] int32, its node in the same tree, < 0: a
    root) writes tree_mask [T][words] int32 (the bits of the token itself and its ancestors) and positions [T] int32
    (committed tokens + depth). context_lens count the drafted tokens.

    ``max_query_len`` bounds every tree on the host (at most 1024); when omitted it is read from query_start_loc, which
    synchronises the call's stream.
    """
    lib = _lib or load()
    dev = parents.get_device()
    _expect_all(dev, "parents query_start_loc context_lens tree_mask positions",
                (parents, query_start_loc, context_lens, tree_mask, positions), _I32)
    T, S = parents.numel(), context_lens.numel()
    if parents.shape != (T,) or context_lens.shape != (S,) or query_start_loc.shape != (S + 1,):
        raise PagedKVError(-1, "parents must be [T], context_lens [S] and query_start_loc [S + 1]")
    if tree_mask.dim() != 2 or tree_mask.shape[0] != T or positions.shape != (T,):
        raise PagedKVError(-1, "tree_mask must be [T][words] and positions [T]")
    if max_query_len is None:
        max_query_len = _longest_query(query_start_loc, stream) if S else 0
    _run_on(dev, stream, lib.paged_kv_tree_layout,
            (parents.data_ptr(), query_start_loc.data_ptr(), context_lens.data_ptr(), S, T, max_query_len,
             tree_mask.data_ptr(), tree_mask.shape[1], positions.data_ptr()))


def paged_attention_tree_workspace_size(num_query_tokens: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                        block_size: int, max_query_len: int, max_context_len: int,
                                        partition_size: int = 0) -> int:
    return int(load().paged_attention_tree_workspace_size(num_query_tokens, num_heads, num_kv_heads, head_dim,
                                                          block_size, max_query_len, max_context_len, partition_size))


def _tree(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, tree_mask, scale, softcap,
          key_begin, max_query_len, max_context_len, partition_size, workspace, stream, fp8, scales):
    lib = _lib or load()
    dtype = query.dtype
    dt = _DTYPE.get(dtype)
    dev = query.get_device()
    if dt is None or dev < 0 or not query.is_contiguous():
        _cuda16("query", query)
    stored = _pool_dtype(key_cache, value_cache, dtype, fp8)
    _expect_all(dev, "out key_cache value_cache block_tables context_lens query_start_loc tree_mask key_begin",
                (out, key_cache, value_cache, block_tables, context_lens, query_start_loc, tree_mask, key_begin),
                (dtype, stored, stored, *_I32))
    shape, pool, tables = query.shape, key_cache.shape, block_tables.shape
    if len(pool) != 4 or len(shape) != 3 or len(tables) != 2:
        raise PagedKVError(-1, "key_cache must be [blocks][kv heads][block size][head dim], query [rows][heads][head "
                               "dim] and block_tables [S][max_blocks]")
    NB, Hkv, B, D = pool
    T, H, D2 = shape
    S, maxb = tables
    if D2 != D or out.shape != shape or value_cache.shape != pool:
        raise PagedKVError(-1, "shape mismatch between query, out and caches")
    if context_lens.shape != (S,) or query_start_loc.shape != (S + 1,):
        raise PagedKVError(-1, "block_tables must be [S][max_blocks], context_lens [S] and query_start_loc [S + 1]")
    if tree_mask.dim() != 2 or tree_mask.shape[0] != T:
        raise PagedKVError(-1, "tree_mask must be [rows][words]")
    words = tree_mask.shape[1]
    if max_query_len is None:
        max_query_len = _longest_query(query_start_loc, stream) if S else 0
    if max_context_len is None:
        max_context_len = maxb * B
    begin = None
    if key_begin is not None:
        if key_begin.shape != (T,):
            raise PagedKVError(-1, "key_begin must have one entry per query row")
        begin = key_begin.data_ptr()
    ws, wbytes = None, 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise PagedKVError(-1, "workspace must be a contiguous tensor on the query's device")
        wbytes = workspace.numel() * workspace.element_size()
    else:
        wbytes = lib.paged_attention_tree_workspace_size(T, H, Hkv, D, B, max_query_len, max_context_len,
                                                         partition_size)
        if wbytes:
            workspace = _new_workspace(wbytes, query, stream)
    if workspace is not None:
        ws = workspace.data_ptr()
    _run_on(dev, stream, lib.paged_attention_tree_fp8 if fp8 else lib.paged_attention_tree,
            (out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), block_tables.data_ptr(),
             maxb, context_lens.data_ptr(), query_start_loc.data_ptr(), S, T, max_query_len, max_context_len,
             tree_mask.data_ptr(), words, scale, softcap, begin, B, H, Hkv, D, NB, dt, *scales, partition_size, ws,
             wbytes))
    return out


def paged_attention_tree(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                         block_tables: torch.Tensor, context_lens: torch.Tensor, query_start_loc: torch.Tensor,
                         tree_mask: torch.Tensor, scale: float, softcap: float = 0.0,
                         key_begin: Optional[torch.Tensor] = None, max_query_len: Optional[int] = None,
                         max_context_len: Optional[int] = None, partition_size: int = 0,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of drafted trees (query/out [T][H][D], packed by query_start_loc [S + 1]): sequence s's q_len tokens
    are its last q_len context positions, and each sees the committed positions before them and the drafted ones whose
    bits are set in its tree_mask row ([T][words] int32, see paged_kv_tree_layout). ``softcap`` as in
    paged_attention_decode_scored; ``key_begin`` [T] int32: a first visible key per token (a window, or 2**31 - 1 for
    the tokens of a sequence that waits). It counts places in the cache, not positions: a window that is not longer than
    the tree is deep also has to leave the ancestors behind it out of tree_mask.

    ``max_query_len`` bounds every tree on the host; when omitted it is read from query_start_loc, which synchronises
    the call's stream.
    """
    return _tree(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, tree_mask, scale,
                 softcap, key_begin, max_query_len, max_context_len, partition_size, workspace, stream, False, ())


def paged_attention_tree_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                             value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                             query_start_loc: torch.Tensor, tree_mask: torch.Tensor, scale: float, k_scale: float,
                             v_scale: float, softcap: float = 0.0, key_begin: Optional[torch.Tensor] = None,
                             max_query_len: Optional[int] = None, max_context_len: Optional[int] = None,
                             partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """paged_attention_tree over an E4M3 pool (elements code * k_scale, code * v_scale); head_dim 128."""
    return _tree(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, tree_mask, scale,
                 softcap, key_begin, max_query_len, max_context_len, partition_size, workspace, stream, True,
                 (k_scale, v_scale))


def paged_kv_compact_accepted(key_cache: torch.Tensor, value_cache: torch.Tensor, block_tables: torch.Tensor,
                              context_lens: torch.Tensor, query_start_loc: torch.Tensor, accepted: torch.Tensor,
                              num_accepted: torch.Tensor, stream=None) -> None:
    """Move each tree's accepted path up behind the committed tokens: the K and V rows of node accepted[s][i] ([S][most]
    int32, increasing) to the place of node i, for i < num_accepted[s] ([S] int32). The caches are one pool
    [NB][Hkv][B][D], or the pools of all layers [layers][NB][Hkv][B][D]. context_lens count the drafted tokens."""
    lib = _lib or load()
    dev = key_cache.get_device()
    dt = _cache_dtype("key_cache", key_cache)
    _expect("value_cache", value_cache, key_cache.dtype, dev)
    pool = key_cache.shape
    if len(pool) not in (4, 5) or value_cache.shape != pool:
        raise PagedKVError(-1, "the caches must both be [blocks][kv heads][block size][head dim], or that per layer")
    _expect_all(dev, "block_tables context_lens query_start_loc accepted num_accepted",
                (block_tables, context_lens, query_start_loc, accepted, num_accepted), _I32)
    layers = pool[0] if len(pool) == 5 else 1
    NB, Hkv, B, D = pool[-4:]
    if block_tables.dim() != 2 or accepted.dim() != 2:
        raise PagedKVError(-1, "block_tables must be [S][max_blocks] and accepted [S][most]")
    S, maxb = block_tables.shape
    if context_lens.shape != (S,) or query_start_loc.shape != (S + 1,) or num_accepted.shape != (S,) or (
            accepted.shape[0] != S):
        raise PagedKVError(-1, "context_lens and num_accepted must be [S], query_start_loc [S + 1], accepted [S][most]")
    _run_on(dev, stream, lib.paged_kv_compact_accepted,
            (key_cache.data_ptr(), value_cache.data_ptr(), layers, block_tables.data_ptr(), maxb,
             context_lens.data_ptr(), query_start_loc.data_ptr(), S, accepted.data_ptr(), accepted.shape[1],
             num_accepted.data_ptr(), Hkv, D, B, NB, dt))


def paged_kv_trim_blocks(block_tables: torch.Tensor, context_lens: torch.Tensor, keep_lens: torch.Tensor,
                         free_blocks: torch.Tensor, num_free: torch.Tensor, context_lens_out: torch.Tensor,
                         num_free_out: torch.Tensor, block_size: int, num_blocks: int, stream=None) -> None:
    """Cut each sequence back to its first keep_lens[s] tokens ([S] int32): push the blocks behind them on the free
    stack free_blocks (in place), and write context_lens_out [S] and num_free_out [1]. What is written must not overlap
    anything else of the call."""
    lib = _lib or load()
    S, maxb, dev = _pool_arrays(block_tables, context_lens, "keep_lens", keep_lens, free_blocks, num_free,
                                context_lens_out, num_free_out)
    _run_on(dev, stream, lib.paged_kv_trim_blocks,
            (block_tables.data_ptr(), maxb, context_lens.data_ptr(), keep_lens.data_ptr(), free_blocks.data_ptr(),
             free_blocks.numel(), num_free.data_ptr(), context_lens_out.data_ptr(), num_free_out.data_ptr(), S,
             block_size, num_blocks))


def device_errors(clear: bool = True) -> int:
    """The current device's error word (PKV_DEVERR_* bits); synchronises the device."""
    lib = load()
    v = ctypes.c_uint32(0)
    _check(lib, lib.paged_kv_device_errors(ctypes.byref(v), 1 if clear else 0))
    return int(v.value)


def paged_attention_decode_static_workspace(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                            value_cache: torch.Tensor, block_tables: torch.Tensor,
                                            context_lens: torch.Tensor, scale: float,
                                            max_context_len: Optional[int] = None, partition_size: int = 0,
                                            stream=None) -> torch.Tensor:
    """paged_attention_decode without a caller workspace, for callers that cannot allocate device memory.

    The split-K scratch is the library's own PKV_STATIC_WORKSPACE_BYTES (32 MiB)
    array on each device, so nothing is allocated here or in the library.
    Calls on one device share that array: calls that overlap on the GPU race.
    """
    lib = load()
    fn = lib.paged_attention_decode_static_workspace
    if fn.argtypes is None:
        P, i32, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
        fn.restype = i32
        fn.argtypes = [P, P, P, P, P, i32, P, i32, i32, f32, i32, i32, i32, i32, i32, i32, i32, P]
    dt = _cuda16("query", query)
    for n, t in (("out", out), ("key_cache", key_cache), ("value_cache", value_cache)):
        if _cuda16(n, t) != dt:
            raise PagedKVError(-1, f"{n} dtype differs from query")
    _cuda_i32("block_tables", block_tables)
    _cuda_i32("context_lens", context_lens)
    NB, Hkv, B, D = key_cache.shape
    S, H, _ = query.shape
    if out.shape != query.shape or value_cache.shape != key_cache.shape:
        raise PagedKVError(-1, "shape mismatch between query, out and caches")
    maxb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = maxb * B
    _check(lib, fn(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables), maxb,
                   _ptr(context_lens), S, int(max_context_len), float(scale), B, H, Hkv, D, NB, dt,
                   int(partition_size), _stream(query, stream)))
    return out


def read_chunks(buffer: torch.Tensor, order: torch.Tensor, chunk_bytes: int, stream=None) -> None:
    """Read the chunks order[i] (int32, on the device) of chunk_bytes from buffer (uint8), one bulk copy each
    into shared memory: the read ceiling of an access pattern (a measurement helper, not a step of the method)."""
    lib = load()
    fn = lib.pkv_read_chunks
    if fn.argtypes is None:
        fn.restype = ctypes.c_int32
        fn.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                       ctypes.c_void_p]
    if buffer.dtype != torch.uint8 or not buffer.is_cuda or not buffer.is_contiguous():
        raise PagedKVError(-1, "buffer must be a contiguous CUDA uint8 tensor")
    _cuda_i32("order", order)
    _check(lib, fn(_ptr(buffer), buffer.numel(), _ptr(order), order.numel(), int(chunk_bytes),
                   _stream(buffer, stream)))


def selftest_wait_timeout(limit_cycles: int = 2_000_000) -> int:
    """Run the bounded-wait self-test; returns the error word it leaves (PKV_DEVERR_TIMEOUT expected)."""
    lib = load()
    _check(lib, lib.pkv_selftest_wait_timeout(int(limit_cycles), _stream(torch.empty(0, device="cuda"), None)))
    return device_errors(clear=True)
