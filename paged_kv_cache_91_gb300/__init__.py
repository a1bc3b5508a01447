"""Paged KV cache decode attention for GB300 (sm_103a).

The CUDA library (``libpaged_kv.so``, C ABI in ``include/paged_kv.h``) does the
work; ``binding`` marshals torch tensors into its calls. Importing this package
does not load the library; the first call does, and fails loudly if it is
missing.
"""
from .binding import (  # noqa: F401
    PagedKVError,
    paged_attention_decode,
    paged_attention_decode_fp8,
    paged_attention_decode_scored,
    paged_attention_decode_scored_fp8,
    paged_attention_decode_shared_prefix,
    paged_attention_decode_shared_prefix_fp8,
    paged_attention_multi_query,
    paged_attention_multi_query_fp8,
    paged_attention_multi_query_scored,
    paged_attention_multi_query_scored_fp8,
    paged_attention_multi_query_workspace_size,
    paged_attention_scored_workspace_size,
    paged_attention_shared_prefix_workspace_size,
    paged_attention_tree,
    paged_attention_tree_fp8,
    paged_attention_tree_workspace_size,
    paged_attention_workspace_size,
    paged_attention_workspace_size_fp8,
    paged_kv_compact_accepted,
    paged_kv_copy_blocks,
    paged_kv_release_blocks,
    paged_kv_reserve_slots,
    paged_kv_tree_layout,
    paged_kv_trim_blocks,
    paged_kv_write,
    paged_kv_write_fp8,
    paged_kv_write_rope,
    paged_kv_write_rope_fp8,
)
