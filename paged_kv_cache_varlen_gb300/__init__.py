"""Paged KV-cache attention for GB300 (sm_103a).

The compute lives in ``libpkv.so`` (hand-written CUDA behind a C ABI, see
``include/pkv.h``); :mod:`.binding` marshals torch tensors into it. The
library is loaded on first use and its absence is an error: there is no CPU
fallback.
"""
from .binding import (  # noqa: F401
    BlockManager,
    PkvError,
    attention_key_weights,
    attention_workspace_size,
    copy_blocks_fp8,
    evict_compact,
    evict_select,
    kv_cache_append_fp8,
    kv_cache_write,
    library_path,
    lse_merge,
    paged_attention_varlen,
    paged_attention_varlen_append,
    paged_attention_varlen_fp8,
    paged_attention_varlen_range,
    paged_attention_varlen_window,
    qk_norm_rope_kv_cache_append_fp8,
    qk_norm_rope_kv_cache_write,
    rope_frequencies,
    rope_kv_cache_write,
    window_attention_workspace_size,
)

__all__ = [
    "BlockManager",
    "PkvError",
    "attention_key_weights",
    "attention_workspace_size",
    "copy_blocks_fp8",
    "evict_compact",
    "evict_select",
    "kv_cache_append_fp8",
    "kv_cache_write",
    "library_path",
    "lse_merge",
    "paged_attention_varlen",
    "paged_attention_varlen_append",
    "paged_attention_varlen_fp8",
    "paged_attention_varlen_range",
    "paged_attention_varlen_window",
    "qk_norm_rope_kv_cache_append_fp8",
    "qk_norm_rope_kv_cache_write",
    "rope_frequencies",
    "rope_kv_cache_write",
    "window_attention_workspace_size",
]
