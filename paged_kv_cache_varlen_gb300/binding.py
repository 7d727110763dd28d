"""Python binding of ``libpkv.so`` (argument marshalling only).

Every function here has the name of the C entry point without its ``pkv_``
prefix (``include/pkv.h``). It checks that the torch tensors have the dtype,
device and dense layout the C ABI expects, passes their device pointers and
the current CUDA stream, and raises :class:`PkvError` on a non-zero status.
All computation happens in the CUDA kernels behind the C ABI; if the library
is missing, the call fails: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

from . import debug_checks

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "libpkv.so")

_lock = threading.Lock()
_handle = None

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32

# name -> (restype, argtypes), mirroring include/pkv.h
_SIGNATURES = {
    "pkv_kv_cache_write": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "pkv_attention_workspace_size": (ctypes.c_size_t, [_i32] * 7),
    "pkv_paged_attention_varlen": (
        _i32, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp] + [_i32] * 9
        + [ctypes.c_float, _i32, _vp, ctypes.c_size_t, _vp, _vp]),
    "pkv_paged_attention_varlen_append": (
        _i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp] + [_i32] * 9
        + [ctypes.c_float, _i32, _vp, ctypes.c_size_t, _vp, _vp]),
    "pkv_paged_attention_varlen_range": (
        _i32, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp] + [_i32] * 9
        + [ctypes.c_float, _i32, _vp, ctypes.c_size_t, _vp, _vp]),
    "pkv_lse_merge": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]),
    "pkv_paged_attention_varlen_noalloc": (
        _i32, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp] + [_i32] * 9
        + [ctypes.c_float, _i32, _vp, _vp]),
    "pkv_cascade_workspace_size": (ctypes.c_size_t, [_i32] * 8),
    "pkv_cascade_decode": (
        _i32, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _i32]
        + [_i32] * 6 + [ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp]),
    "pkv_copy_blocks": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "pkv_copy_blocks_fp8": (_i32, [_vp] * 4 + [_i32] * 5 + [_vp, _vp]),
    "pkv_rope_frequencies": (
        _i32, [_vp, _vp, _i32, ctypes.c_double, _i32] + [ctypes.c_double] * 4),
    "pkv_rope_kv_cache_write": (
        _i32, [_vp] * 5 + [ctypes.c_int64] * 3 + [_vp] * 3 + [ctypes.c_float] + [_i32] * 8
        + [_vp, _vp]),
    "pkv_qk_norm_rope_kv_cache_write": (
        _i32, [_vp] * 5 + [ctypes.c_int64] * 3 + [_vp] * 5 + [_i32] + [ctypes.c_float] * 3
        + [_i32] * 8 + [_vp, _vp]),
    "pkv_kv_cache_append_fp8": (
        _i32, [_vp] * 4 + [ctypes.c_int64] * 2 + [_vp, _i32, _vp, _vp] + [_i32] * 7 + [_vp, _vp]),
    "pkv_qk_norm_rope_kv_cache_append_fp8": (
        _i32, [_vp] * 6 + [ctypes.c_int64] * 3 + [_vp, _vp, _i32] + [_vp] * 5 + [_i32]
        + [ctypes.c_float] * 3 + [_i32] * 10 + [_vp, _vp]),
    "pkv_window_attention_workspace_size": (ctypes.c_size_t, [_i32] * 8),
    "pkv_paged_attention_varlen_window": (
        _i32, [_vp, _i32] + [_vp] * 4 + [_i32, _vp, _vp] + [_i32] * 11
        + [ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp]),
    "pkv_paged_attention_varlen_fp8": (
        _i32, [_vp, _i32] + [_vp] * 5 + [_i32, _vp, _vp] + [_i32] * 11
        + [ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp]),
    "pkv_attention_key_weights": (
        _i32, [_vp] * 6 + [_i32] + [_vp] * 4 + [_i32] * 11
        + [ctypes.c_float, ctypes.c_float, _vp, _vp]),
    "pkv_evict_select": (_i32, [_vp] * 6 + [_i32] * 8 + [_vp, _vp]),
    "pkv_evict_compact": (
        _i32, [_vp, _vp, _i32, _vp, _i32, _vp, _i32, _vp] + [_i32] * 5 + [_vp, _vp]),
    "pkv_bm_create": (_i32, [_i32, _i32, _vp, ctypes.POINTER(_vp)]),
    "pkv_bm_destroy": (None, [_vp]),
    "pkv_bm_add_seq": (_i32, [_vp, ctypes.c_int64]),
    "pkv_bm_fork": (_i32, [_vp, ctypes.c_int64, ctypes.c_int64]),
    "pkv_bm_free_seq": (_i32, [_vp, ctypes.c_int64]),
    "pkv_bm_append": (_i32, [_vp, ctypes.c_int64, _i32, _vp, _vp, _vp, _i32, _vp]),
    "pkv_bm_build_step": (_i32, [_vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                 _vp]),
    "pkv_bm_evict_step": (_i32, [_vp, _vp, _vp, _i32, _i32, _vp, _i32, _vp]),
    "pkv_bm_num_free": (_i32, [_vp]),
    "pkv_bm_seq_len": (ctypes.c_int64, [_vp, ctypes.c_int64]),
    "pkv_bm_refcount": (_i32, [_vp, _i32]),
    "pkv_bm_block_table": (_i32, [_vp, ctypes.c_int64, _vp, _i32, _vp]),
    "pkv_status_string": (ctypes.c_char_p, [_i32]),
    "pkv_abi_version": (_i32, []),
}

DEV_BAD_SLOT = 1
DEV_BAD_BLOCK = 2
DEV_BAD_LENGTHS = 4
DEV_TIMEOUT = 8
DEV_V_RANGE = 16
DEV_BAD_POSITION = 32
DEV_BAD_ROW = 64
DEV_BAD_KEPT = 128


class PkvError(RuntimeError):
    """A libpkv call returned an error status (or the library is missing)."""

    def __init__(self, message: str, status: int | None = None):
        super().__init__(message)
        self.status = status


def library_path() -> str:
    return LIBRARY


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load ``libpkv.so`` once and declare the C signatures."""
    global _handle
    with _lock:
        if _handle is not None and path is None:
            return _handle
        p = path or LIBRARY
        if not os.path.exists(p):
            raise PkvError(
                f"{p} is missing: build it first (python -c 'import __graft_entry__ as g; "
                "g.build()'). There is no CPU fallback.")
        lib = ctypes.CDLL(p)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _handle = lib
        return lib


def _check(status: int, what: str) -> None:
    if status != 0:
        msg = load_library().pkv_status_string(status).decode()
        raise PkvError(f"{what}: {msg} (status {status})", status)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


# the current stream's handle without the Stream object around it (2 us less)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device) -> int:
    if stream is None:
        if _raw_stream is not None and device.index is not None:
            return _raw_stream(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, dtype, ndim: int, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def kv_cache_write(kv_pool: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                   slot_mapping: torch.Tensor, dev_status: torch.Tensor | None = None,
                   stream=None) -> None:
    """Scatter k_new/v_new [T,Hkv,D] bf16 into kv_pool [2,NB,BS,Hkv,D] bf16."""
    _need(kv_pool, torch.bfloat16, 5, "kv_pool")
    _need(k_new, torch.bfloat16, 3, "k_new")
    _need(v_new, torch.bfloat16, 3, "v_new")
    _need(slot_mapping, torch.int32, 1, "slot_mapping")
    _, nb, bs, hkv, d = kv_pool.shape
    t = slot_mapping.shape[0]
    if tuple(k_new.shape) != (t, hkv, d) or tuple(v_new.shape) != (t, hkv, d):
        raise ValueError("k_new / v_new must be [num_tokens, num_kv_heads, head_dim]")
    if dev_status is not None:
        _need(dev_status, torch.int32, 1, "dev_status")
    if debug_checks.enabled():
        debug_checks.check_slot_mapping(slot_mapping, num_blocks=nb, block_size=bs)
    st = load_library().pkv_kv_cache_write(
        _ptr(kv_pool), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), t, nb, bs, hkv, d,
        _ptr(dev_status), _stream(stream, kv_pool.device))
    _check(st, "kv_cache_write")


def attention_workspace_size(num_seqs: int, num_tokens: int, num_heads: int, num_kv_heads: int,
                             head_dim: int, max_seq_len: int, partition_size: int = -1) -> int:
    return int(load_library().pkv_attention_workspace_size(
        num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, max_seq_len, partition_size))


def paged_attention_varlen(q: torch.Tensor, kv_pool: torch.Tensor, block_table: torch.Tensor,
                           cu_seqlens: torch.Tensor, seq_lens: torch.Tensor,
                           max_query_len: int, max_seq_len: int, *,
                           out: torch.Tensor | None = None, out_lse: torch.Tensor | None = None,
                           scale: float | None = None, partition_size: int = -1,
                           workspace: torch.Tensor | None = None,
                           dev_status: torch.Tensor | None = None, stream=None):
    """Causal GQA attention of q [T,H,D] bf16 over the paged pool.

    Returns ``(out, out_lse)``; ``out`` is fp32 [T,H,D], ``out_lse`` fp32
    [T,H] or None. Missing ``out`` / ``workspace`` buffers are allocated with
    torch (the library itself never allocates); a workspace passed in must
    have been zero-filled before its first use (``attention_workspace_size``).
    """
    _need(q, torch.bfloat16, 3, "q")
    _need(kv_pool, torch.bfloat16, 5, "kv_pool")
    _need(block_table, torch.int32, 2, "block_table")
    _need(cu_seqlens, torch.int32, 1, "cu_seqlens")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    t, h, d = q.shape
    _, nb, bs, hkv, d2 = kv_pool.shape
    if d2 != d:
        raise ValueError("q and kv_pool head_dim differ")
    b = seq_lens.shape[0]
    if cu_seqlens.shape[0] != b + 1 or block_table.shape[0] != b:
        raise ValueError("cu_seqlens must be [B+1] and block_table [B, max_blocks]")
    if out is None:
        out = torch.empty((t, h, d), dtype=torch.float32, device=q.device)
    _need(out, torch.float32, 3, "out")
    if out_lse is not None:
        _need(out_lse, torch.float32, 2, "out_lse")
    if dev_status is not None:
        _need(dev_status, torch.int32, 1, "dev_status")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if debug_checks.enabled():
        debug_checks.check_attention_tables(
            cu_seqlens, seq_lens, block_table, num_tokens=t, max_query_len=int(max_query_len),
            max_seq_len=int(max_seq_len), num_blocks=nb, block_size=bs)
    need = attention_workspace_size(b, t, h, hkv, d, max_seq_len, partition_size)
    if need and workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().pkv_paged_attention_varlen(
        _ptr(out), _ptr(out_lse), _ptr(q), _ptr(kv_pool), _ptr(block_table),
        block_table.shape[1], _ptr(cu_seqlens), _ptr(seq_lens), b, t, int(max_query_len),
        int(max_seq_len), h, hkv, d, bs, nb, float(scale), int(partition_size),
        _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream, q.device))
    _check(st, "paged_attention_varlen")
    return out, out_lse


def paged_attention_varlen_append(q: torch.Tensor, kv_pool: torch.Tensor, k_new: torch.Tensor,
                                  v_new: torch.Tensor, slot_mapping: torch.Tensor,
                                  block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                                  seq_lens: torch.Tensor, max_query_len: int, max_seq_len: int, *,
                                  out: torch.Tensor | None = None,
                                  out_lse: torch.Tensor | None = None, scale: float | None = None,
                                  partition_size: int = -1, workspace: torch.Tensor | None = None,
                                  dev_status: torch.Tensor | None = None, stream=None):
    """A step's KV write and attention in one call (``kv_cache_write`` then
    ``paged_attention_varlen``, overlapped). ``slot_mapping[t]`` must be the
    pool slot ``block_table`` gives to token t's position (the step's
    appended slots). Returns ``(out, out_lse)`` as ``paged_attention_varlen``."""
    _need(q, torch.bfloat16, 3, "q")
    _need(kv_pool, torch.bfloat16, 5, "kv_pool")
    _need(k_new, torch.bfloat16, 3, "k_new")
    _need(v_new, torch.bfloat16, 3, "v_new")
    _need(slot_mapping, torch.int32, 1, "slot_mapping")
    _need(block_table, torch.int32, 2, "block_table")
    _need(cu_seqlens, torch.int32, 1, "cu_seqlens")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    t, h, d = q.shape
    _, nb, bs, hkv, d2 = kv_pool.shape
    if d2 != d:
        raise ValueError("q and kv_pool head_dim differ")
    if slot_mapping.shape[0] != t or tuple(k_new.shape) != (t, hkv, d) or \
            tuple(v_new.shape) != (t, hkv, d):
        raise ValueError("k_new / v_new must be [num_tokens, num_kv_heads, head_dim] and "
                         "slot_mapping [num_tokens]")
    b = seq_lens.shape[0]
    if cu_seqlens.shape[0] != b + 1 or block_table.shape[0] != b:
        raise ValueError("cu_seqlens must be [B+1] and block_table [B, max_blocks]")
    if out is None:
        out = torch.empty((t, h, d), dtype=torch.float32, device=q.device)
    _need(out, torch.float32, 3, "out")
    if out_lse is not None:
        _need(out_lse, torch.float32, 2, "out_lse")
    if dev_status is not None:
        _need(dev_status, torch.int32, 1, "dev_status")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if debug_checks.enabled():
        debug_checks.check_slot_mapping(slot_mapping, num_blocks=nb, block_size=bs)
        debug_checks.check_attention_tables(
            cu_seqlens, seq_lens, block_table, num_tokens=t, max_query_len=int(max_query_len),
            max_seq_len=int(max_seq_len), num_blocks=nb, block_size=bs)
        debug_checks.check_append_slots(cu_seqlens, seq_lens, block_table, slot_mapping,
                                        block_size=bs)
    need = attention_workspace_size(b, t, h, hkv, d, max_seq_len, partition_size)
    if need and workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().pkv_paged_attention_varlen_append(
        _ptr(out), _ptr(out_lse), _ptr(q), _ptr(kv_pool), _ptr(k_new), _ptr(v_new),
        _ptr(slot_mapping), _ptr(block_table), block_table.shape[1], _ptr(cu_seqlens),
        _ptr(seq_lens), b, t, int(max_query_len), int(max_seq_len), h, hkv, d, bs, nb,
        float(scale), int(partition_size), _ptr(workspace), ws_bytes, _ptr(dev_status),
        _stream(stream, q.device))
    _check(st, "paged_attention_varlen_append")
    return out, out_lse


def paged_attention_varlen_range(q: torch.Tensor, kv_pool: torch.Tensor,
                                 block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                                 seq_lens: torch.Tensor, key_start_pos: torch.Tensor,
                                 query_start_pos: torch.Tensor, max_query_len: int,
                                 max_seq_len: int, *, out: torch.Tensor | None = None,
                                 out_lse: torch.Tensor | None = None, scale: float | None = None,
                                 partition_size: int = -1, workspace: torch.Tensor | None = None,
                                 dev_status: torch.Tensor | None = None, stream=None):
    """Attention over a range of each request's keys (``pkv_paged_attention_varlen_range``).

    Request i's table holds ``seq_lens[i]`` keys at absolute positions
    ``key_start_pos[i] + p``; its queries sit at ``query_start_pos[i] + j``
    and see the keys at or before their own position. Returns the normalised
    piece ``(out, out_lse)``; pieces of one context merge with :func:`lse_merge`.
    """
    _need(q, torch.bfloat16, 3, "q")
    _need(kv_pool, torch.bfloat16, 5, "kv_pool")
    _need(block_table, torch.int32, 2, "block_table")
    for t, name in ((cu_seqlens, "cu_seqlens"), (seq_lens, "seq_lens"),
                    (key_start_pos, "key_start_pos"), (query_start_pos, "query_start_pos")):
        _need(t, torch.int32, 1, name)
    t, h, d = q.shape
    _, nb, bs, hkv, d2 = kv_pool.shape
    if d2 != d:
        raise ValueError("q and kv_pool head_dim differ")
    b = seq_lens.shape[0]
    if (cu_seqlens.shape[0] != b + 1 or block_table.shape[0] != b
            or key_start_pos.shape[0] != b or query_start_pos.shape[0] != b):
        raise ValueError("cu_seqlens must be [B+1]; block_table, key_start_pos and "
                         "query_start_pos one row per request")
    if out is None:
        out = torch.empty((t, h, d), dtype=torch.float32, device=q.device)
    _need(out, torch.float32, 3, "out")
    if out_lse is not None:
        _need(out_lse, torch.float32, 2, "out_lse")
    if dev_status is not None:
        _need(dev_status, torch.int32, 1, "dev_status")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if debug_checks.enabled():
        debug_checks.check_attention_tables(
            cu_seqlens, seq_lens, block_table, num_tokens=t, max_query_len=int(max_query_len),
            max_seq_len=int(max_seq_len), num_blocks=nb, block_size=bs,
            key_start=key_start_pos, query_start=query_start_pos)
    need = attention_workspace_size(b, t, h, hkv, d, max_seq_len, partition_size)
    if need and workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().pkv_paged_attention_varlen_range(
        _ptr(out), _ptr(out_lse), _ptr(q), _ptr(kv_pool), _ptr(block_table),
        block_table.shape[1], _ptr(cu_seqlens), _ptr(seq_lens), _ptr(key_start_pos),
        _ptr(query_start_pos), b, t, int(max_query_len), int(max_seq_len), h, hkv, d, bs, nb,
        float(scale), int(partition_size), _ptr(workspace), ws_bytes, _ptr(dev_status),
        _stream(stream, q.device))
    _check(st, "paged_attention_varlen_range")
    return out, out_lse


def lse_merge(part_out: torch.Tensor, part_lse: torch.Tensor, *,
              out: torch.Tensor | None = None, out_lse: torch.Tensor | None = None,
              stream=None):
    """Merge part_out [P,T,H,D] / part_lse [P,T,H] fp32 into out [T,H,D]."""
    _need(part_out, torch.float32, 4, "part_out")
    _need(part_lse, torch.float32, 3, "part_lse")
    p, t, h, d = part_out.shape
    if tuple(part_lse.shape) != (p, t, h):
        raise ValueError("part_lse must be [P, T, H]")
    if out is None:
        out = torch.empty((t, h, d), dtype=torch.float32, device=part_out.device)
    _need(out, torch.float32, 3, "out")
    if out_lse is not None:
        _need(out_lse, torch.float32, 2, "out_lse")
    st = load_library().pkv_lse_merge(_ptr(out), _ptr(out_lse), _ptr(part_out), _ptr(part_lse),
                                      p, t, h, d, _stream(stream, part_out.device))
    _check(st, "lse_merge")
    return out, out_lse


def paged_attention_varlen_noalloc(q: torch.Tensor, kv_pool: torch.Tensor,
                                   block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                                   seq_lens: torch.Tensor, max_query_len: int, max_seq_len: int,
                                   *, out: torch.Tensor, out_lse: torch.Tensor | None = None,
                                   scale: float | None = None, partition_size: int = -1,
                                   dev_status: torch.Tensor | None = None, stream=None):
    """:func:`paged_attention_varlen` for callers that cannot allocate.

    For code that may not allocate device memory (its memory manager owns
    the GPU, or it is not allowed to call cudaMalloc while serving): the
    split-KV scratch comes from a fixed 16 MiB array inside the library, so
    nothing is allocated here and ``out`` must be passed in. Raises
    :class:`PkvError` (status 4) when the sizes need more scratch than that.
    Calls that may overlap on the GPU share the array and race.
    """
    _need(q, torch.bfloat16, 3, "q")
    _need(kv_pool, torch.bfloat16, 5, "kv_pool")
    _need(block_table, torch.int32, 2, "block_table")
    _need(cu_seqlens, torch.int32, 1, "cu_seqlens")
    _need(seq_lens, torch.int32, 1, "seq_lens")
    _need(out, torch.float32, 3, "out")
    t, h, d = q.shape
    _, nb, bs, hkv, d2 = kv_pool.shape
    if d2 != d:
        raise ValueError("q and kv_pool head_dim differ")
    b = seq_lens.shape[0]
    if cu_seqlens.shape[0] != b + 1 or block_table.shape[0] != b:
        raise ValueError("cu_seqlens must be [B+1] and block_table [B, max_blocks]")
    if out_lse is not None:
        _need(out_lse, torch.float32, 2, "out_lse")
    if dev_status is not None:
        _need(dev_status, torch.int32, 1, "dev_status")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if debug_checks.enabled():
        debug_checks.check_attention_tables(
            cu_seqlens, seq_lens, block_table, num_tokens=t, max_query_len=int(max_query_len),
            max_seq_len=int(max_seq_len), num_blocks=nb, block_size=bs)
    st = load_library().pkv_paged_attention_varlen_noalloc(
        _ptr(out), _ptr(out_lse), _ptr(q), _ptr(kv_pool), _ptr(block_table),
        block_table.shape[1], _ptr(cu_seqlens), _ptr(seq_lens), b, t, int(max_query_len),
        int(max_seq_len), h, hkv, d, bs, nb, float(scale), int(partition_size),
        _ptr(dev_status), _stream(stream, q.device))
    _check(st, "paged_attention_varlen_noalloc")
    return out, out_lse


def copy_blocks(kv_pool: torch.Tensor, copy_src: torch.Tensor, copy_dst: torch.Tensor, *,
                dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Whole-block copies inside the pool (device int32 ``copy_src``/``copy_dst``),
    the device half of copy-on-write; run before the step's KV write."""
    _need(kv_pool, torch.bfloat16, 5, "kv_pool")
    _need(copy_src, torch.int32, 1, "copy_src")
    _need(copy_dst, torch.int32, 1, "copy_dst")
    if copy_src.shape != copy_dst.shape:
        raise ValueError("copy_src and copy_dst differ in length")
    if dev_status is not None:
        _need(dev_status, torch.int32, 1, "dev_status")
    _, nb, bs, hkv, d = kv_pool.shape
    st = load_library().pkv_copy_blocks(
        _ptr(kv_pool), _ptr(copy_src), _ptr(copy_dst), copy_src.shape[0], nb, bs, hkv, d,
        _ptr(dev_status), _stream(stream, kv_pool.device))
    _check(st, "copy_blocks")


def copy_blocks_fp8(kv_pool: torch.Tensor, kv_scales: torch.Tensor, copy_src: torch.Tensor,
                    copy_dst: torch.Tensor, *, dev_status: torch.Tensor | None = None,
                    stream=None) -> None:
    """:func:`copy_blocks` in the 8-bit pool of :func:`kv_cache_append_fp8`: the blocks
    and their scales, bit for bit."""
    _need(kv_pool, torch.float8_e4m3fn, 5, "kv_pool")
    _need(kv_scales, torch.float32, 3, "kv_scales")
    _need(copy_src, torch.int32, 1, "copy_src")
    _need(copy_dst, torch.int32, 1, "copy_dst")
    two, nb, bs, hkv, d = kv_pool.shape
    if two != 2 or tuple(kv_scales.shape) != (2, nb, hkv):
        raise ValueError("kv_pool must be [2, NB, BS, Hkv, D] and kv_scales [2, NB, Hkv]")
    if copy_src.shape != copy_dst.shape:
        raise ValueError("copy_src and copy_dst differ in length")
    if dev_status is not None:
        _need(dev_status, torch.int32, 1, "dev_status")
    st = load_library().pkv_copy_blocks_fp8(
        _ptr(kv_pool), _ptr(kv_scales), _ptr(copy_src), _ptr(copy_dst), copy_src.shape[0], nb, bs,
        hkv, d, _ptr(dev_status), _stream(stream, kv_pool.device))
    _check(st, "copy_blocks_fp8")


class BlockManager:
    """The host block manager of ``libpkv`` (native C++ behind the C ABI):
    free pool, per-sequence block tables, fork and copy-on-write."""

    def __init__(self, num_blocks: int, block_size: int, free_order=None):
        import numpy as np

        self._np = np
        lib = load_library()
        h = _vp()
        order = None
        if free_order is not None:
            order = np.ascontiguousarray(free_order, dtype=np.int32)
            if order.shape != (num_blocks,):
                raise ValueError("free_order must hold every block id once")
        st = lib.pkv_bm_create(num_blocks, block_size,
                               order.ctypes.data if order is not None else None, ctypes.byref(h))
        _check(st, "bm_create")
        self._lib, self._h = lib, h
        self.num_blocks, self.block_size = num_blocks, block_size

    def close(self):
        if self._h:
            self._lib.pkv_bm_destroy(self._h)
            self._h = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_seq(self, seq_id: int):
        _check(self._lib.pkv_bm_add_seq(self._h, seq_id), "bm_add_seq")

    def fork(self, parent: int, child: int):
        _check(self._lib.pkv_bm_fork(self._h, parent, child), "bm_fork")

    def free_seq(self, seq_id: int):
        _check(self._lib.pkv_bm_free_seq(self._h, seq_id), "bm_free_seq")

    def append(self, seq_id: int, num_tokens: int):
        """Returns (slots, copies) like the reference manager."""
        np = self._np
        slots = np.zeros(max(num_tokens, 1), dtype=np.int32)
        src = np.zeros(1, dtype=np.int32)
        dst = np.zeros(1, dtype=np.int32)
        n = ctypes.c_int32(0)
        st = self._lib.pkv_bm_append(self._h, seq_id, num_tokens, slots.ctypes.data,
                                     src.ctypes.data, dst.ctypes.data, 1, ctypes.byref(n))
        _check(st, "bm_append")
        return slots[:num_tokens].tolist(), list(zip(src[:n.value].tolist(), dst[:n.value].tolist()))

    def build_step(self, seq_ids, num_new, max_blocks: int):
        """One batch: (block_table, seq_lens, cu_seqlens, slot_mapping, copy_src, copy_dst)
        as numpy int32 arrays, ready to be copied to the device."""
        np = self._np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        nn = np.ascontiguousarray(num_new, dtype=np.int32)
        b = ids.shape[0]
        table = np.full((max(b, 1), max_blocks), -1, dtype=np.int32)
        lens = np.zeros(max(b, 1), dtype=np.int32)
        cu = np.zeros(b + 1, dtype=np.int32)
        slots = np.zeros(max(int(nn.sum()), 1), dtype=np.int32)
        cap = max(b, 1)
        src = np.zeros(cap, dtype=np.int32)
        dst = np.zeros(cap, dtype=np.int32)
        n = ctypes.c_int32(0)
        st = self._lib.pkv_bm_build_step(
            self._h, ids.ctypes.data, nn.ctypes.data, b, max_blocks, table.ctypes.data,
            lens.ctypes.data, cu.ctypes.data, slots.ctypes.data, src.ctypes.data, dst.ctypes.data,
            cap, ctypes.byref(n))
        _check(st, "bm_build_step")
        return (table[:b], lens[:b], cu, slots[:int(nn.sum())], src[:n.value], dst[:n.value])

    def evict_step(self, seq_ids, keep_lens, max_src_blocks: int, max_dst_blocks: int):
        """Cut each sequence back to ``keep_lens`` tokens in fresh blocks.

        Returns ``(src_table, dst_table)`` as numpy int32 arrays, the tables of
        :func:`evict_compact`. Enqueue that copy before the next step's
        writes, on the same stream: the old blocks may be handed out again."""
        np = self._np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        keep = np.ascontiguousarray(keep_lens, dtype=np.int32)
        if ids.ndim != 1 or keep.shape != ids.shape:
            raise ValueError("seq_ids and keep_lens must be one-dimensional, of one length")
        b = ids.shape[0]
        src = np.full((b, max_src_blocks), -1, dtype=np.int32)
        dst = np.full((b, max_dst_blocks), -1, dtype=np.int32)
        st = self._lib.pkv_bm_evict_step(self._h, ids.ctypes.data, keep.ctypes.data, b,
                                         max_src_blocks, src.ctypes.data, max_dst_blocks,
                                         dst.ctypes.data)
        _check(st, "bm_evict_step")
        return src, dst

    def num_free(self) -> int:
        return int(self._lib.pkv_bm_num_free(self._h))

    def seq_len(self, seq_id: int) -> int:
        return int(self._lib.pkv_bm_seq_len(self._h, seq_id))

    def refcount(self, block: int) -> int:
        return int(self._lib.pkv_bm_refcount(self._h, block))

    def block_table(self, seq_id: int):
        np = self._np
        n = ctypes.c_int32(0)
        cap = max(self.num_blocks, 1)
        out = np.zeros(cap, dtype=np.int32)
        st = self._lib.pkv_bm_block_table(self._h, seq_id, out.ctypes.data, cap, ctypes.byref(n))
        _check(st, "bm_block_table")
        return out[:n.value].tolist()


def cascade_workspace_size(num_seqs: int, num_prefix_groups: int, max_group_size: int,
                           max_prefix_len: int, max_tail_len: int, num_heads: int,
                           num_kv_heads: int, head_dim: int) -> int:
    return int(load_library().pkv_cascade_workspace_size(
        num_seqs, num_prefix_groups, max_group_size, max_prefix_len, max_tail_len, num_heads,
        num_kv_heads, head_dim))


def cascade_decode(q: torch.Tensor, kv_pool: torch.Tensor, group_starts: torch.Tensor,
                   prefix_lens: torch.Tensor, prefix_tables: torch.Tensor, max_group_size: int,
                   max_prefix_len: int, tail_tables: torch.Tensor, tail_lens: torch.Tensor,
                   max_tail_len: int, *, out: torch.Tensor | None = None,
                   out_lse: torch.Tensor | None = None, scale: float | None = None,
                   workspace: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                   stream=None):
    """Decode attention with copy-on-write prefixes read once per group
    (see ``pkv_cascade_decode``). Allocates a zeroed workspace when none is given."""
    _need(q, torch.bfloat16, 3, "q")
    _need(kv_pool, torch.bfloat16, 5, "kv_pool")
    for t, name in ((group_starts, "group_starts"), (prefix_lens, "prefix_lens"),
                    (tail_lens, "tail_lens")):
        _need(t, torch.int32, 1, name)
    _need(prefix_tables, torch.int32, 2, "prefix_tables")
    _need(tail_tables, torch.int32, 2, "tail_tables")
    b, h, d = q.shape
    _, nb, bs, hkv, d2 = kv_pool.shape
    if d2 != d:
        raise ValueError("q and kv_pool head_dim differ")
    g = prefix_lens.shape[0]
    if group_starts.shape[0] != g + 1 or prefix_tables.shape[0] != g:
        raise ValueError("group_starts must be [G+1] and prefix_tables [G, max_prefix_blocks]")
    if tail_tables.shape[0] != b or tail_lens.shape[0] != b:
        raise ValueError("tail_tables and tail_lens must have one row per request")
    if out is None:
        out = torch.empty((b, h, d), dtype=torch.float32, device=q.device)
    _need(out, torch.float32, 3, "out")
    if out_lse is not None:
        _need(out_lse, torch.float32, 2, "out_lse")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = cascade_workspace_size(b, g, int(max_group_size), int(max_prefix_len),
                                  int(max_tail_len), h, hkv, d)
    if workspace is None:
        workspace = torch.zeros(max(need, 1), dtype=torch.uint8, device=q.device)
    st = load_library().pkv_cascade_decode(
        _ptr(out), _ptr(out_lse), _ptr(q), _ptr(kv_pool), g, _ptr(group_starts), _ptr(prefix_lens),
        _ptr(prefix_tables), prefix_tables.shape[1], int(max_group_size), int(max_prefix_len),
        _ptr(tail_tables), tail_tables.shape[1], _ptr(tail_lens), int(max_tail_len), b, h, hkv, d,
        bs, nb, float(scale), _ptr(workspace), workspace.numel(), _ptr(dev_status),
        _stream(stream, q.device))
    _check(st, "cascade_decode")
    return out, out_lse


ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}


def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str = "none",
                     stretch: float = 1.0, original_len: float = 0.0, low: float = 1.0,
                     high: float | None = None):
    """Rotary frequencies ``(inv_freq, factor)``: a float64 CPU tensor
    [rotary_dim / 2] in radians per position (move it to the device once) and
    the scale of the rotated values.

    ``scaling`` stretches the context by ``stretch``: "none", "linear"
    (positions interpolated), "base" (a larger base), "bands" (pairs that make
    fewer than ``low`` turns over ``original_len`` positions are stretched,
    those above ``high``, default 4, are not) or "ramp" (the same between pair
    indexes, ``high`` 32 by default, with a scale on the rotated values). The
    formulas stand with ``pkv_rope_frequencies`` in ``include/pkv.h``."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(ROPE_SCALINGS)}, got {scaling!r}")
    if high is None:
        high = 32.0 if scaling == "ramp" else 4.0
    inv_freq = torch.empty(max(int(rotary_dim) // 2, 1), dtype=torch.float64)
    factor = ctypes.c_float(0.0)
    st = load_library().pkv_rope_frequencies(
        inv_freq.data_ptr(), ctypes.addressof(factor), int(rotary_dim), float(base),
        ROPE_SCALINGS[scaling], float(stretch), float(original_len), float(low), float(high))
    _check(st, "rope_frequencies")
    return inv_freq, float(factor.value)


# The calls below are made once a layer and step, on a handful of small tensors:
# the module `_marshal` checks their tensors as `_need` does and calls libpkv.
_native = None


def _marshal():
    global _native
    if _native is None:
        load_library()  # a missing library is reported the same way
        import importlib

        try:
            module = importlib.import_module("._marshal", __package__)
        except ImportError as e:
            raise PkvError(f"{_HERE}/_marshal.so cannot be loaded ({e}): build it first (python -c "
                           "'import __graft_entry__ as g; g.build()')") from e
        module.set_error(PkvError)
        _native = module
    return _native


def _handle_of(stream):
    """None, or the stream's integer handle."""
    if stream is None:
        return None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on_stream(stream, device):
    """The stream as torch sees it, for allocations that the call's work uses."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def rope_kv_cache_write(q: torch.Tensor, kv_pool: torch.Tensor, k_new: torch.Tensor,
                        v_new: torch.Tensor, positions: torch.Tensor, slot_mapping: torch.Tensor,
                        inv_freq: torch.Tensor, *, interleaved: bool = False, factor: float = 1.0,
                        q_out: torch.Tensor | None = None,
                        dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotate q and k_new by ``positions`` and write k_new/v_new into the pool.

    q [T,H,D], k_new/v_new [T,Hkv,D] bf16; a token's heads contiguous, tokens
    any distance apart (slices of one projection output do). ``inv_freq`` is
    the float64 device tensor of ``rope_frequencies``; the first
    ``2 * len(inv_freq)`` dimensions rotate. ``positions`` are independent of
    ``slot_mapping`` (-1: nothing is written). Returns ``q_out`` [T,H,D],
    which may be a dense q itself."""
    native = _native or _marshal()
    if native.debug_checks():
        debug_checks.check_slot_mapping(slot_mapping, num_blocks=kv_pool.shape[1],
                                        block_size=kv_pool.shape[2])
        debug_checks.check_positions(positions)
    if q_out is None and stream is not None:
        with _on_stream(stream, q.device):
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    return native.rope_kv_cache_write(
        q, kv_pool, k_new, v_new, positions, slot_mapping, inv_freq, interleaved, factor, q_out,
        dev_status, _handle_of(stream))


def qk_norm_rope_kv_cache_write(q: torch.Tensor, kv_pool: torch.Tensor, k_new: torch.Tensor,
                                v_new: torch.Tensor, positions: torch.Tensor,
                                slot_mapping: torch.Tensor, inv_freq: torch.Tensor | None,
                                q_weight: torch.Tensor | None, k_weight: torch.Tensor | None, *,
                                eps: float = 1e-6, weight_offset: float = 0.0,
                                interleaved: bool = False, factor: float = 1.0,
                                q_out: torch.Tensor | None = None,
                                dev_status: torch.Tensor | None = None,
                                stream=None) -> torch.Tensor:
    """:func:`rope_kv_cache_write` with a norm over each query and key head first.

    ``q_weight`` / ``k_weight`` [D], bf16 or fp32 (None: not normed):
    ``x * rsqrt(mean(x^2) + eps) * (weight + weight_offset)`` over each head,
    then the rotation (``inv_freq`` None: none). Returns ``q_out`` [T,H,D],
    which may be a dense q itself."""
    native = _native or _marshal()
    if native.debug_checks():
        debug_checks.check_slot_mapping(slot_mapping, num_blocks=kv_pool.shape[1],
                                        block_size=kv_pool.shape[2])
        debug_checks.check_positions(positions)
    if q_out is None and stream is not None:
        with _on_stream(stream, q.device):
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    return native.qk_norm_rope_kv_cache_write(
        q, kv_pool, k_new, v_new, positions, slot_mapping, inv_freq, q_weight, k_weight, eps,
        weight_offset, interleaved, factor, q_out, dev_status, _handle_of(stream))


def kv_cache_append_fp8(kv_pool: torch.Tensor, kv_scales: torch.Tensor, k_new: torch.Tensor,
                        v_new: torch.Tensor, block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                        seq_lens: torch.Tensor, max_query_len: int, *,
                        dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Write a step's k_new/v_new [T,Hkv,D] bf16 into the 8-bit pool.

    ``kv_pool`` [2,NB,BS,Hkv,D] float8_e4m3fn, ``kv_scales`` [2,NB,Hkv] fp32.
    Token j of request i goes to position ``seq_lens[i] - query_len + j`` of its
    table (what :meth:`BlockManager.build_step` returns says where). A block's
    scale is the power of two that its largest magnitude needs; rows that are
    there are rescaled where it grows (``pkv_kv_cache_append_fp8`` in
    ``include/pkv.h``)."""
    native = _native or _marshal()
    if native.debug_checks():
        _check_append_tables(kv_pool, k_new, block_table, cu_seqlens, seq_lens, max_query_len)
    native.kv_cache_append_fp8(kv_pool, kv_scales, k_new, v_new, block_table, cu_seqlens, seq_lens,
                               max_query_len, dev_status, _handle_of(stream))


def qk_norm_rope_kv_cache_append_fp8(q: torch.Tensor, kv_pool: torch.Tensor,
                                     kv_scales: torch.Tensor, k_new: torch.Tensor,
                                     v_new: torch.Tensor, positions: torch.Tensor,
                                     block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                                     seq_lens: torch.Tensor, max_query_len: int,
                                     inv_freq: torch.Tensor | None,
                                     q_weight: torch.Tensor | None = None,
                                     k_weight: torch.Tensor | None = None, *, eps: float = 1e-6,
                                     weight_offset: float = 0.0, interleaved: bool = False,
                                     factor: float = 1.0, q_out: torch.Tensor | None = None,
                                     dev_status: torch.Tensor | None = None,
                                     stream=None) -> torch.Tensor:
    """The norms and the rotation of :func:`qk_norm_rope_kv_cache_write` on the way
    into the 8-bit pool of :func:`kv_cache_append_fp8`: keys are quantised from
    the fp32 result, queries come back in bf16. Without weights the heads are
    rotated only."""
    native = _native or _marshal()
    if native.debug_checks():
        _check_append_tables(kv_pool, k_new, block_table, cu_seqlens, seq_lens, max_query_len)
        debug_checks.check_positions(positions)
    if q_out is None and stream is not None:
        with _on_stream(stream, q.device):
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    return native.qk_norm_rope_kv_cache_append_fp8(
        q, kv_pool, kv_scales, k_new, v_new, positions, block_table, cu_seqlens, seq_lens,
        max_query_len, inv_freq, q_weight, k_weight, eps, weight_offset, interleaved, factor, q_out,
        dev_status, _handle_of(stream))


def _check_append_tables(kv_pool, k_new, block_table, cu_seqlens, seq_lens, max_query_len):
    debug_checks.check_append_tables(
        cu_seqlens, seq_lens, block_table, num_tokens=k_new.shape[0],
        max_query_len=int(max_query_len), num_blocks=kv_pool.shape[1],
        block_size=kv_pool.shape[2])


def window_attention_workspace_size(max_query_len: int, num_heads: int, num_kv_heads: int,
                                    head_dim: int, max_seq_len: int, window: int = 0,
                                    num_sink: int = 0, eight_bit: bool = False) -> int:
    """Bytes of scratch of :func:`paged_attention_varlen_window` and, with
    ``eight_bit``, of :func:`paged_attention_varlen_fp8`."""
    return int(load_library().pkv_window_attention_workspace_size(
        max_query_len, num_heads, num_kv_heads, head_dim, max_seq_len, window, num_sink,
        int(eight_bit)))


def paged_attention_varlen_window(q: torch.Tensor, kv_pool: torch.Tensor,
                                  block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                                  seq_lens: torch.Tensor, max_query_len: int, max_seq_len: int,
                                  window: int, *, num_sink: int = 0,
                                  out: torch.Tensor | None = None,
                                  out_lse: torch.Tensor | None = None, scale: float | None = None,
                                  workspace: torch.Tensor | None = None,
                                  dev_status: torch.Tensor | None = None, stream=None):
    """:func:`paged_attention_varlen` where the query at position p sees key j only
    if ``p - j < window`` or ``j < num_sink`` (window 0: every key before it).

    Blocks that hide every key from every query of their request are not read:
    their ``block_table`` entries may hold anything. Returns ``(out, out_lse)``;
    ``out`` is bf16 [T,H,D] (fp32 where a fp32 tensor is given). The workspace
    (``window_attention_workspace_size`` bytes, uint8) needs no clearing and is
    allocated for the call where none is given."""
    return _window_attention(q, kv_pool, None, block_table, cu_seqlens, seq_lens, max_query_len,
                             max_seq_len, window, num_sink, out, out_lse, scale, workspace,
                             dev_status, stream)


def paged_attention_varlen_fp8(q: torch.Tensor, kv_pool: torch.Tensor, kv_scales: torch.Tensor,
                               block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                               seq_lens: torch.Tensor, max_query_len: int, max_seq_len: int, *,
                               window: int = 0, num_sink: int = 0,
                               out: torch.Tensor | None = None,
                               out_lse: torch.Tensor | None = None, scale: float | None = None,
                               workspace: torch.Tensor | None = None,
                               dev_status: torch.Tensor | None = None, stream=None):
    """Causal GQA attention over the 8-bit pool [2,NB,BS,Hkv,D] float8_e4m3fn,
    whose values stand for themselves times ``kv_scales`` [2,NB,Hkv] fp32; through
    a window where one is given (:func:`paged_attention_varlen_window`, whose
    other arguments and results these are)."""
    return _window_attention(q, kv_pool, kv_scales, block_table, cu_seqlens, seq_lens,
                             max_query_len, max_seq_len, window, num_sink, out, out_lse, scale,
                             workspace, dev_status, stream)


def _window_attention(q, kv_pool, kv_scales, block_table, cu_seqlens, seq_lens, max_query_len,
                      max_seq_len, window, num_sink, out, out_lse, scale, workspace, dev_status,
                      stream):
    native = _native or _marshal()
    if native.debug_checks():
        debug_checks.check_attention_tables(
            cu_seqlens, seq_lens, block_table, num_tokens=q.shape[0],
            max_query_len=int(max_query_len), max_seq_len=int(max_seq_len),
            num_blocks=kv_pool.shape[1], block_size=kv_pool.shape[2], window=int(window),
            num_sink=int(num_sink), padded=True)
    if stream is not None and (out is None or workspace is None):
        # what is made here belongs to the call's stream
        with _on_stream(stream, q.device):
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if workspace is None:
                workspace = torch.empty(window_attention_workspace_size(
                    int(max_query_len), q.shape[1], kv_pool.shape[3], q.shape[2], int(max_seq_len),
                    int(window), int(num_sink), kv_scales is not None), dtype=torch.uint8, device=q.device)
    out = native.window_attention(
        q, kv_pool, kv_scales, block_table, cu_seqlens, seq_lens, max_query_len, max_seq_len,
        window, num_sink, out, out_lse, scale, workspace, dev_status, _handle_of(stream))
    return out, out_lse


def attention_key_weights(q: torch.Tensor, kv_pool: torch.Tensor, lse: torch.Tensor,
                          block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                          seq_lens: torch.Tensor, max_query_len: int, max_seq_len: int,
                          weights: torch.Tensor, *, out: torch.Tensor | None = None,
                          weight_rows: torch.Tensor | None = None,
                          prior_lens: torch.Tensor | None = None, decay: float = 1.0,
                          scale: float | None = None, dev_status: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """Add a step's softmax weights to each cached key's running sum.

    ``lse`` [T,H] is the attention call's ``out_lse``; ``weights``
    [rows,Hkv,row_len] fp32 the sums so far, request i's in row
    ``weight_rows[i]`` (default i). Keys at or behind ``prior_lens[i]``
    (default: the step's own tokens) start from zero; ``decay`` scales the
    others' old sums. Writes and returns ``out`` (default: ``weights``, in place)."""
    native = _native or _marshal()
    if native.debug_checks():
        debug_checks.check_attention_tables(
            cu_seqlens, seq_lens, block_table, num_tokens=q.shape[0],
            max_query_len=int(max_query_len), max_seq_len=int(max_seq_len),
            num_blocks=kv_pool.shape[1], block_size=kv_pool.shape[2])
        debug_checks.check_weight_rows(weight_rows, num_seqs=seq_lens.shape[0],
                                       num_rows=weights.shape[0])
    return native.attention_key_weights(
        q, kv_pool, lse, block_table, cu_seqlens, seq_lens, max_query_len, max_seq_len, weights,
        out, weight_rows, prior_lens, decay, scale, dev_status, _handle_of(stream))


def evict_select(weights: torch.Tensor, seq_lens: torch.Tensor, keep_lens: torch.Tensor,
                 max_seq_len: int, max_keep_len: int, *, num_sink: int = 0, num_recent: int = 0,
                 weight_rows: torch.Tensor | None = None, kept: torch.Tensor | None = None,
                 weights_out: torch.Tensor | None = None,
                 dev_status: torch.Tensor | None = None, stream=None):
    """Choose the ``keep_lens[i]`` keys that each KV head of request i keeps.

    The last ``num_recent`` and first ``num_sink`` keys stay whatever their
    weight, the rest of the budget goes to the heaviest (ties: the lowest
    index). Returns ``(kept, weights_out)``: kept [B,Hkv,max_keep_len] int32,
    ascending, filled up to ``keep_lens[i]`` (a tensor made here holds -1
    behind that); ``weights_out``, when given, receives the kept keys' weights
    at the front of the same rows. ``weights`` keeps the sums of the uncut
    contexts: go on with ``weights_out`` when every row in use was in the call,
    else copy its rows back."""
    native = _native or _marshal()
    if native.debug_checks():
        debug_checks.check_weight_rows(weight_rows, num_seqs=seq_lens.shape[0],
                                       num_rows=weights.shape[0])
        debug_checks.check_keep_lens(seq_lens, keep_lens, max_seq_len=int(max_seq_len),
                                     max_keep_len=int(max_keep_len))
    if kept is None:
        _need(weights, torch.float32, 3, "weights")
        shape, device = (seq_lens.shape[0], weights.shape[1], int(max_keep_len)), weights.device
        if stream is None:
            kept = torch.full(shape, -1, dtype=torch.int32, device=device)
        else:
            with _on_stream(stream, device):
                kept = torch.full(shape, -1, dtype=torch.int32, device=device)
    native.evict_select(
        weights, seq_lens, keep_lens, max_seq_len, max_keep_len, num_sink, num_recent, weight_rows,
        kept, weights_out, dev_status, _handle_of(stream))
    return kept, weights_out


def evict_compact(kv_pool: torch.Tensor, src_table: torch.Tensor, dst_table: torch.Tensor,
                  kept: torch.Tensor, keep_lens: torch.Tensor, *,
                  dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Copy the kept keys' K and V rows (``kept`` of :func:`evict_select`) from
    the blocks of ``src_table`` to the front of those of ``dst_table``, which
    must be other blocks (``BlockManager.evict_step`` hands both out)."""
    native = _native or _marshal()
    if native.debug_checks():
        debug_checks.check_compaction(src_table, dst_table, kept, keep_lens,
                                      num_blocks=kv_pool.shape[1], block_size=kv_pool.shape[2])
    native.evict_compact(kv_pool, src_table, dst_table, kept, keep_lens, dev_status,
                         _handle_of(stream))
