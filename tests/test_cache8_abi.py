"""Refusals of the normed writes, of the 8-bit cache and of attention through a
window, at the C ABI and by the debug checks (CPU only: on a host without a GPU
a call that passes every check fails at its first CUDA step, status 3)."""
import ctypes

import numpy as np
import pytest

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)
MB = 1 << 20
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_varlen_gb300 import binding, build

    build.build()
    return binding.load_library()


# Every buffer has an address range of its own.
def _write(lib, **over):
    args = dict(q_out=256 * MB, kv_pool=512 * MB, q=64 * MB, k=96 * MB, v=128 * MB, q_stride=1024,
                k_stride=256, v_stride=256, positions=16 * MB, slots=17 * MB, inv_freq=18 * MB,
                q_weight=19 * MB, k_weight=20 * MB, weights_f32=0, weight_offset=0.0, eps=1e-6,
                factor=1.0, interleaved=0, num_tokens=10, num_heads=8, num_kv_heads=2,
                head_dim=128, rotary_dim=128, num_blocks=64, block_size=16, dev_status=None,
                stream=None)
    assert set(over) <= set(args)
    args.update(over)
    return lib.pkv_qk_norm_rope_kv_cache_write(*args.values())


def _append(lib, **over):
    args = dict(kv_pool=512 * MB, scales=21 * MB, k=96 * MB, v=128 * MB, k_stride=256,
                v_stride=256, block_table=22 * MB, max_blocks=8, cu=23 * MB, lens=24 * MB,
                num_seqs=3, num_tokens=10, max_query_len=6, num_kv_heads=2, head_dim=128,
                num_blocks=64, block_size=16, dev_status=None, stream=None)
    assert set(over) <= set(args)
    args.update(over)
    return lib.pkv_kv_cache_append_fp8(*args.values())


def _norm_append(lib, **over):
    args = dict(q_out=256 * MB, kv_pool=512 * MB, scales=21 * MB, q=64 * MB, k=96 * MB, v=128 * MB,
                q_stride=1024, k_stride=256, v_stride=256, positions=16 * MB, block_table=22 * MB,
                max_blocks=8, cu=23 * MB, lens=24 * MB, inv_freq=18 * MB, q_weight=19 * MB,
                k_weight=20 * MB, weights_f32=0, weight_offset=0.0, eps=1e-6, factor=1.0,
                interleaved=0, num_seqs=3, num_tokens=10, max_query_len=6, num_heads=8,
                num_kv_heads=2, head_dim=128, rotary_dim=128, num_blocks=64, block_size=16,
                dev_status=None, stream=None)
    assert set(over) <= set(args)
    args.update(over)
    return lib.pkv_qk_norm_rope_kv_cache_append_fp8(*args.values())


def _window(lib, eight=False, **over):
    args = dict(out=256 * MB, out_f32=0, out_lse=None, q=64 * MB, kv_pool=512 * MB)
    if eight:
        args["scales"] = 21 * MB
    args.update(block_table=22 * MB, max_blocks=64, cu=23 * MB, lens=24 * MB, num_seqs=3,
                num_tokens=10, max_query_len=6, max_seq_len=1000, num_heads=8, num_kv_heads=2,
                head_dim=128, block_size=16, num_blocks=64, window=100, num_sink=4, scale=0.088,
                workspace=1024 * MB, workspace_bytes=64 * MB, dev_status=None, stream=None)
    assert set(over) <= set(args)
    args.update(over)
    f = lib.pkv_paged_attention_varlen_fp8 if eight else lib.pkv_paged_attention_varlen_window
    return f(*args.values())


def _copy(lib, **over):
    args = dict(kv_pool=512 * MB, scales=21 * MB, src=16 * MB, dst=17 * MB, num_copies=2,
                num_blocks=64, block_size=16, num_kv_heads=2, head_dim=128, dev_status=None,
                stream=None)
    assert set(over) <= set(args)
    args.update(over)
    return lib.pkv_copy_blocks_fp8(*args.values())


ROWS = [
    ({"kv_pool": None}, INVALID), ({"k": None}, INVALID), ({"v": None}, INVALID),
    ({"kv_pool": 512 * MB + 8}, INVALID), ({"k": 96 * MB + 2}, INVALID),
    ({"v": 128 * MB + 8}, INVALID), ({"k_stride": 255}, INVALID), ({"v_stride": 248}, INVALID),
    ({"k_stride": 260}, INVALID), ({"num_tokens": -1}, INVALID), ({"num_kv_heads": 0}, INVALID),
    ({"head_dim": 0}, INVALID), ({"num_blocks": 0}, INVALID), ({"block_size": -16}, INVALID),
    ({"num_tokens": 0}, OK), ({}, CUDA),
]
NORMS = [
    ({"q": None}, INVALID), ({"q_out": None}, INVALID), ({"positions": None}, INVALID),
    ({"inv_freq": None}, INVALID), ({"inv_freq": None, "rotary_dim": 0}, CUDA),
    ({"q": 64 * MB + 8}, INVALID), ({"q_out": 256 * MB + 4}, INVALID),
    ({"inv_freq": 18 * MB + 4}, INVALID), ({"q_weight": 19 * MB + 1}, INVALID),
    ({"k_weight": 20 * MB + 2, "weights_f32": 1}, INVALID),
    ({"q_weight": None, "k_weight": None}, CUDA), ({"q_stride": 1016}, INVALID),
    ({"q_stride": 1028}, INVALID), ({"rotary_dim": 130}, INVALID), ({"rotary_dim": 33}, INVALID),
    ({"rotary_dim": -2}, INVALID), ({"eps": -1e-9}, INVALID), ({"eps": float("nan")}, INVALID),
    ({"eps": float("inf")}, INVALID), ({"weight_offset": float("inf")}, INVALID),
    ({"factor": float("nan")}, INVALID), ({"num_heads": 0}, INVALID),
    # q_out over what is read or written; over q itself only as a whole
    ({"q_out": 512 * MB}, INVALID), ({"q_out": 96 * MB}, INVALID), ({"q_out": 128 * MB}, INVALID),
    ({"q_out": 64 * MB}, CUDA), ({"q_out": 64 * MB + 16}, INVALID),
    ({"q_out": 64 * MB, "q_stride": 1032}, INVALID),
    ({"q_out": 64 * MB, "q_stride": 1032, "num_tokens": 1, "k_stride": 256}, CUDA),
]


@pytest.mark.parametrize("over,status", ROWS + NORMS + [
    ({"slots": None}, INVALID), ({"head_dim": 100, "rotary_dim": 100}, UNSUPPORTED),
    ({"head_dim": 520, "q_stride": 4160, "k_stride": 1040, "v_stride": 1040}, UNSUPPORTED),
    ({"head_dim": 40, "rotary_dim": 40}, CUDA), ({"block_size": 7}, CUDA),
    ({"num_tokens": INT_MAX}, UNSUPPORTED),
    ({"num_heads": INT_MAX // 128, "q_stride": 2 ** 31}, UNSUPPORTED),
])
def test_normed_write(lib, over, status):
    assert _write(lib, **over) == status


APPENDS = [
    ({"scales": None}, INVALID), ({"block_table": None}, INVALID), ({"cu": None}, INVALID),
    ({"lens": None}, INVALID), ({"scales": 21 * MB + 2}, INVALID), ({"num_seqs": 0}, INVALID),
    ({"num_seqs": -1}, INVALID), ({"max_query_len": 0}, INVALID), ({"max_blocks": 0}, INVALID),
    ({"max_query_len": 1}, CUDA), ({"scales": 512 * MB + 1024}, INVALID),
    ({"block_size": 8}, UNSUPPORTED), ({"block_size": 24}, UNSUPPORTED),
    ({"block_size": 272}, UNSUPPORTED), ({"block_size": 256}, CUDA),
    ({"max_blocks": INT_MAX // 8}, UNSUPPORTED), ({"num_blocks": 2 ** 27}, UNSUPPORTED),
    ({"num_tokens": INT_MAX - 70000, "num_seqs": 2 ** 30}, UNSUPPORTED),
]


@pytest.mark.parametrize("over,status", ROWS + APPENDS + [
    ({"head_dim": 96}, UNSUPPORTED), ({"head_dim": 256, "k_stride": 512, "v_stride": 512},
                                      UNSUPPORTED)])
def test_append(lib, over, status):
    assert _append(lib, **over) == status


@pytest.mark.parametrize("over,status", ROWS + NORMS + APPENDS + [
    ({"head_dim": 96, "rotary_dim": 96}, UNSUPPORTED),
    ({"q_out": 21 * MB}, INVALID),   # over the scales
])
def test_norm_append(lib, over, status):
    assert _norm_append(lib, **over) == status


@pytest.mark.parametrize("over,status", [
    ({"kv_pool": None}, INVALID), ({"scales": None}, INVALID), ({"src": None}, INVALID),
    ({"dst": None}, INVALID), ({"kv_pool": 512 * MB + 8}, INVALID),
    ({"scales": 21 * MB + 1}, INVALID), ({"num_copies": -1}, INVALID), ({"num_copies": 0}, OK),
    ({"num_blocks": 0}, INVALID), ({"head_dim": 1, "num_kv_heads": 1, "block_size": 8}, UNSUPPORTED),
    ({"num_copies": 65536}, UNSUPPORTED), ({}, CUDA),
])
def test_copy_blocks(lib, over, status):
    assert _copy(lib, **over) == status


ATTENTION = [
    ({"out": None}, INVALID), ({"q": None}, INVALID), ({"kv_pool": None}, INVALID),
    ({"block_table": None}, INVALID), ({"cu": None}, INVALID), ({"lens": None}, INVALID),
    ({"out": 256 * MB + 8}, INVALID), ({"q": 64 * MB + 8}, INVALID),
    ({"kv_pool": 512 * MB + 8}, INVALID), ({"out_lse": 25 * MB + 2}, INVALID),
    ({"num_seqs": 0}, INVALID), ({"num_seqs": -1}, INVALID), ({"num_tokens": -1}, INVALID),
    ({"num_tokens": 0}, OK), ({"num_seqs": 65535}, UNSUPPORTED), ({"num_heads": 7}, INVALID),
    ({"num_kv_heads": 0}, INVALID), ({"max_query_len": 0}, INVALID),
    ({"max_seq_len": 5}, INVALID), ({"window": -1}, INVALID), ({"num_sink": -1}, INVALID),
    ({"scale": 0.0}, INVALID), ({"scale": float("nan")}, INVALID),
    ({"scale": float("inf")}, INVALID), ({"max_blocks": 0}, INVALID), ({"block_size": 0}, INVALID),
    ({"num_blocks": 0}, INVALID), ({"head_dim": 96}, UNSUPPORTED), ({"block_size": 8}, UNSUPPORTED),
    ({"block_size": 272}, UNSUPPORTED), ({"num_blocks": 2 ** 27}, UNSUPPORTED),
    ({"max_blocks": INT_MAX // 8}, UNSUPPORTED), ({"max_seq_len": 2 ** 30}, UNSUPPORTED),
    ({"workspace": None}, WORKSPACE), ({"workspace_bytes": 255}, WORKSPACE),
    ({"workspace": 1024 * MB + 128}, WORKSPACE),
    # longer requests: more heads to a KV head than a query tile has rows, more requests
    # than their list has room for
    ({"max_query_len": 40, "num_heads": 258}, UNSUPPORTED),
    ({"max_query_len": 40, "num_seqs": 4416}, UNSUPPORTED),
    ({"max_query_len": 1, "num_heads": 258, "num_seqs": 4416}, CUDA),
    # results over inputs, over one another, over the workspace
    ({"out": 64 * MB}, INVALID), ({"out": 512 * MB + 1024}, INVALID),
    ({"out_lse": 256 * MB + 64}, INVALID), ({"out_lse": 512 * MB}, INVALID),
    ({"out_lse": 64 * MB + 4}, INVALID), ({"workspace": 64 * MB}, INVALID),
    ({"workspace": 256 * MB}, INVALID), ({"workspace": 512 * MB}, INVALID),
    ({"out_lse": 25 * MB}, CUDA), ({"out": 64 * MB + 20480}, CUDA),
    ({"window": 0}, CUDA), ({"window": INT_MAX, "num_sink": INT_MAX}, CUDA),
    ({"max_query_len": 40}, CUDA), ({}, CUDA),
]


@pytest.mark.parametrize("over,status", ATTENTION)
@pytest.mark.parametrize("eight", [False, True])
def test_attention(lib, eight, over, status):
    assert _window(lib, eight, **over) == status


@pytest.mark.parametrize("over", [{"scales": None}, {"scales": 21 * MB + 2}, {"out": 21 * MB},
                                  {"workspace": 21 * MB}])
def test_attention_over_no_scales(lib, over):
    assert _window(lib, True, **over) == INVALID


def test_workspace_sizes(lib):
    size = lib.pkv_window_attention_workspace_size
    # nothing to join, no longer requests: a few bytes
    assert size(1, 32, 8, 128, 256, 0, 0, 0) == 256
    assert size(1, 32, 8, 128, 1 << 20, 100, 4, 1) == 256
    for eight in (0, 1):
        for q in (1, 8, 9, 8192):
            for d in (64, 128):
                n = size(q, 32, 8, d, 131072, 0, 0, eight)
                assert 256 <= n <= (13 * 10 ** 6 if q <= 8 else 54 * 10 ** 6)
                assert _window(lib, bool(eight), max_query_len=q, num_heads=32, num_kv_heads=8,
                               head_dim=d, max_seq_len=131072, window=0, num_sink=0,
                               max_blocks=8192, workspace_bytes=n) == CUDA
                assert _window(lib, bool(eight), max_query_len=q, num_heads=32, num_kv_heads=8,
                               head_dim=d, max_seq_len=131072, window=0, num_sink=0,
                               max_blocks=8192, workspace_bytes=n - 1) == WORKSPACE
    for bad in ((0, 32, 8, 128, 10, 0, 0, 0), (1, 0, 8, 128, 10, 0, 0, 0),
                (1, 30, 8, 128, 10, 0, 0, 0), (1, 32, 8, 96, 10, 0, 0, 0),
                (1, 32, 8, 128, 0, 0, 0, 0), (1, 32, 8, 128, 10, -1, 0, 0),
                (1, 32, 8, 128, 10, 0, -1, 0)):
        assert size(*bad) == 0


def test_debug_checks():
    from paged_kv_cache_varlen_gb300 import debug_checks as dc

    table = np.array([[3, 1, -1, 7], [2, 0, 4, -1]])
    ok = dict(num_tokens=4, max_query_len=3, num_blocks=8, block_size=16)
    # the new tokens' blocks alone count: entry 0 of a row may be anything
    dc.check_append_tables([0, 1, 4], [20, 40], table, **ok)
    dc.check_append_tables([0, 1, 4], [20, 40], np.where(table == 3, 99, table), **ok)
    for cu, lens, t in (
            ([0, 1, 4], [20, 50], table),                             # a block that is not there
            ([0, 1, 4], [2, 40], np.where(table == 3, 4, table)),     # a block of both
            ([0, 4, 4], [20, 40], table),                             # too many queries
            ([0, 1, 4], [20, 2], table)):                             # shorter than its queries
        with pytest.raises(ValueError):
            dc.check_append_tables(cu, lens, t, **ok)
    # attention through a window: entries that no query sees may be anything
    t = np.array([[0, -1, -1, 5, 6]])
    args = dict(num_tokens=2, max_query_len=2, max_seq_len=80, num_blocks=8, block_size=16)
    dc.check_attention_tables([0, 2], [80], t, window=31, num_sink=9, **args)
    for w, s in ((32, 9), (31, 17), (0, 0)):
        with pytest.raises(ValueError):
            dc.check_attention_tables([0, 2], [80], t, window=w, num_sink=s, **args)


def test_the_library_has_every_signature(lib):
    from paged_kv_cache_varlen_gb300 import binding

    for n in ("pkv_copy_blocks_fp8", "pkv_kv_cache_append_fp8", "pkv_paged_attention_varlen_fp8",
              "pkv_paged_attention_varlen_window", "pkv_qk_norm_rope_kv_cache_append_fp8",
              "pkv_qk_norm_rope_kv_cache_write", "pkv_window_attention_workspace_size"):
        assert isinstance(getattr(lib, n), ctypes._CFuncPtr) and n in binding._SIGNATURES
