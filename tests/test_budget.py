"""Rotary frequencies, refusals of the rotary cache write and the cache-budget
calls, the block manager's eviction step and the debug checks (CPU only: no
kernel runs here)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_varlen_gb300 import binding, build, debug_checks


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


# ---------------------------------------------------------------- frequencies
def test_plain_and_linear_frequencies(lib):
    f, m = binding.rope_frequencies(8, 10000.0)
    assert m == 1.0 and f.dtype == torch.float64
    np.testing.assert_allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-14)
    g, m = binding.rope_frequencies(8, 10000.0, scaling="linear", stretch=4.0)
    np.testing.assert_allclose(g.numpy(), f.numpy() / 4, rtol=1e-14)
    assert m == 1.0


def test_base_scaling_stretches_the_slowest_pair_in_full(lib):
    f, _ = binding.rope_frequencies(64, 10000.0)
    g, _ = binding.rope_frequencies(64, 10000.0, scaling="base", stretch=8.0)
    assert g[0] == f[0]
    assert math.isclose(g[-1], f[-1] / 8, rel_tol=1e-12)


def test_band_scaling(lib):
    n, s = 8192.0, 8.0
    f, _ = binding.rope_frequencies(128, 500000.0)
    g, m = binding.rope_frequencies(128, 500000.0, scaling="bands", stretch=s, original_len=n)
    assert m == 1.0
    for a, b in zip(f.tolist(), g.tolist()):
        turns = n * a / (2 * math.pi)
        if turns >= 4:
            assert b == a
        elif turns <= 1:
            assert math.isclose(b, a / s, rel_tol=1e-14)
        else:
            w = (turns - 1) / 3
            assert math.isclose(b, (1 - w) * a / s + w * a, rel_tol=1e-13)


def test_ramp_scaling(lib):
    n, s, r, base = 4096.0, 16.0, 128, 10000.0
    f, _ = binding.rope_frequencies(r, base)
    g, m = binding.rope_frequencies(r, base, scaling="ramp", stretch=s, original_len=n)
    assert math.isclose(m, 0.1 * math.log(s) + 1, rel_tol=1e-7)
    index = lambda turns: r * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(0, math.floor(index(32))), min(r - 1, math.ceil(index(1)))
    for p, (a, b) in enumerate(zip(f.tolist(), g.tolist())):
        w = min(1.0, max(0.0, (p - lo) / (hi - lo)))
        assert math.isclose(b, a * (1 - w) + a / s * w, rel_tol=1e-13)


@pytest.mark.parametrize("args,kw", [
    ((7,), {}), ((0,), {}), ((-2,), {}), ((8, 1.0), {}), ((8, float("inf")), {}),
    ((8,), dict(scaling="linear", stretch=0.5)),
    ((8,), dict(scaling="linear", stretch=float("nan"))),
    ((2,), dict(scaling="base", stretch=2.0)),
    ((8,), dict(scaling="bands", stretch=2.0)),
    ((8,), dict(scaling="bands", stretch=2.0, original_len=100, low=4.0, high=4.0)),
    ((8,), dict(scaling="ramp", stretch=2.0, original_len=100, low=0.0)),
])
def test_frequency_refusals(lib, args, kw):
    with pytest.raises(binding.PkvError) as e:
        binding.rope_frequencies(*args, **kw)
    assert e.value.status == 1


def test_unknown_scaling_is_refused(lib):
    with pytest.raises(ValueError):
        binding.rope_frequencies(8, scaling="other")


# ------------------------------------------------------------------- refusals
A = 1 << 20  # fake, 16-byte aligned device addresses, far apart: nothing launches


def _rope(lib, **over):
    a = dict(q_out=A, kv_pool=2 * A, q=3 * A, k=4 * A, v=5 * A, q_stride=512, k_stride=256,
             v_stride=256, positions=6 * A, slots=7 * A, inv_freq=8 * A, factor=1.0, inter=0,
             tokens=2, heads=4, kv_heads=2, head_dim=128, rotary=128, blocks=4, bs=16, status=None,
             stream=None)
    a.update(over)
    return lib.pkv_rope_kv_cache_write(*a.values())


@pytest.mark.parametrize("over,status", [
    ({"tokens": -1}, 1), ({"heads": 0}, 1), ({"kv_heads": 0}, 1), ({"blocks": 0}, 1),
    ({"bs": 0}, 1), ({"rotary": 0}, 1), ({"rotary": 7}, 1), ({"rotary": 130}, 1),
    ({"factor": float("nan")}, 1), ({"factor": float("inf")}, 1),
    ({"q_out": None}, 1), ({"kv_pool": None}, 1), ({"q": None}, 1), ({"k": None}, 1),
    ({"v": None}, 1), ({"positions": None}, 1), ({"slots": None}, 1), ({"inv_freq": None}, 1),
    ({"q": 3 * A + 8}, 1), ({"inv_freq": 8 * A + 4}, 1),
    ({"q_stride": 504}, 1), ({"k_stride": 260}, 1), ({"v_stride": 248}, 1),
    ({"head_dim": 132, "rotary": 64, "q_stride": 528, "k_stride": 264, "v_stride": 264}, 2),
    ({"head_dim": 520, "rotary": 64, "q_stride": 2080, "k_stride": 1040, "v_stride": 1040}, 2),
    # halves that are no multiple of a vector stage a token's heads on chip
    ({"heads": 1024, "rotary": 20, "q_stride": 131072}, 2),
    ({"q_out": 4 * A}, 1),                      # over k_new
    ({"q_out": 5 * A - 2048 + 16}, 1),          # into v_new
    ({"q_out": 3 * A + 1024}, 1),               # half over q
    ({"q_out": 3 * A, "q_stride": 1024}, 1),    # in place, but q is not dense
])
def test_rope_refusals(lib, over, status):
    assert _rope(lib, **over) == status


def test_rope_output_over_the_pool_and_token_counts_past_the_grid(lib):
    assert _rope(lib, q_out=2 * A) == 1                    # over the K half
    assert _rope(lib, q_out=2 * A + 4 * 16 * 256 * 2) == 1   # over the V half
    assert _rope(lib, tokens=2 ** 31 - 1) == 2


def test_contexts_past_the_index_range_are_refused(lib):
    assert _weights(lib, max_len=2 ** 30, row_len=2 ** 30, inp=A) == 2
    assert _select(lib, max_len=2 ** 30, row_len=2 ** 30) == 2


def test_rope_of_no_tokens_is_a_no_op(lib):
    assert _rope(lib, tokens=0, q=None, q_out=None) == 0


def _weights(lib, **over):
    a = dict(out=A, inp=A, q=2 * A, pool=3 * A, lse=4 * A, table=5 * A, max_blocks=4, cu=6 * A,
             lens=7 * A, prior=None, rows=None, num_rows=2, row_len=64, seqs=2, tokens=2, max_q=1,
             max_len=64, heads=4, kv_heads=2, head_dim=128, bs=16, blocks=8, scale=0.1, decay=1.0,
             status=None, stream=None)
    a.update(over)
    return lib.pkv_attention_key_weights(*a.values())


@pytest.mark.parametrize("over,status", [
    ({"tokens": -1}, 1), ({"seqs": 0}, 1), ({"seqs": 65535, "num_rows": 65535}, 2),
    ({"out": None}, 1), ({"inp": None}, 1), ({"q": None}, 1), ({"pool": None}, 1),
    ({"lse": None}, 1), ({"table": None}, 1), ({"cu": None}, 1), ({"lens": None}, 1),
    ({"heads": 5}, 1), ({"max_blocks": 0}, 1), ({"num_rows": 0}, 1), ({"num_rows": 1}, 1),
    ({"max_q": 0}, 1), ({"max_q": 65}, 1), ({"row_len": 63}, 1),
    ({"scale": 0.0}, 1), ({"scale": float("nan")}, 1), ({"decay": -0.5}, 1),
    ({"decay": float("inf")}, 1), ({"q": 2 * A + 2}, 1),
    ({"inp": A + 4}, 1),                        # overlaps the output
    ({"head_dim": 96}, 2), ({"bs": 8}, 2), ({"bs": 512}, 2),
    ({"blocks": 1 << 27}, 2),
])
def test_key_weights_refusals(lib, over, status):
    assert _weights(lib, **over) == status


def test_key_weights_of_no_tokens_is_a_no_op(lib):
    assert _weights(lib, tokens=0, out=None) == 0


def _select(lib, **over):
    a = dict(kept=A, out=None, weights=2 * A, lens=3 * A, keep=4 * A, rows=None, num_rows=2,
             row_len=64, seqs=2, kv_heads=2, max_len=64, max_keep=32, sink=1, recent=2,
             status=None, stream=None)
    a.update(over)
    return lib.pkv_evict_select(*a.values())


@pytest.mark.parametrize("over,status", [
    ({"seqs": -1}, 1), ({"kv_heads": 0}, 1), ({"sink": -1}, 1), ({"recent": -1}, 1),
    ({"max_len": -1}, 1), ({"max_keep": -1}, 1), ({"seqs": 65535, "num_rows": 65535}, 2),
    ({"kept": None}, 1), ({"weights": None}, 1), ({"lens": None}, 1), ({"keep": None}, 1),
    ({"row_len": 63}, 1), ({"num_rows": 1}, 1), ({"out": 2 * A}, 1), ({"out": 2 * A + 1020}, 1),
    ({"out": 5 * A, "max_keep": 65}, 1), ({"weights": 2 * A + 2}, 1),
])
def test_select_refusals(lib, over, status):
    assert _select(lib, **over) == status


def test_select_of_nothing_is_a_no_op(lib):
    assert _select(lib, seqs=0, kept=None) == 0
    assert _select(lib, max_keep=0, kept=None) == 0


def _compact(lib, **over):
    a = dict(pool=A, src=2 * A, max_src=4, dst=3 * A, max_dst=4, kept=4 * A, max_keep=32,
             keep=5 * A, seqs=2, kv_heads=2, head_dim=128, bs=16, blocks=16, status=None,
             stream=None)
    a.update(over)
    return lib.pkv_evict_compact(*a.values())


@pytest.mark.parametrize("over,status", [
    ({"seqs": -1}, 1), ({"kv_heads": 0}, 1), ({"bs": 0}, 1), ({"blocks": 0}, 1),
    ({"max_src": -1}, 1), ({"max_keep": -1}, 1), ({"seqs": 65535}, 2),
    ({"pool": None}, 1), ({"src": None}, 1), ({"dst": None}, 1), ({"kept": None}, 1),
    ({"keep": None}, 1), ({"pool": A + 8}, 1), ({"head_dim": 100}, 2), ({"head_dim": 1024}, 2),
    ({"max_src": 1 << 28}, 2),
])
def test_compact_refusals(lib, over, status):
    assert _compact(lib, **over) == status


def test_compact_of_nothing_is_a_no_op(lib):
    assert _compact(lib, seqs=0, pool=None) == 0
    assert _compact(lib, max_keep=0, pool=None) == 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 2, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.rope_kv_cache_write(x[0, 0, :2], x, x[0, 0, :2], x[0, 0, :2], i, i,
                                    torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.evict_select(torch.zeros(2, 2, 8), i, i, 8, 4)
    with pytest.raises(ValueError):
        binding.evict_compact(x, i.view(2, 1), i.view(2, 1), i.view(2, 1, 1), i)


# --------------------------------------------------------------- block manager
def test_evict_step_moves_to_fresh_blocks(lib):
    bm = binding.BlockManager(16, 4)
    for s, n in ((1, 13), (2, 9)):
        bm.add_seq(s)
        bm.append(s, n)
    old = {s: bm.block_table(s) for s in (1, 2)}
    src, dst = bm.evict_step([2, 1], [5, 4], 4, 3)
    assert src.tolist() == [old[2] + [-1], old[1]]
    assert dst.tolist() == [bm.block_table(2) + [-1], bm.block_table(1) + [-1, -1]]
    assert len(bm.block_table(2)) == 2 and len(bm.block_table(1)) == 1
    assert not set(dst[dst >= 0].tolist()) & set(src[src >= 0].tolist())
    assert bm.seq_len(1) == 4 and bm.seq_len(2) == 5
    assert bm.num_free() == 13
    slots, copies = bm.append(2, 1)
    assert slots == [bm.block_table(2)[1] * 4 + 1] and copies == []


def test_evict_step_leaves_shared_blocks_with_their_other_owner(lib):
    bm = binding.BlockManager(8, 4)
    bm.add_seq(1)
    bm.append(1, 8)
    bm.fork(1, 2)
    table = bm.block_table(1)
    src, dst = bm.evict_step([2], [4], 2, 1)
    assert src.tolist() == [table]
    assert bm.block_table(1) == table and [bm.refcount(b) for b in table] == [1, 1]
    assert bm.refcount(int(dst[0, 0])) == 1 and bm.num_free() == 5


def test_evict_step_to_nothing_and_of_nothing(lib):
    bm = binding.BlockManager(4, 4)
    bm.add_seq(1)
    bm.append(1, 5)
    src, dst = bm.evict_step([1], [0], 2, 0)
    assert dst.shape == (1, 0) and bm.num_free() == 4 and bm.seq_len(1) == 0
    src, dst = bm.evict_step([], [], 2, 2)
    assert src.shape == (0, 2)


@pytest.mark.parametrize("ids,keep,ms,md,status", [
    ([9], [1], 4, 4, 1), ([1, 1], [1, 1], 4, 4, 1), ([1], [-1], 4, 4, 1), ([1], [10], 4, 4, 1),
    ([1], [5], 2, 4, 1), ([1], [5], 4, 1, 1), ([1, 2], [9, 9], 4, 4, 5),
])
def test_evict_step_refusals_change_nothing(lib, ids, keep, ms, md, status):
    bm = binding.BlockManager(8, 4)
    for s in (1, 2):
        bm.add_seq(s)
        bm.append(s, 9)
    before = (bm.num_free(), bm.block_table(1), bm.block_table(2))
    with pytest.raises(binding.PkvError) as e:
        bm.evict_step(ids, keep, ms, md)
    assert e.value.status == status
    assert before == (bm.num_free(), bm.block_table(1), bm.block_table(2))


# ---------------------------------------------------------------- debug checks
def test_debug_checks_of_the_budget_calls():
    debug_checks.check_positions([0, 5])
    debug_checks.check_weight_rows(None, num_seqs=2, num_rows=2)
    debug_checks.check_weight_rows([1, 0], num_seqs=2, num_rows=2)
    debug_checks.check_keep_lens([4, 0], [4, 0], max_seq_len=4, max_keep_len=4)
    ok = dict(num_blocks=8, block_size=4)
    debug_checks.check_compaction([[0, 1]], [[2]], [[[1, 6]]], [2], **ok)
    for call in (
        lambda: debug_checks.check_positions([3, -1]),
        lambda: debug_checks.check_weight_rows([0, 2], num_seqs=2, num_rows=2),
        lambda: debug_checks.check_weight_rows([1, 1], num_seqs=2, num_rows=2),
        lambda: debug_checks.check_keep_lens([4], [5], max_seq_len=4, max_keep_len=8),
        lambda: debug_checks.check_keep_lens([4], [3], max_seq_len=4, max_keep_len=2),
        lambda: debug_checks.check_keep_lens([5], [3], max_seq_len=4, max_keep_len=4),
        lambda: debug_checks.check_compaction([[0, 1]], [[2]], [[[1, 8]]], [2], **ok),
        lambda: debug_checks.check_compaction([[0, 8]], [[2]], [[[1, 6]]], [2], **ok),
        lambda: debug_checks.check_compaction([[0, 1]], [[-1]], [[[1, 6]]], [2], **ok),
        lambda: debug_checks.check_compaction([[0, 1]], [[1]], [[[1, 6]]], [2], **ok),
        lambda: debug_checks.check_compaction([[0, 1]], [[2]], [[[1, 6]]], [3], **ok),
        lambda: debug_checks.check_compaction([[0], [1]], [[2], [2]], [[[1]], [[1]]], [1, 1], **ok),
    ):
        with pytest.raises(ValueError):
            call()
