"""Block writes into the 8-bit cache beside requests whose lengths are no good: those
are flagged and skipped, every other request is written whole, nothing else changes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv
from paged_kv_cache_varlen_gb300 import binding

from . import plain_cache8 as plain
from .gpu_util import guarded, guards_intact
from .test_gpu_norm_write import f64, i32, normal, pool8, status_word, values

pytestmark = pytest.mark.gpu


def bad_lengths(cu, lens, t, max_q, room):
    """Whether each request is flagged, from the header's definition."""
    return [not (0 <= cu[i] <= cu[i + 1] <= t)
            or (cu[i] < cu[i + 1] and not (cu[i + 1] - cu[i] <= min(max_q, lens[i])
                                           and lens[i] <= room))
            for i in range(len(lens))]


def tables(cu, lens, bad, bs, room, seed):
    """Each good request's written blocks, shuffled, within a pool; -1 elsewhere."""
    r = np.random.RandomState(seed)
    spans = [(0, 0) if bad[i] or cu[i] == cu[i + 1]
             else ((lens[i] - cu[i + 1] + cu[i]) // bs, (lens[i] - 1) // bs + 1)
             for i in range(len(lens))]
    n = sum(b - a for a, b in spans)
    ids, at = r.permutation(n + 3), 0
    table = np.full((len(lens), room // bs), -1, np.int32)
    for i, (a, b) in enumerate(spans):
        table[i, a:b] = ids[at:at + b - a]
        at += b - a
    return table, n + 3


def many(seed):
    # cu_seqlens that now and then falls, is negative or passes the tokens
    r = np.random.RandomState(seed)
    n, t = 300, 2500
    cu = np.concatenate([[0], np.cumsum(r.choice([0, 1, 5, 17], n))])
    for i in r.permutation(n)[:25]:
        cu[i] = r.choice([-3, t + 9, int(r.randint(0, t))])
    lens = [max(1, int(b - a)) + int(r.randint(0, 60)) for a, b in zip(cu, cu[1:])]
    lens = [min(x, 512) for x in lens]
    return cu.tolist(), lens, t, 40


# cu_seqlens, seq_lens, tokens, max_query_len
CASES = {
    "falls": ([0, 160, 170, 0, 10], [160, 10, 7, 10], 170, 160),
    "falls far": ([0, 1000, 1010, 5, 40], [1000, 10, 7, 35], 1010, 1000),
    "negative": ([0, 50, -7, 30, 60], [70, 9, 40, 30], 60, 50),
    "past the tokens": ([0, 40, 5000, 40, 90], [41, 5000, 3, 100], 90, 50),
    "the same tokens": ([0, 100, 0, 100, 0, 100], [100, 5, 117, 5, 133], 100, 100),
    "not from 0": ([5, 30], [40], 33, 25),
    "too long": ([0, 60, 70, 90], [60, 2000, 25], 90, 60),
    "too many queries": ([0, 60, 70, 90], [60, 40, 25], 90, 20),
    "all bad": ([9, 3, 2], [20, 20], 12, 9),
    "many": many(1),
    "many more": many(2),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("bs,d", [(16, 128), (16, 64), (64, 128), (256, 64)])
def test_other_requests_are_written_whole(name, bs, d):
    cu, lens, t, max_q = CASES[name]
    h, hkv, room = 4, 2, 1024 if name.startswith("falls far") else 512
    bad = bad_lengths(cu, lens, t, max_q, room)
    assert any(bad) == (name != "not from 0")
    table, nb = tables(cu, lens, bad, bs, room, d)
    q, k, v = normal((t, h, d), 1), normal((t, hkv, d), 2, 3.0), normal((t, hkv, d), 3)
    pool, scales = pool8(nb, bs, hkv, d, bs)
    scales.view(-1)[::3] = 0.0  # (blocks as a new pool leaves them)
    want, ws = values(pool), f64(scales)
    seen = np.zeros(t, bool)
    for i, b in enumerate(bad):
        if not b:
            want, ws, _ = plain.append(want, ws, f64(k), f64(v), table[i:i + 1], cu[i:i + 2],
                                       lens[i:i + 1])
            seen[cu[i]:cu[i + 1]] = True
    for both in (False, True):
        buf, gp = guarded(pool.shape, torch.uint8)
        gp.copy_(pool.view(torch.uint8))
        sbuf, gs = guarded(scales.shape, torch.float32)
        gs.copy_(scales)
        obuf, out = guarded(q.shape, torch.bfloat16)
        out.fill_(7.0)
        # the table between entries that name a block of the pool
        wide = np.full((table.shape[0] + 200, table.shape[1]), 1, np.int32)
        wide[100:-100] = table
        tab, st = i32(wide)[100:-100], status_word()
        where = (tab, i32(cu), i32(lens), max_q)
        if both:
            pkv.qk_norm_rope_kv_cache_append_fp8(q, gp.view(torch.float8_e4m3fn), gs, k, v,
                                                 i32(np.arange(t)), *where, None, q_out=out,
                                                 dev_status=st)
            assert torch.equal(out[torch.from_numpy(seen)], q[torch.from_numpy(seen)])
            assert torch.all(out[torch.from_numpy(~seen)] == 7.0)
        else:
            pkv.kv_cache_append_fp8(gp.view(torch.float8_e4m3fn), gs, k, v, *where, dev_status=st)
        assert st.item() == (binding.DEV_BAD_LENGTHS if any(bad) else 0)
        assert np.array_equal(f64(gs), ws)
        assert np.array_equal(values(gp.view(torch.float8_e4m3fn)), want)
        assert guards_intact(buf, pool.numel()) and guards_intact(sbuf, scales.numel())
        assert guards_intact(obuf, q.numel())
