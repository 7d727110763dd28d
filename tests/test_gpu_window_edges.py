"""Attention through a window and over the 8-bit cache: padded batches, blocks that are
not there, scales whose products leave the fp32 range."""
import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv
from paged_kv_cache_varlen_gb300 import binding

from .gpu_util import guarded, guards_intact
from .test_gpu_window import BOTH, Step, f64, i32

pytestmark = pytest.mark.gpu


@BOTH
@pytest.mark.parametrize("rows", [20, 40, 200])
@pytest.mark.parametrize("ql", [[1, 40], [1, 40, 3, 0, 8, 33], [1, 2, 1, 40]])
@pytest.mark.parametrize("window,sink", [(0, 0), (30, 2)])
def test_padded_batches(eight, rows, ql, window, sink):
    # as many rows behind the last request as hide that some requests are short
    lens = [n + 60 * (i + 1) for i, n in enumerate(ql)]
    s = Step(lens, ql, 4, 2, 128, 16, window, sink, eight, seed=rows)
    t = s.q.shape[0]
    s.q = torch.cat([s.q, torch.full_like(s.q[:1], float("nan")).expand(rows, -1, -1)])
    buf, out = guarded(s.q.shape, torch.bfloat16)
    lbuf, lse = guarded(s.q.shape[:2], torch.float32)
    out.fill_(7.0)
    lse.fill_(7.0)
    s.call(out=out, out_lse=lse)
    assert torch.all(out[t:] == 7.0) and torch.all(lse[t:] == 7.0)
    s.q = s.q[:t].contiguous()
    s.check(out[:t], lse[:t])
    assert guards_intact(buf, out.numel()) and guards_intact(lbuf, lse.numel())


@pytest.mark.parametrize("ql", [[1, 3], [70, 40]])
@pytest.mark.parametrize("scale", [1e-20, 1e-38])
def test_factors_that_vanish(ql, scale):
    # blocks of next to no keys (the smallest scale that the writes leave) and a small
    # score scale: their product is 0 in fp32, and every key counts the same
    s = Step([100, 90], ql, 4, 2, 128, 16, 40, 3, True, seed=7)
    s.scales[0] *= 2.0 ** -90
    for k in s.k:
        k *= 2.0 ** -90
    s.check(*s.call(scale=scale), scale=scale)


@BOTH
@pytest.mark.parametrize("window,sink", [(0, 0), (60, 40)])
def test_prompts_over_blocks_that_are_not_there(eight, window, sink):
    # flagged; a key of a bad block counts as zeros, whatever the SMs held before
    s = Step([300, 200], [90, 200], 4, 2, 128, 16, window, sink, eight, seed=8)
    args = (i32(s.cu), i32(s.lens), 200, 300)

    def call(table, pool):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        a = (s.q, pool) + ((s.scales,) if eight else ()) + (i32(table),) + args
        f = pkv.paged_attention_varlen_fp8 if eight else pkv.paged_attention_varlen_window
        out, _ = f(*a, window=window, num_sink=sink, dev_status=st,
                   out=torch.empty(s.q.shape, device="cuda"))
        return out, st.item()

    table = s.table.copy()
    table[0, [0, 15]], table[1, 3] = s.nb, -1
    zeros = s.pool.clone()
    for blk in (s.table[0, 0], s.table[0, 15], s.table[1, 3]):
        zeros.view(torch.uint8 if eight else torch.int16)[:, int(blk)] = 0
    want, st = call(s.table, zeros)
    assert st == 0
    nan = torch.full_like(s.pool.float(), float("nan")).to(s.pool.dtype)
    for dirty in (s.pool, nan):
        call(s.table, dirty)
        got, st = call(table, s.pool)
        assert st == binding.DEV_BAD_BLOCK
        # (8 bits: a bad block has no scales, so that the weights' roundings differ: half a
        # step of fp16 in either call, of at most the largest value)
        most = max(np.abs(v).max() for v in s.v)
        assert torch.allclose(got, want, rtol=0, atol=(2.0 ** -10 + 2.0 ** -13) * most)
