"""Attention through a window and over the 8-bit cache: padded batches, blocks that are
not there, scales whose products leave the fp32 range."""
import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv

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
