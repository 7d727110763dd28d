"""Rotary cache write on the GPU: forms and values beside those of
test_gpu_budget, against the plain 64-bit form."""
import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv

from .test_gpu_budget import check_rope, f64, i32, rope_inputs, status_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h,hkv,d,rot", [
    (192, 8, 128, 20),     # 51 KB of heads: past the 48 KB that need no opt-in
    (760, 24, 128, 126),   # 196 KB, the most that fits
])
def test_rope_write_of_heads_that_fill_shared_memory(h, hkv, d, rot):
    q, k, v, pool, pos, slots = rope_inputs(5, h, hkv, d, rot, skip=[2])
    inv = pkv.rope_frequencies(rot, 10000.0)[0].cuda()
    pool0, st = pool.clone(), status_word()
    out = pkv.rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots), inv, dev_status=st)
    assert st.item() == 0
    check_rope(q, k, v, pool0, pos, slots, inv, 1.0, False, out, pool)


@pytest.mark.parametrize("inter,rot", [(False, 64), (False, 36), (True, 36), (True, 128)])
def test_rope_write_with_a_frequency_that_is_no_number(inter, rot):
    # m f is no number then, at position 0 too: the pair becomes NaN, and the
    # other pairs stay as they are
    q, k, v, pool, pos, slots = rope_inputs(9, 4, 2, 128, 21, packed=False)
    pos[0] = 0
    inv = pkv.rope_frequencies(rot)[0].cuda()
    clean = pool.clone()
    want = pkv.rope_kv_cache_write(q, clean, k, v, i32(pos), i32(slots), inv, interleaved=inter)
    bad = {1: float("inf"), 4: -float("inf"), rot // 2 - 1: float("nan")}
    for p, x in bad.items():
        inv[p] = x
    out = pkv.rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots), inv, interleaved=inter)
    dims = [x for p in bad for x in ((2 * p, 2 * p + 1) if inter else (p, p + rot // 2))]
    lost = torch.zeros(128, dtype=torch.bool, device="cuda")
    lost[dims] = True
    at = torch.from_numpy(slots).long().cuda()
    rows, clean_rows = pool.view(2, -1, 2, 128)[:, at], clean.view(2, -1, 2, 128)[:, at]
    assert torch.isnan(out[..., lost]).all() and torch.isnan(rows[0][..., lost]).all()
    assert torch.equal(out[..., ~lost], want[..., ~lost])
    assert torch.equal(rows[0][..., ~lost], clean_rows[0][..., ~lost])
    assert torch.equal(rows[1], clean_rows[1])
