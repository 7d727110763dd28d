"""Rotary cache write on the GPU: forms and values beside those of
test_gpu_budget, against the plain 64-bit form."""
import pytest

import paged_kv_cache_varlen_gb300 as pkv

from .test_gpu_budget import check_rope, i32, rope_inputs, status_word

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
