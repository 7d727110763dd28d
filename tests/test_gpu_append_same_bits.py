"""What a token leaves in the 8-bit cache does not depend on the rest of its step: single
tokens by rows (max_query_len 1) and by blocks (a larger bound) are the same bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv

from .test_gpu_norm_write import frequencies, heads, i32, pool8, status_word, step, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter,rot", [(False, 128), (False, 64), (True, 128), (True, 50),
                                       (False, 60), (False, 0)])
@pytest.mark.parametrize("h,hkv,n", [(1, 8, 20000), (6, 3, 300)])
@pytest.mark.parametrize("wide", [False, True])
def test_single_tokens_by_rows_and_by_blocks(h, hkv, n, inter, rot, wide):
    d, bs = 64 if rot == 64 else 128, 32 if wide else 16
    r = np.random.RandomState(n + rot)
    lens = r.randint(1, 40, n)
    table, cu, nb = step(lens.tolist(), [1] * n, bs, 1)
    q, k, v = heads(n, h, hkv, d, rot, std=2.0)
    qw, kw = weights(d, 3, torch.float32 if wide else torch.bfloat16)
    pool, scales = pool8(nb, bs, hkv, d, 4)
    pos = i32(r.randint(0, 1 << 17, n))
    got = []
    for bound in (1, 2):
        p, s, st = pool.clone(), scales.clone(), status_word()
        out = pkv.qk_norm_rope_kv_cache_append_fp8(
            q, p, s, k, v, pos, i32(table), i32(cu), i32(lens), bound, frequencies(rot), qw, kw,
            eps=1e-5, weight_offset=0.5, interleaved=inter, factor=1.1, dev_status=st)
        assert st.item() == 0
        got.append((p.view(torch.uint8), s, out))
    for name, a, b in zip(("pool", "scales", "q_out"), *got):
        assert torch.equal(a, b), (name, int((a != b).sum()))
