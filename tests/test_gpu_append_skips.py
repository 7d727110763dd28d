"""Tokens of bad positions in writes into the 8-bit cache: left out, values, scale and
q_out alike; the rows of a block that are there are rescaled, and only these."""
import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv
from paged_kv_cache_varlen_gb300 import binding

from . import plain_cache8 as plain
from .test_gpu_norm_write import f64, i32, normal, pool8, status_word, step, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,ql,bad", [
    # the first new token of a fresh block; one behind rows that are there; the last;
    # a whole block's; single tokens
    ([20], [4], [0]), ([27], [4], [1]), ([27], [4], [3]), ([40], [30], [6, 7, 20]),
    ([16], [16], list(range(16))), ([20, 5, 17, 33], [1, 1, 1, 1], [0, 2]),
])
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_of_bad_positions_are_left_out(lens, ql, bad, d):
    h, hkv, bs = 4, 2, 16
    table, cu, nb = step(lens, ql, bs, 5)
    t = int(cu[-1])
    q, k, v = normal((t, h, d), 1), normal((t, hkv, d), 2, 30.0), normal((t, hkv, d), 3, 30.0)
    k[bad], v[bad] = 1e30, -1e30  # (no scale takes these up)
    pool, scales = pool8(nb, bs, hkv, d, 7)
    before, sb = values(pool), f64(scales)
    pos = np.arange(t)
    pos[bad] = -1
    st, out = status_word(), torch.full((t, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.qk_norm_rope_kv_cache_append_fp8(q, pool, scales, k, v, i32(pos), i32(table), i32(cu),
                                         i32(lens), max(ql), None, q_out=out, dev_status=st)
    assert st.item() == binding.DEV_BAD_POSITION
    # as if the skipped tokens were zeros, but that their rows stay as they were
    kz, vz = f64(k), f64(v)
    kz[bad], vz[bad] = 0, 0
    want, ws, raw = plain.append(before, sb, kz, vz, table, cu, lens)
    for i in range(len(lens)):
        for j in range(ql[i]):
            if cu[i] + j in bad:
                at = lens[i] - ql[i] + j
                blk, row = table[i, at // bs], at % bs
                want[:, blk, row] = before[:, blk, row]
    assert np.array_equal(f64(scales), ws)
    assert np.array_equal(values(pool), want)
    assert not np.array_equal(ws, sb)
    good = np.setdiff1d(np.arange(t), bad)
    assert torch.all(out[bad] == 7.0) and torch.equal(out[good], q[good])
