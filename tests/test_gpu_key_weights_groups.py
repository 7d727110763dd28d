"""Key weights of groups of more than 128 heads on the GPU: the sum over very
many columns is held to a bound that does not grow with their number."""
import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv

from .test_gpu_budget import Batch, check_weights, f64, i32, normal, status_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,n", [(256, 2000), (130, 3001)])
def test_key_weights_of_a_wide_group_over_many_queries(heads, n):
    d, bs = 64, 16
    blocks = -(-n // bs)
    q = torch.zeros((n, heads, d), dtype=torch.bfloat16, device="cuda")  # every score is 0
    pool = normal((2, blocks, bs, 1, d), 2)
    lse = torch.full((n, heads), np.float32(-np.log(1.0013)), device="cuda")
    w, st = torch.zeros((1, 1, n), device="cuda"), status_word()
    pkv.attention_key_weights(q, pool, lse, i32(np.arange(blocks))[None], i32([0, n]), i32([n]),
                              n, n, w, dev_status=st)
    assert st.item() == 0
    want = np.exp(-float(lse[0, 0])) * heads * (n - np.arange(n))
    # Equal addends round to the same side for a whole octave of the sum, so a
    # chain of c additions may be off by c 2^-24, and no long one may be there:
    # chains of 256 and of one addition for every 1024 columns (at most 500),
    # and 4 to join the lanes; the exponent's roundings and ex2 add 2^-21.
    tol = (256 + 500 + 4) * 2.0 ** -24 + 2.0 ** -21
    err = np.abs(f64(w[0, 0]) - want) / want
    assert err.max() <= tol, err.max()


def test_key_weights_of_a_wide_group_whose_sums_are_folded():
    # a few thousand columns of ordinary scores, on both sides of a fold, the
    # first keys seen by all of them and the last by a few
    b = Batch([150, 64, 9], [20, 9, 4], 256, 1, 128, seed=3)
    w = torch.rand((3, 1, 150), device="cuda")
    old, st = w.clone(), status_word()
    got = b.call(w, decay=0.5, st=st)
    assert st.item() == 0
    check_weights(got, *b.expect(f64(old), f64(old), decay=0.5), old)
