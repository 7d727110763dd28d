"""Key weights of prompts on the GPU: the launch shapes that test_gpu_budget's
short cases do not reach (clusters of 2 and 4 CTAs an item, CTAs of more than
16 Q tiles, whose sums are folded on the way), against the plain 64-bit form.

On 152 SMs an item's Q tiles (128 // group queries each) are split over 2 CTAs
from 16 tiles on, over 4 from 32 on, while items * CTAs stay below 304."""
import numpy as np
import pytest
import torch

from paged_kv_cache_varlen_gb300 import binding

from .gpu_util import guarded, guards_intact
from .test_gpu_budget import Batch, check_weights, f64, status_word

pytestmark = pytest.mark.gpu

CASES = {
    # clusters of 4, 17 Q tiles a CTA; the last keys have one Q tile: three CTAs
    # of their cluster have none
    "four CTAs": ([1034], [1034], 8, 1, 128),
    "four CTAs, 64": ([1034], [1034], 8, 1, 64),
    "four CTAs, whole heads": ([1100], [1100], 8, 2, 128),
    "four CTAs, a query a tile": ([40, 300], [40, 39], 128, 1, 128),
    "four CTAs, groups of 7": ([900, 70], [600, 1], 7, 1, 128),
    "four CTAs, single tokens between": ([700, 1100, 90, 1300], [1, 1001, 2, 1050], 4, 1, 128),
    # clusters of 2
    "two CTAs": ([700, 520], [520, 1], 8, 2, 128),
    "two CTAs, 64": ([700, 520], [520, 1], 8, 2, 64),
    "two CTAs, one head a group": ([2300], [2100], 2, 2, 64),
    "two CTAs, more tiles": ([257, 400], [257, 300], 12, 1, 128),
    # a CTA an item, 17 Q tiles each
    "one CTA": ([19456], [136], 64, 4, 64),
}


@pytest.mark.parametrize("name", CASES)
def test_key_weights_of_prompts(name):
    lens, qlens, h, hkv, d = CASES[name]
    b = Batch(lens, qlens, h, hkv, d, seed=len(name))
    n = len(lens)
    w = torch.rand((n, hkv, max(lens) + 3), device="cuda")
    buf, out = guarded(tuple(w.shape), torch.float32)
    out.fill_(7.0)
    old, st = out.clone(), status_word()
    b.call(w, out=out, decay=0.5, st=st)
    assert st.item() == 0 and guards_intact(buf, out.numel())
    check_weights(out, *b.expect(f64(w), f64(old), decay=0.5), old)


@pytest.mark.parametrize("d", [64, 128])
def test_key_weights_of_a_listed_prompt(d):
    # a loose bound: each CTA goes through listed items of up to 65 Q tiles
    b = Batch([1034, 50, 700], [1034, 1, 300], 8, 1, d, seed=11)
    b.max_len = 1 << 20
    w = torch.full((3, 1, 1 << 20), 3.0, device="cuda")
    old, st = w.clone(), status_word()
    got = b.call(w, prior=[0, 0, 0], st=st)
    assert st.item() == 0
    check_weights(got, *b.expect(f64(old), f64(old), prior=[0, 0, 0]), old)


@pytest.mark.parametrize("d", [64, 128])
def test_key_weights_of_a_bad_page_in_a_cluster(d):
    b = Batch([1034], [1034], 8, 1, d, seed=13)
    w = torch.rand((1, 1, 1034), device="cuda")
    good = b.call(w.clone())
    b.table[0, 20] = -1
    b.table[0, 64] = b.nb       # the last page, of a cluster with idle CTAs
    out, st = torch.full_like(w, 5.0), status_word()
    b.call(w, out=out, st=st)
    assert st.item() == binding.DEV_BAD_BLOCK
    lost = np.zeros(1034, dtype=bool)
    lost[320:336] = lost[1024:] = True
    lost = torch.from_numpy(lost).cuda()
    assert (out[:, :, lost] == 5.0).all()
    assert torch.equal(out[:, :, ~lost], good[:, :, ~lost])


def test_key_weights_of_prompts_twice_the_same_bits():
    b = Batch([1300, 900], [1300, 700], 8, 1, 128, seed=14)
    w = torch.rand((2, 1, 1300), device="cuda")
    a, c = torch.zeros_like(w), torch.zeros_like(w)
    b.call(w, out=a)
    b.call(w, out=c)
    assert torch.equal(a, c)
