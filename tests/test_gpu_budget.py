"""The rotary cache write and the cache-budget calls on the GPU, against plain
64-bit forms written from their definitions."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv
from paged_kv_cache_varlen_gb300 import binding

from . import plain_budget as plain
from .gpu_util import guarded, guards_intact

pytestmark = pytest.mark.gpu

BF16_HALF_STEP = 2.0 ** -8


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * std).to(torch.bfloat16)


# ----------------------------------------------------------------------- rope
def rope_inputs(t, h, hkv, d, seed, bs=16, packed=True, max_pos=4096, skip=()):
    r = np.random.RandomState(seed)
    qkv = normal((t, (h + 2 * hkv) * d), seed)
    q = qkv[:, :h * d].view(t, h, d)
    k = qkv[:, h * d:(h + hkv) * d].view(t, hkv, d)
    v = qkv[:, (h + hkv) * d:].view(t, hkv, d)
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = -(-t // bs) + 2
    slots = r.permutation(nb * bs)[:t]
    slots[list(skip)] = -1
    pos = r.randint(0, max_pos, t)
    return q, k, v, normal((2, nb, bs, hkv, d), seed + 1), pos, slots


def check_rope(q, k, v, pool0, pos, slots, inv_freq, factor, inter, got_q, got_pool):
    hkv, d = pool0.shape[3:]
    f = inv_freq.cpu().numpy()
    for x, got in ((q, got_q), (k, None)):
        want, mag = plain.rope(f64(x), pos, f, factor, inter)
        # one rounding to bf16; before it fp32 products of sines and cosines
        # whose angle is off by at most 2^-21 rad (its rounding to 24 bits of
        # at most half a turn, and the function's own few ulp)
        tol = BF16_HALF_STEP * np.abs(want) + 2.0 ** -20 * mag
        if got is None:
            rows = f64(got_pool[0].reshape(-1, hkv, d))
            got = rows[slots[slots >= 0]]
            want, tol = want[slots >= 0], tol[slots >= 0]
        else:
            got = f64(got)
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)
    # values are bit copies; every other slot is as it was
    flat = got_pool.view(torch.int16).view(2, -1, hkv, d)
    used = torch.from_numpy(slots[slots >= 0]).long().cuda()
    keep = torch.from_numpy(np.nonzero(slots >= 0)[0]).cuda()
    assert torch.equal(flat[1][used], v.contiguous().view(torch.int16)[keep])
    other = torch.ones(flat.shape[1], dtype=torch.bool, device="cuda")
    other[used] = False
    assert torch.equal(flat[:, other], pool0.view(torch.int16).view(2, -1, hkv, d)[:, other])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,h,hkv,d,rot", [
    (1, 32, 8, 128, 128), (7, 4, 2, 64, 64), (65, 32, 8, 128, 64), (33, 16, 2, 64, 48),
    (5, 12, 2, 128, 20), (9, 5, 5, 128, 126), (3, 1, 1, 64, 2), (17, 28, 4, 128, 40),
    (4, 71, 1, 64, 64), (6, 3, 3, 8, 8), (2, 2, 1, 24, 10), (300, 40, 8, 128, 128),
    (3, 2, 2, 512, 512),
])
def test_rope_write(t, h, hkv, d, rot, inter):
    q, k, v, pool, pos, slots = rope_inputs(t, h, hkv, d, t + rot, skip=[t // 2] if t > 3 else [])
    inv, factor = pkv.rope_frequencies(rot, 10000.0, scaling="ramp", stretch=4.0,
                                       original_len=1024) if rot > 2 else (
        torch.ones(1, dtype=torch.float64), 1.0)
    inv = inv.cuda()
    pool0, st = pool.clone(), status_word()
    out = pkv.rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots), inv, interleaved=inter,
                                  factor=factor, dev_status=st)
    check_rope(q, k, v, pool0, pos, slots, inv, factor, inter, out, pool)
    assert st.item() == 0


@pytest.mark.parametrize("rot", [128, 64, 36])
def test_rope_far_positions(rot):
    # the last positions an int32 holds: an angle formed in fp32 would be off
    # by many turns
    q, k, v, pool, _, slots = rope_inputs(6, 4, 2, 128, rot)
    pos = np.array([0, 1, 2 ** 20 + 1, 10 ** 9 + 7, 2 ** 31 - 2, 2 ** 31 - 1])
    inv = pkv.rope_frequencies(rot, 500000.0)[0].cuda()
    pool0 = pool.clone()
    out = pkv.rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots), inv)
    # the products of the 64-bit reference itself are off by up to 2^-53 of
    # 2^31 rad, far below the tolerance
    check_rope(q, k, v, pool0, pos, slots, inv, 1.0, False, out, pool)


@pytest.mark.parametrize("inter,rot", [(False, 128), (False, 60), (True, 60)])
def test_rope_in_place(inter, rot):
    q, k, v, pool, pos, slots = rope_inputs(19, 8, 2, 128, 5, packed=False)
    inv = pkv.rope_frequencies(rot)[0].cuda()
    pool2, q2 = pool.clone(), q.clone()
    want = pkv.rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots), inv, interleaved=inter)
    got = pkv.rope_kv_cache_write(q2, pool2, k, v, i32(pos), i32(slots), inv, interleaved=inter,
                                  q_out=q2)
    assert got is q2 and torch.equal(got, want) and torch.equal(pool, pool2)


def test_rope_passes_special_values_through():
    # infinities and NaN in dimensions that do not rotate stay where they are,
    # bit for bit, and do not reach the rotated ones
    for inter, rot in ((False, 64), (False, 36), (True, 36)):
        q, k, v, pool, pos, slots = rope_inputs(3, 4, 2, 128, 9, packed=False)
        for x in (q, k, v):
            x[:, :, rot] = float("nan")
            x[:, :, rot + 1] = float("inf")
        v[:, :, 0] = -float("inf")
        inv = pkv.rope_frequencies(rot)[0].cuda()
        out = pkv.rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots), inv, interleaved=inter)
        assert torch.equal(out.view(torch.int16)[:, :, rot:], q.view(torch.int16)[:, :, rot:])
        assert torch.isfinite(out[:, :, :rot]).all()
        rows = pool.view(2, -1, 2, 128)[:, torch.from_numpy(slots).long().cuda()]
        assert torch.isfinite(rows[0][..., :rot]).all()
        assert torch.equal(rows[1].view(torch.int16), v.view(torch.int16))


def test_rope_bad_positions_and_slots():
    q, k, v, pool, pos, slots = rope_inputs(6, 4, 2, 64, 3)
    inv = pkv.rope_frequencies(64)[0].cuda()
    bad_pos, bad_slots = pos.copy(), slots.copy()
    bad_pos[2] = -1
    bad_slots[4] = pool.shape[1] * pool.shape[2]
    bad_slots[5] = -7
    buf, out = guarded((6, 4, 64), torch.bfloat16)
    before, pool0, st = out.clone(), pool.clone(), status_word()
    pkv.rope_kv_cache_write(q, pool, k, v, i32(bad_pos), i32(bad_slots), inv, q_out=out,
                            dev_status=st)
    assert st.item() == binding.DEV_BAD_POSITION | binding.DEV_BAD_SLOT
    assert guards_intact(buf, out.numel())
    assert torch.equal(out[2].view(torch.int16), before[2].view(torch.int16))
    written = np.where(np.isin(np.arange(6), [2, 4, 5]), -1, slots)
    good = [0, 1, 3, 4, 5]
    check_rope(q[good], k[good], v[good], pool0, pos[good], written[good], inv, 1.0, False,
               out[good], pool)


def test_rope_binding_refusals():
    q, k, v, pool, pos, slots = rope_inputs(4, 4, 2, 64, 3)
    inv = pkv.rope_frequencies(64)[0].cuda()
    p, s = i32(pos), i32(slots)
    with pytest.raises(TypeError):
        pkv.rope_kv_cache_write(q.float(), pool, k, v, p, s, inv)
    with pytest.raises(TypeError):
        pkv.rope_kv_cache_write(q, pool, k, v, p, s, inv.float())
    with pytest.raises(ValueError):
        pkv.rope_kv_cache_write(q, pool, k[:3], v, p, s, inv)
    with pytest.raises(ValueError):
        pkv.rope_kv_cache_write(q, pool, k, v, p[:3], s, inv)
    with pytest.raises(ValueError):  # a token's heads are not contiguous
        pkv.rope_kv_cache_write(q.transpose(0, 1).contiguous().transpose(0, 1), pool, k, v, p, s,
                                inv)
    with pytest.raises(binding.PkvError):  # more rotated dimensions than the head has
        pkv.rope_kv_cache_write(q, pool, k, v, p, s, pkv.rope_frequencies(66)[0].cuda())
    with pytest.raises(binding.PkvError):  # in place needs a dense q
        pkv.rope_kv_cache_write(q, pool, k, v, p, s, inv, q_out=torch.as_strided(
            q, (4, 4, 64), (256, 64, 1)))


# ---------------------------------------------------------------- key weights
class Batch:
    """A ragged batch with its cached keys, and the log-sum-exp of its rows."""

    def __init__(self, lens, qlens, h, hkv, d, bs=16, seed=1, std=2.0, poison=True):
        r = np.random.RandomState(seed)
        self.lens, self.qlens = np.array(lens), np.array(qlens)
        self.h, self.hkv, self.d, self.bs = h, hkv, d, bs
        n = -(-self.lens // bs)
        ids = r.permutation(int(n.sum()) + 3)
        self.nb = len(ids)
        self.table = np.full((len(lens), max(1, int(n.max()))), -1)
        at = 0
        for i, m in enumerate(n):
            self.table[i, :m] = ids[at:at + m]
            at += m
        self.cu = np.concatenate([[0], np.cumsum(self.qlens)])
        self.pool = normal((2, self.nb, bs, hkv, d), seed + 1)
        if poison:  # slots past a context hold anything
            full = torch.ones(self.nb * bs, dtype=torch.bool)
            for i, L in enumerate(lens):
                p = np.arange(L)
                full[torch.from_numpy(self.table[i, p // bs] * bs + p % bs)] = False
            self.pool.view(2, -1, hkv, d)[:, full.cuda()] = float("nan")
        self.q = normal((int(self.cu[-1]), h, d), seed + 2, std)
        self.scale = 1.0 / math.sqrt(d)
        self.max_q, self.max_len = int(self.qlens.max()), int(self.lens.max())
        self.lse = self.reference_lse()

    def keys(self, i):
        p = np.arange(self.lens[i])
        slots = torch.from_numpy(self.table[i, p // self.bs] * self.bs + p % self.bs).cuda()
        return f64(self.pool[0].view(-1, self.hkv, self.d)[slots])

    def reference_lse(self):
        out = np.zeros((int(self.cu[-1]), self.h), dtype=np.float32)
        g = self.h // self.hkv
        for i, L in enumerate(self.lens):
            n = int(self.qlens[i])
            if n == 0:
                continue
            k, q = self.keys(i), f64(self.q[self.cu[i]:self.cu[i + 1]])
            hidden = np.arange(L)[None, :] > (L - n + np.arange(n))[:, None]
            for a in range(self.h):
                s = np.where(hidden, -np.inf, q[:, a] @ k[:, a // g].T * self.scale)
                m = s.max(1)
                out[self.cu[i]:self.cu[i + 1], a] = m + np.log(np.exp(s - m[:, None]).sum(1))
        return out

    def call(self, weights, out=None, rows=None, prior=None, decay=1.0, st=None, **kw):
        return pkv.attention_key_weights(
            self.q, self.pool, torch.from_numpy(self.lse).cuda(), i32(self.table), i32(self.cu),
            i32(self.lens), self.max_q, self.max_len, weights, out=out,
            weight_rows=None if rows is None else i32(rows),
            prior_lens=None if prior is None else i32(prior), decay=decay, scale=self.scale,
            dev_status=st, **kw)

    def expect(self, weights, out, rows=None, prior=None, decay=1.0):
        return plain.key_weights(weights, f64(self.q), self.keys, self.lse.astype(np.float64),
                                 self.cu, self.lens, rows or list(range(len(self.lens))), prior,
                                 decay, self.scale, out)


def check_weights(got, want, bound, old):
    got, old = f64(got), f64(old)
    assert np.all(np.isfinite(got) == np.isfinite(want))
    ok = np.isfinite(want)
    assert np.all(np.abs(got - want)[ok] <= bound[ok]), np.max((np.abs(got - want) - bound)[ok])
    untouched = bound == 0
    assert np.array_equal(got[untouched], old[untouched], equal_nan=True)


CASES = {
    "one key": ([1], [1], 4, 2, 128),
    "single tokens": ([1, 15, 16, 17, 130, 257], [1] * 6, 32, 8, 128),
    "single tokens, 64": ([1, 33, 500], [1, 1, 1], 16, 4, 64),
    "groups of 5": ([40, 129], [1, 1], 40, 8, 128),
    "groups of 7, short steps": ([90, 64, 31], [3, 4, 2], 28, 4, 128),
    "one head a group": ([77, 300], [1, 6], 8, 8, 64),
    "16 columns": ([200, 18], [4, 3], 32, 8, 128),
    "32 columns": ([200, 18, 1030], [8, 5, 7], 32, 8, 128),
    "a row past 32 heads": ([70, 5], [1, 1], 40, 1, 64),
    "no queries beside some": ([50, 20, 60], [0, 3, 0], 8, 2, 64),
    "whole prompts": ([1, 129, 300, 256], [1, 129, 300, 256], 32, 8, 128),
    "chunks": ([1000, 513, 700], [100, 257, 3], 32, 8, 128),
    "chunks, 64": ([600, 385, 130], [33, 385, 1], 16, 4, 64),
    "chunks, groups of 6": ([400, 300], [50, 90], 12, 2, 128),
    "chunks, groups of 7": ([260, 515], [37, 130], 28, 4, 64),
    "chunks, many heads a group": ([300, 50], [20, 9], 128, 1, 64),
    "a group of 256": ([70, 33], [5, 1], 256, 1, 64),
    "one head": ([520], [300], 1, 1, 128),
    "long context, short chunk": ([3000], [65], 8, 2, 128),
}


@pytest.mark.parametrize("bs", [16, 64, 256])
@pytest.mark.parametrize("name", CASES)
def test_key_weights(name, bs):
    lens, qlens, h, hkv, d = CASES[name]
    b = Batch(lens, qlens, h, hkv, d, bs=bs, seed=len(name))
    n = len(lens)
    rows = list(np.random.RandomState(3).permutation(n + 2)[:n])
    w = torch.rand((n + 2, hkv, max(lens) + 5), device="cuda")
    buf, out = guarded(tuple(w.shape), torch.float32)
    out.fill_(7.0)
    old, st = out.clone(), status_word()
    got = b.call(w, out=out, rows=rows, decay=0.75, st=st)
    assert got is out and st.item() == 0 and guards_intact(buf, out.numel())
    check_weights(got, *b.expect(f64(w), f64(old), rows, decay=0.75), old)


@pytest.mark.parametrize("qlens", [[1, 1, 1], [1, 40, 300]])
def test_key_weights_in_place_and_prior(qlens):
    lens = [300, 170, 301]
    b = Batch(lens, qlens, 32, 8, 128, seed=4)
    prior = [0, 100, 400]  # none kept, a part, more than there are keys
    w = torch.rand((3, 8, 301), device="cuda")
    old = w.clone()
    want = b.expect(f64(w), f64(w), prior=prior)
    got = b.call(w, prior=prior)
    assert got is w
    check_weights(w, *want, old)
    # a decay of zero drops what is there unread
    w2 = torch.full((3, 8, 301), float("nan"), device="cuda")
    zero = np.zeros((3, 8, 301))
    old, want = w2.clone(), b.expect(zero, f64(w2), decay=0.0)
    check_weights(b.call(w2, decay=0.0), *want, old)


def test_key_weights_sum_to_the_number_of_query_heads():
    b = Batch([700, 90], [90, 1], 32, 8, 128, seed=8)
    w = b.call(torch.zeros((2, 8, 700), device="cuda"))
    total = f64(w).sum((1, 2))
    # every row's softmax adds up to 1
    np.testing.assert_allclose(total, np.array([90, 1]) * 32, rtol=1e-5)


@pytest.mark.parametrize("qlens", [[1, 1], [50, 40]])
def test_key_weights_of_empty_rows_and_special_keys(qlens):
    b = Batch([60, 45], qlens, 8, 2, 128, seed=6)
    b.lse[0, :] = -np.inf        # a row without keys
    b.lse[b.cu[1], 3] = np.inf   # weights of zero
    p = 17
    slot = b.table[1, p // 16] * 16 + p % 16
    b.pool[0].view(-1, 2, 128)[slot, 1, :] = float("nan")  # one cached key is NaN
    w = torch.zeros((2, 2, 60), device="cuda")
    got = f64(b.call(w.clone()))
    with np.errstate(invalid="ignore"):
        want, bound = b.expect(f64(w), f64(w))
    # the NaN stays in its own key and head
    assert np.isnan(got[1, 1, p]) and np.isnan(want[1, 1, p])
    got[1, 1, p] = want[1, 1, p] = bound[1, 1, p] = 0
    assert np.all(np.abs(got - want) <= bound)


def test_key_weights_neighbours_with_nan_queries():
    # a NaN query of one request stays out of the others' sums
    b = Batch([90, 260, 150], [30, 37, 33], 32, 8, 128, seed=12)
    clean = b.call(torch.zeros((3, 8, 260), device="cuda"))
    b.q[b.cu[1]:b.cu[2]] = float("nan")
    st = status_word()
    got = b.call(torch.zeros((3, 8, 260), device="cuda"), st=st)
    assert st.item() == 0
    for i in (0, 2):
        assert torch.equal(got[i], clean[i])
    assert torch.isnan(got[1, :, :223]).all()


@pytest.mark.parametrize("qlens", [[1, 1, 1], [1, 40, 60]])
def test_key_weights_bad_entries(qlens):
    b = Batch([64, 100, 200], qlens, 8, 2, 64, seed=2)
    w = torch.rand((3, 2, 200), device="cuda")
    good = b.call(w.clone())
    # a block outside the pool: its page keeps the old entries
    b.table[2, 3] = b.nb
    out, st = torch.full_like(w, 5.0), status_word()
    b.call(w, out=out, st=st)
    assert st.item() == binding.DEV_BAD_BLOCK
    assert torch.equal(out[:2, :, :64], good[:2, :, :64])
    assert torch.equal(out[2, :, :48], good[2, :, :48])
    assert torch.equal(out[2, :, 64:200], good[2, :, 64:200])
    assert (out[2, :, 48:64] == 5.0).all()
    # rows outside the weights, lengths that do not fit: the request is skipped
    b = Batch([64, 100, 200], qlens, 8, 2, 64, seed=2)
    st = status_word()
    out = torch.full_like(w, 5.0)
    b.call(w, out=out, rows=[0, 3, 2], st=st)
    assert st.item() == binding.DEV_BAD_ROW and (out[1] == 5.0).all()
    b.lens[1] = 0
    st = status_word()
    out = torch.full_like(w, 5.0)
    b.call(w, out=out, st=st)
    assert st.item() == binding.DEV_BAD_LENGTHS and (out[1] == 5.0).all()
    assert torch.equal(out[2], good[2]) and torch.equal(out[0, :, :64], good[0, :, :64])


def test_key_weights_twice_the_same_bits():
    b = Batch([900, 400, 80], [300, 1, 33], 32, 8, 128, seed=5)
    w = torch.rand((3, 8, 900), device="cuda")
    a, c = torch.zeros_like(w), torch.zeros_like(w)
    b.call(w, out=a)
    b.call(w, out=c)
    assert torch.equal(a, c)


# ------------------------------------------------------------------- eviction
def weight_rows_of(kind, shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn(shape, device="cuda", generator=g)
    if kind == "tail":
        return w.mul_(2).exp_()
    if kind == "ties":
        return (w * 2).round().clamp(-2, 2)
    if kind == "zeros":
        return torch.zeros_like(w)
    if kind == "signed zeros":
        return torch.where(w > 0, 0.0, -0.0)
    assert kind == "special"
    w[w > 1.5] = float("nan")
    w[w < -1.5] = -float("inf")
    w[(w > 1.2) & (w < 1.4)] = float("inf")
    w[(w > 0) & (w < 0.1)] = -0.0
    return w


def check_select(w, lens, keep, rows, sink, recent, kept, out, old_kept, old_out):
    wn, kn = w.cpu().numpy(), kept.cpu().numpy()
    want_k, want_o = old_kept.cpu().numpy().copy(), None
    if out is not None:
        want_o = old_out.cpu().numpy().copy()
    for i, (L, n) in enumerate(zip(lens, keep)):
        for h in range(w.shape[1]):
            row = wn[rows[i], h, :L]
            ids = plain.select(row, n, sink, recent) if n else np.zeros(0, int)
            want_k[i, h, :n] = ids
            if out is not None:
                want_o[rows[i], h, :n] = row[ids]
    assert np.array_equal(kn, want_k)
    if out is not None:
        assert np.array_equal(out.cpu().numpy().view(np.int32), want_o.view(np.int32))


@pytest.mark.parametrize("kind", ["tail", "ties", "zeros", "signed zeros", "special"])
@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([1, 1, 5], [1, 0, 2], 0, 0),
    ([40, 33, 31, 64], [10, 33, 1, 63], 2, 3),
    ([700, 1000, 513], [100, 999, 512], 4, 64),
    ([2000, 9000], [5, 4000], 8, 3),            # budgets below and above the protected keys
    ([5000, 4097, 20], [300, 300, 20], 0, 400),
    ([300, 0, 7], [0, 0, 7], 1, 1),
])
def test_evict_select(kind, lens, keep, sink, recent):
    n, hkv = len(lens), 3
    rows = list(np.random.RandomState(2).permutation(n + 1)[:n])
    w = weight_rows_of(kind, (n + 1, hkv, max(lens) + 9), 3)
    kbuf, kept = guarded((n, hkv, max(keep) + 2), torch.int32)
    obuf, out = guarded(tuple(w.shape), torch.float32)
    old_kept, old_out, st = kept.clone(), out.clone(), status_word()
    pkv.evict_select(w, i32(lens), i32(keep), max(lens), max(keep) + 2, num_sink=sink,
                     num_recent=recent, weight_rows=i32(rows), kept=kept, weights_out=out,
                     dev_status=st)
    assert st.item() == 0
    assert guards_intact(kbuf, kept.numel()) and guards_intact(obuf, out.numel())
    check_select(w, lens, keep, rows, sink, recent, kept, out, old_kept, old_out)


@pytest.mark.parametrize("kind", ["tail", "zeros", "special"])
@pytest.mark.parametrize("L,keep", [(16384, 2000), (40001, 39000), (131072, 8192), (200003, 1)])
def test_evict_select_long_rows(kind, L, keep):
    w = weight_rows_of(kind, (1, 2, L), 5)
    kept, none = pkv.evict_select(w, i32([L]), i32([keep]), L, keep, num_sink=3, num_recent=50)
    assert none is None
    check_select(w, [L], [keep], [0], 3, 50, kept, None, torch.full_like(kept, -1), None)


@pytest.mark.parametrize("kind", ["tiny", "huge", "negative", "around 2^-40", "around 2^24"])
@pytest.mark.parametrize("L,keep", [(3001, 700), (600, 300), (150000, 60000)])
def test_evict_select_outside_the_first_bins(kind, L, keep):
    # the keep-th weight is below, above or at an end of the range that the first pass resolves
    w = weight_rows_of("tail", (1, 2, L), 7)
    if kind == "tiny":
        w = w * 1e-30
    elif kind == "huge":
        w = w * 1e30
    elif kind == "negative":
        w = -w
    else:
        edge = torch.full_like(w, 2.0 ** -40 if kind == "around 2^-40" else 2.0 ** 24)
        at = (w * 1000).to(torch.int32) % 5 - 2  # up to two neighbours to either side
        w = (edge.view(torch.int32) + at).view(torch.float32)
    kept, _ = pkv.evict_select(w, i32([L]), i32([keep]), L, keep, num_sink=2, num_recent=5)
    check_select(w, [L], [keep], [0], 2, 5, kept, None, torch.full_like(kept, -1), None)


@pytest.mark.parametrize("off", [0, 1])  # a row on a 16-byte boundary, or 4 bytes off it
@pytest.mark.parametrize("seqs,hkv,L,keep", [
    (19, 8, 4096, 512),     # a row for each SM
    (20, 8, 2052, 700),     # more rows than SMs: rows of one, two and three groups of keys
    (40, 8, 17000, 100),
    (20, 8, 45000, 20000),  # too long to stage
    (32, 8, 41000, 500),    # and more rows than clusters would help
    (70, 4, 1500, 300),     # short rows
    (170, 1, 200001, 5000),
    (2, 8, 100004, 8192),   # few rows: CTAs in clusters of different sizes
    (3, 8, 30000, 29999),
    (9, 4, 30000, 1),
    (5, 8, 9000, 4500),
    (2, 2, 8196, 1000),
])
def test_evict_select_rows_and_lengths(seqs, hkv, L, keep, off):
    flat = weight_rows_of("tail", (seqs * hkv * L + 4,), 9)
    w = flat[off:off + seqs * hkv * L].view(seqs, hkv, L)
    lens = [max(1, L - 37 * i * (L // 4000 + 1)) for i in range(seqs)]
    ns = [min(n, keep) for n in lens]
    out = torch.full((seqs, hkv, L), -7.0, device="cuda")
    old_out = out.clone()
    kept, _ = pkv.evict_select(w, i32(lens), i32(ns), L, keep, num_sink=4, num_recent=33,
                               weights_out=out)
    old_kept = torch.full_like(kept, -1)
    for i, n in enumerate(ns):
        old_kept[i, :, n:] = kept[i, :, n:]
    check_select(w, lens, ns, list(range(seqs)), 4, 33, kept, out, old_kept, old_out)


def test_evict_select_very_long_row():
    # longer than any on-chip copy of the row could be
    L, keep = 700001, 1234
    w = weight_rows_of("tail", (1, 1, L), 6)
    kept, _ = pkv.evict_select(w, i32([L]), i32([keep]), L, keep, num_sink=1, num_recent=9)
    check_select(w, [L], [keep], [0], 1, 9, kept, None, torch.full_like(kept, -1), None)


def test_evict_select_bad_entries():
    w = weight_rows_of("tail", (3, 2, 100), 1)
    for lens, keep, rows, bit in (([50, 101, 60], [5, 5, 5], [0, 1, 2], binding.DEV_BAD_LENGTHS),
                                  ([50, -1, 60], [5, 0, 5], [0, 1, 2], binding.DEV_BAD_LENGTHS),
                                  ([50, 40, 60], [5, 41, 5], [0, 1, 2], binding.DEV_BAD_LENGTHS),
                                  ([50, 40, 60], [5, -1, 5], [0, 1, 2], binding.DEV_BAD_LENGTHS),
                                  ([50, 90, 60], [5, 21, 5], [0, 1, 2], binding.DEV_BAD_LENGTHS),
                                  ([50, 40, 60], [5, 5, 5], [0, 3, 2], binding.DEV_BAD_ROW),
                                  ([50, 40, 60], [5, 5, 5], [0, -1, 2], binding.DEV_BAD_ROW)):
        st = status_word()
        kept, _ = pkv.evict_select(w, i32(lens), i32(keep), 100, 20, weight_rows=i32(rows),
                                   dev_status=st)
        assert st.item() == bit
        assert (kept[1] == -1).all()
        check_select(w, [50, 60], [5, 5], [0, 2], 0, 0, kept[[0, 2]], None,
                     torch.full((2, 2, 20), -1, dtype=torch.int32), None)


def compaction(lens, keep, hkv, d, bs, seed):
    r = np.random.RandomState(seed)
    n_src, n_dst = -(-np.array(lens) // bs), -(-np.array(keep) // bs)
    ids = r.permutation(int(n_src.sum() + n_dst.sum()) + 2)
    n = len(lens)
    src = np.full((n, max(1, n_src.max())), -1)
    dst = np.full((n, max(1, n_dst.max())), -1)
    at = 0
    for i in range(n):
        src[i, :n_src[i]] = ids[at:at + n_src[i]]
        at += n_src[i]
        dst[i, :n_dst[i]] = ids[at:at + n_dst[i]]
        at += n_dst[i]
    kept = np.full((n, hkv, max(1, max(keep))), 1 << 30)
    for i in range(n):
        for h in range(hkv):
            kept[i, h, :keep[i]] = np.sort(r.permutation(lens[i])[:keep[i]])
    return src, dst, kept, normal((2, len(ids), bs, hkv, d), seed)


def moved(pool, src, dst, kept, keep, bs):
    want = pool.clone()
    flat = want.view(2, -1, *pool.shape[3:])
    old = pool.view(2, -1, *pool.shape[3:])
    for i, n in enumerate(keep):
        j = np.arange(n)
        to = torch.from_numpy(dst[i, j // bs] * bs + j % bs).cuda()
        for h in range(pool.shape[3]):
            s = kept[i, h, :n]
            flat[:, to, h] = old[:, torch.from_numpy(src[i, s // bs] * bs + s % bs).cuda(), h]
    return want


@pytest.mark.parametrize("lens,keep,hkv,d,bs", [
    ([1], [1], 1, 64, 16), ([33, 64, 100], [10, 64, 1], 8, 128, 16),
    ([500, 7, 300], [450, 0, 33], 2, 64, 32), ([90, 91], [17, 18], 5, 128, 64),
    ([40, 41], [20, 39], 3, 8, 16), ([60, 30], [50, 30], 2, 512, 16), ([77], [50], 3, 24, 5),
    ([3000, 2000], [1500, 16], 8, 128, 256),
])
def test_evict_compact(lens, keep, hkv, d, bs):
    src, dst, kept, pool = compaction(lens, keep, hkv, d, bs, 4)
    want, st = moved(pool, src, dst, kept, keep, bs), status_word()
    pkv.evict_compact(pool, i32(src), i32(dst), i32(kept), i32(keep), dev_status=st)
    assert st.item() == 0
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))


def test_evict_compact_repeats_and_any_order():
    src, dst, kept, pool = compaction([64], [40], 2, 64, 16, 4)
    kept[0, :, :40] = np.random.RandomState(1).randint(0, 64, (2, 40))
    want = moved(pool, src, dst, kept, [40], 16)
    pkv.evict_compact(pool, i32(src), i32(dst), i32(kept), i32([40]))
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))


def test_evict_compact_bad_entries():
    lens, keep, bs = [100, 64, 90], [40, 30, 20], 16
    src, dst, kept, pool = compaction(lens, keep, 2, 64, bs, 4)
    cases = []
    k = kept.copy(); k[1, 0, 5] = -1; k[1, 1, 6] = src.shape[1] * bs
    cases.append((src, dst, k, keep, binding.DEV_BAD_KEPT, [(1, 0, 5), (1, 1, 6)]))
    d = dst.copy(); d[1, 1] = pool.shape[1]
    cases.append((src, d, kept, keep, binding.DEV_BAD_BLOCK,
                  [(1, h, j) for h in range(2) for j in range(16, 30)]))
    cases.append((src, dst, kept, [40, -1, 20], binding.DEV_BAD_LENGTHS,
                  [(1, h, j) for h in range(2) for j in range(30)]))
    cases.append((src, dst, kept, [40, 41, 20], binding.DEV_BAD_LENGTHS,
                  [(1, h, j) for h in range(2) for j in range(30)]))
    for s, d, k, n, bit, skipped in cases:
        want = moved(pool, src, dst, kept, keep, bs)
        for i, h, j in skipped:
            at = dst[i, j // bs]
            want[:, at, j % bs, h] = pool[:, at, j % bs, h]
        got, st = pool.clone(), status_word()
        pkv.evict_compact(got, i32(s), i32(d), i32(k), i32(n), dev_status=st)
        assert st.item() == bit
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


# ------------------------------------------------------ together, as it is used
def test_a_request_held_inside_its_budget(oracle):
    """Rotate and write, attend, accumulate, evict, and go on: the attention
    over the shortened contexts equals the plain one over the kept rows."""
    h, hkv, d, bs, budget = 8, 2, 64, 16, 48
    prompts = [70, 33, 120]
    bm = binding.BlockManager(64, bs)
    for i in range(3):
        bm.add_seq(i)
    inv, factor = pkv.rope_frequencies(d, 10000.0)
    inv = inv.cuda()
    pool = torch.zeros((2, 64, bs, hkv, d), dtype=torch.bfloat16, device="cuda")
    weights = torch.zeros((3, hkv, 256), device="cuda")
    spare = torch.zeros_like(weights)
    shadow = [[[] for _ in range(hkv)] for _ in range(3)]  # (K, V) rows per head
    total = [[np.zeros(0) for _ in range(hkv)] for _ in range(3)]
    position = [0, 0, 0]
    st = status_word()
    for step in range(5):
        new = prompts if step == 0 else [1, 2, 1]
        t = sum(new)
        table, lens, cu, slots, cs, cd = bm.build_step([0, 1, 2], new, 16)
        assert len(cs) == 0
        pos = np.concatenate([position[i] + np.arange(n) for i, n in enumerate(new)])
        qkv = normal((t, (h + 2 * hkv) * d), 100 + step)
        q = qkv[:, :h * d].view(t, h, d)
        k = qkv[:, h * d:(h + hkv) * d].view(t, hkv, d)
        v = qkv[:, (h + hkv) * d:].view(t, hkv, d)
        q2 = pkv.rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots), inv, dev_status=st)
        lse = torch.empty((t, h), device="cuda")
        out, _ = pkv.paged_attention_varlen(q2, pool, i32(table), i32(cu), i32(lens), max(new),
                                            int(lens.max()), out_lse=lse, dev_status=st)
        pkv.attention_key_weights(q2, pool, lse, i32(table), i32(cu), i32(lens), max(new),
                                  int(lens.max()), weights, dev_status=st)
        # the same with plain rows per head
        qr, _ = plain.rope(f64(q), pos, inv.cpu().numpy(), factor, False)
        kr, _ = plain.rope(f64(k), pos, inv.cpu().numpy(), factor, False)
        q_bits = f64(q2)
        rows = f64(pool[0].view(-1, hkv, d)[torch.from_numpy(slots).long().cuda()])
        assert np.max(np.abs(q_bits - qr)) < 0.05 and np.max(np.abs(rows - kr)) < 0.05
        for i, n in enumerate(new):
            for a in range(hkv):
                for j in range(n):
                    shadow[i][a].append((rows[cu[i] + j, a], f64(v[cu[i] + j, a])))
                total[i][a] = np.concatenate([total[i][a], np.zeros(n)])
            for a in range(h):
                kk = np.stack([x[0] for x in shadow[i][a // 4]])
                vv = np.stack([x[1] for x in shadow[i][a // 4]])
                s = q_bits[cu[i]:cu[i + 1], a] @ kk.T / math.sqrt(d)
                s[np.arange(len(kk))[None, :] > (len(kk) - n + np.arange(n))[:, None]] = -np.inf
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                assert np.max(np.abs(f64(out[cu[i]:cu[i + 1], a]) - p @ vv)) < 2e-3
                total[i][a // 4] += p.sum(0)
            position[i] += n
        w = f64(weights)
        for i in range(3):
            for a in range(hkv):
                # the lse is the attention kernel's (within 2e-3 of exact)
                np.testing.assert_allclose(w[i, a, :lens[i]], total[i][a], rtol=5e-3, atol=1e-6)
        if max(lens) > budget:
            keep = [min(int(n), budget) for n in lens]
            src, dst = bm.evict_step([0, 1, 2], keep, 16, 4)
            kept, _ = pkv.evict_select(weights, i32(lens), i32(keep), int(lens.max()), budget,
                                       num_sink=4, num_recent=8, weights_out=spare, dev_status=st)
            pkv.evict_compact(pool, i32(src), i32(dst), kept, i32(keep), dev_status=st)
            ids = kept.cpu().numpy()
            for i in range(3):
                for a in range(hkv):
                    got = ids[i, a, :keep[i]]
                    assert np.array_equal(got, plain.select(weights[i, a, :lens[i]].cpu().numpy(),
                                                            keep[i], 4, 8))
                    shadow[i][a] = [shadow[i][a][x] for x in got]
                    total[i][a] = total[i][a][got]
            weights, spare = spare, weights
    assert st.item() == 0
    assert position == [74, 41, 124]


def test_streams_and_graphs():
    """The calls run on the stream they are given and replay from a graph."""
    b = Batch([300, 90], [40, 1], 8, 2, 64, seed=3, poison=False)
    w0 = torch.rand((2, 2, 300), device="cuda")
    q, k, v, pool, pos, slots = rope_inputs(30, 8, 2, 64, 1)
    p, s, inv = i32(pos), i32(slots), pkv.rope_frequencies(64)[0].cuda()
    q_out = torch.empty((30, 8, 64), dtype=torch.bfloat16, device="cuda")
    lens, keep = i32([300, 90]), i32([100, 50])
    lse, table, cu = torch.from_numpy(b.lse).cuda(), i32(b.table), i32(b.cu)
    src, dst, kept_in, mpool = compaction([300, 90], [100, 50], 2, 64, 16, 5)
    src, dst = i32(src), i32(dst)

    def step(out, kept, sel, pools, stream=None):
        pkv.rope_kv_cache_write(q, pools[0], k, v, p, s, inv, q_out=q_out, stream=stream)
        pkv.attention_key_weights(b.q, b.pool, lse, table, cu, lens, 40, 300, w0, out=out,
                                  scale=b.scale, stream=stream)
        pkv.evict_select(out, lens, keep, 300, 100, num_sink=2, num_recent=5, kept=kept,
                         weights_out=sel, stream=stream)
        pkv.evict_compact(pools[1], src, dst, kept, keep, stream=stream)

    def buffers():
        return (torch.zeros_like(w0), torch.full((2, 2, 100), -1, dtype=torch.int32,
                                                 device="cuda"),
                torch.zeros_like(w0), (pool.clone(), mpool.clone()))

    want = buffers()
    step(*want)
    other = buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(*other, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    captured = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*captured)
    for x in (captured[0], captured[1], captured[2]):
        x.zero_()
    captured[1].fill_(-1)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for got in (other, captured):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(got[2], want[2])
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16))
                   for x, y in zip(got[3], want[3]))


def test_offsets_past_32_bits():
    """Slots whose byte and element offsets pass 2^31 and 2^32."""
    hkv, d, bs = 8, 128, 16
    nb = (1 << 32) // (bs * hkv * d) + 64   # K half alone has over 2^32 elements
    if torch.cuda.mem_get_info()[0] < 5 * nb * bs * hkv * d:
        pytest.skip("not enough free memory")
    pool = torch.zeros((2, nb, bs, hkv, d), dtype=torch.bfloat16, device="cuda")
    q = normal((2, 32, d), 1)
    k, v = normal((2, hkv, d), 2), normal((2, hkv, d), 3)
    slots = [nb * bs - 1, nb * bs - 2]
    inv = pkv.rope_frequencies(d)[0].cuda()
    st = status_word()
    pkv.rope_kv_cache_write(q, pool, k, v, i32([0, 0]), i32(slots), inv, dev_status=st)
    assert torch.equal(pool[0, nb - 1, 15], k[0]) and torch.equal(pool[1, nb - 1, 14], v[1])
    src, dst = i32([[nb - 1]]), i32([[nb - 2]])
    kept = i32(np.full((1, hkv, 2), 14) + np.arange(2))
    pkv.evict_compact(pool, src, dst, kept, i32([2]), dev_status=st)
    assert torch.equal(pool[0, nb - 2, 0], k[1]) and torch.equal(pool[1, nb - 2, 1], v[0])
    w = torch.zeros((1, hkv, 2), device="cuda")
    lse = torch.zeros((1, 32), device="cuda")
    pkv.attention_key_weights(q[:1], pool, lse, dst, i32([0, 1]), i32([2]), 1, 2, w, scale=0.01,
                              dev_status=st)
    want = np.exp(f64(q[0]).reshape(hkv, 4, d) @ np.stack([f64(k[1]), f64(k[0])], -1) * 0.01).sum(1)
    # 4 terms of about 1, each within a few fp32 steps
    np.testing.assert_allclose(f64(w[0]), want, rtol=2.0 ** -19)
    assert st.item() == 0


# ------------------------------------------ bounds far above what is there, and
# more work than CTAs
@pytest.mark.parametrize("qlens,name", [
    ([1] * 9, "single tokens"), ([1, 40, 300, 2, 90, 64, 1, 33, 257], "a mixed batch"),
    ([60, 40, 300, 33, 90, 64, 70, 34, 257], "chunks"),
])
def test_key_weights_under_a_loose_bound(qlens, name):
    # max_seq_len only bounds the lengths: a million of them changes how the
    # work is handed out, not a bit of the result
    lens = [max(x) for x in zip([1, 700, 1300, 257, 90, 64, 2049, 333, 512], qlens)]
    b = Batch(lens, qlens, 8, 2, 128, seed=21, poison=False)
    tight = b.call(torch.zeros((9, 2, 2049), device="cuda"))
    w = torch.full((9, 2, 1 << 20), 3.0, device="cuda")
    b.max_len = 1 << 20
    st = status_word()
    got = b.call(w, prior=[0] * 9, st=st)
    assert st.item() == 0
    for i, L in enumerate(lens):
        assert torch.equal(got[i, :, :L], tight[i, :, :L])
        assert (got[i, :, L:] == 3.0).all()


def test_key_weights_of_many_requests_under_a_loose_bound():
    # more requests than a CTA lists
    n = 300
    r = np.random.RandomState(5)
    qlens = r.randint(30, 50, n)
    lens = qlens + r.randint(0, 200, n)
    b = Batch(list(lens), list(qlens), 4, 2, 64, seed=22, poison=False)
    tight = b.call(torch.zeros((n, 2, int(lens.max())), device="cuda"))
    b.max_len = 20000
    got = b.call(torch.zeros((n, 2, 20000), device="cuda"), prior=[0] * n)
    assert torch.equal(got[:, :, :int(lens.max())], tight)
    assert (got[:, :, int(lens.max()):] == 0).all()


def test_evict_select_under_a_loose_bound():
    w = weight_rows_of("special", (3, 2, 150000), 8)
    lens, keep = [700, 90, 3000], [100, 90, 1]
    kept, _ = pkv.evict_select(w, i32(lens), i32(keep), 150000, 120, num_sink=2, num_recent=9)
    check_select(w, lens, keep, [0, 1, 2], 2, 9, kept, None, torch.full_like(kept, -1), None)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_of_more_tokens_than_resident_warps(inter):
    t = 10007
    q, k, v, pool, pos, slots = rope_inputs(t, 3, 1, 64, 77, max_pos=1 << 20)
    inv = pkv.rope_frequencies(64, 500000.0)[0].cuda()
    pool0 = pool.clone()
    out = pkv.rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots), inv, interleaved=inter)
    check_rope(q, k, v, pool0, pos, slots, inv, 1.0, inter, out, pool)


def test_two_streams_at_once():
    # no call keeps anything that another one on another stream could share
    batches = [Batch([900, 70], [300, 1], 8, 2, 64, seed=s, poison=False) for s in (31, 32)]
    want = [b.call(torch.zeros((2, 2, 900), device="cuda")) for b in batches]
    sel = [pkv.evict_select(w, i32([900, 70]), i32([200, 10]), 900, 200)[0] for w in want]
    streams = [torch.cuda.Stream() for _ in batches]
    outs = [torch.zeros((2, 2, 900), device="cuda") for _ in batches]
    kept = [torch.full((2, 2, 200), -1, dtype=torch.int32, device="cuda") for _ in batches]
    lens, keep = i32([900, 70]), i32([200, 10])
    torch.cuda.synchronize()
    for _ in range(20):
        for b, s, o, kk in zip(batches, streams, outs, kept):
            b.call(o, decay=0.0, stream=s)
            pkv.evict_select(o, lens, keep, 900, 200, kept=kk, stream=s)
    torch.cuda.synchronize()
    for w, o, s, kk in zip(want, outs, sel, kept):
        assert torch.equal(w, o) and torch.equal(s, kk)


def test_budget_binding_refusals():
    b = Batch([40, 20], [1, 1], 8, 2, 64, seed=3)
    w = torch.zeros((2, 2, 40), device="cuda")
    with pytest.raises(TypeError):
        b.call(w.double())
    with pytest.raises(ValueError):
        b.call(w[:, :, ::2])                       # not contiguous
    with pytest.raises(ValueError):
        b.call(torch.zeros((2, 3, 40), device="cuda"))
    with pytest.raises(ValueError):
        b.call(w, out=torch.zeros((3, 2, 40), device="cuda"))
    with pytest.raises(ValueError):
        b.call(w, rows=[0, 1, 2])
    with pytest.raises(ValueError):
        b.call(w.cpu())
    with pytest.raises(binding.PkvError) as e:     # rows shorter than the contexts
        b.call(torch.zeros((2, 2, 39), device="cuda"))
    assert e.value.status == 1
    lens, keep = i32([40, 20]), i32([5, 5])
    with pytest.raises(ValueError):
        pkv.evict_select(w, lens, keep[:1], 40, 5)
    with pytest.raises(ValueError):
        pkv.evict_select(w, lens, keep, 40, 5, kept=torch.zeros((2, 2, 6), dtype=torch.int32,
                                                                device="cuda"))
    with pytest.raises(TypeError):
        pkv.evict_select(w, lens.long(), keep, 40, 5)
    with pytest.raises(binding.PkvError):          # the weights would overwrite their source
        pkv.evict_select(w, lens, keep, 40, 5, weights_out=w)
    src, dst, kept, pool = compaction([40, 20], [5, 5], 2, 64, 16, 1)
    with pytest.raises(ValueError):
        pkv.evict_compact(pool, i32(src), i32(dst), i32(kept[:, :1]), keep)
    with pytest.raises(ValueError):
        pkv.evict_compact(pool, i32(src[:1]), i32(dst), i32(kept), keep)
    with pytest.raises(TypeError):
        pkv.evict_compact(pool.float(), i32(src), i32(dst), i32(kept), keep)


def test_debug_checks_name_the_bad_entry_of_budget_calls(monkeypatch):
    monkeypatch.setenv("PKV_DEBUG_CHECKS", "1")
    b = Batch([40, 20], [1, 1], 8, 2, 64, seed=3)
    w = torch.zeros((2, 2, 40), device="cuda")
    with pytest.raises(ValueError, match="weight_rows"):
        b.call(w, rows=[1, 1])
    with pytest.raises(ValueError, match="keep_len"):
        pkv.evict_select(w, i32([40, 20]), i32([5, 21]), 40, 30)
    src, dst, kept, pool = compaction([40, 20], [5, 5], 2, 64, 16, 1)
    dst[1, 0] = src[0, kept[0, 0, 0] // 16]
    with pytest.raises(ValueError, match="both a source and a destination"):
        pkv.evict_compact(pool, i32(src), i32(dst), i32(kept), i32([5, 5]))
    q, k, v, pool, pos, slots = rope_inputs(3, 4, 2, 64, 3)
    pos[1] = -4
    with pytest.raises(ValueError, match="positions"):
        pkv.rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots),
                                pkv.rope_frequencies(64)[0].cuda())


def test_a_pool_without_its_v_half_is_refused():
    q, k, v, pool, pos, slots = rope_inputs(3, 4, 2, 64, 3)
    inv = pkv.rope_frequencies(64)[0].cuda()
    with pytest.raises(ValueError, match="kv_pool"):
        pkv.rope_kv_cache_write(q, pool[:1], k, v, i32(pos), i32(slots), inv)
    b = Batch([40, 20], [1, 1], 4, 2, 64, seed=3)
    b.pool = b.pool[:1]
    with pytest.raises(ValueError, match="kv_pool"):
        b.call(torch.zeros((2, 2, 40), device="cuda"))
    src, dst, kept, mpool = compaction([40, 20], [5, 5], 2, 64, 16, 1)
    with pytest.raises(ValueError, match="kv_pool"):
        pkv.evict_compact(mpool[:1], i32(src), i32(dst), i32(kept), i32([5, 5]))


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured (nothing has been set up by an
    eager one) replays the right results."""
    code = """
import torch, paged_kv_cache_varlen_gb300 as pkv
w = torch.rand((2, 2, 50000), device="cuda")
lens = torch.tensor([50000, 20000], dtype=torch.int32, device="cuda")
keep = torch.tensor([700, 300], dtype=torch.int32, device="cuda")
kept = torch.full((2, 2, 700), -1, dtype=torch.int32, device="cuda")
q = torch.randn((70, 8, 128), device="cuda").bfloat16()
k = torch.randn((70, 2, 128), device="cuda").bfloat16()
pool = torch.zeros((2, 8, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
ids = torch.arange(70, dtype=torch.int32, device="cuda")
inv = pkv.rope_frequencies(128)[0].cuda()
q_out = torch.zeros_like(q)
table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
n = torch.tensor([70], dtype=torch.int32, device="cuda")
lse = torch.full((70, 8), 4.0, device="cuda")
sums = torch.zeros((1, 2, 128), device="cuda")
def step():
    pkv.rope_kv_cache_write(q, pool, k, k, ids, ids, inv, q_out=q_out)
    pkv.attention_key_weights(q_out, pool, lse, table, cu, n, 70, 70, sums)
    pkv.evict_select(w, lens, keep, 50000, 700, num_recent=9, kept=kept)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in (q_out, pool, sums, kept)]
for x in (q_out, pool, sums):
    x.zero_()
kept.fill_(-1)
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (q_out, pool, sums, kept)))
assert int(kept[0, 0, 699]) == 49999 and float(sums.sum()) > 0
print("the same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("n", [1, 2])
def test_key_weights_far_before_the_queries(n):
    """A key 70 million places before its queries, times 32 heads, passes 32 bits."""
    L, G, d, bs, nb = 70_000_000, 32, 64, 256, 4
    q = normal((n, G, d), 1)
    pool = normal((2, nb, bs, 1, d), 2)
    blocks = (L + bs - 1) // bs
    table = torch.arange(blocks, dtype=torch.int32, device="cuda") % nb  # the same pages again
    lse = torch.full((n, G), 1.0, device="cuda")
    w = torch.zeros((1, 1, L), device="cuda")
    st = status_word()
    pkv.attention_key_weights(q, pool, lse, table[None], i32([0, n]), i32([L]), n, L, w,
                              dev_status=st)
    assert st.item() == 0
    s = f64(pool[0, :, :, 0]).reshape(-1, d) @ f64(q).reshape(n * G, d).T / math.sqrt(d)
    p = np.exp(s - 1.0)
    page = torch.from_numpy(p.sum(1)).cuda()
    want = page.repeat((L + nb * bs - 1) // (nb * bs))[:L]
    want[L - 1] = p[(L - 1) % (nb * bs), (n - 1) * G:].sum()     # the last key: the last query alone
    # sums of n * 32 weights, scores of 64 products in fp32: far inside 1e-4
    assert float(((w[0, 0].double() - want).abs() / want).max()) < 1e-4
