"""Attention through a window and over the 8-bit cache on the GPU, against a
plain 64-bit form written from the definition."""
import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv
from paged_kv_cache_varlen_gb300 import binding

from . import plain_cache8 as plain
from .gpu_util import guarded, guards_intact

pytestmark = pytest.mark.gpu

BF16_HALF_STEP = 2.0 ** -8
FP16_HALF_STEP = 2.0 ** -11


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


class Step:
    """A step's inputs. Every slot that no query may see holds NaN (behind the
    contexts, in hidden blocks that were given back, in blocks of nobody), and
    hidden blocks' table entries are bad ids."""

    def __init__(self, lens, ql, h, hkv, d, bs, window, sink, eight, seed, std=2.0, spread=0.3,
                 empty_entry=-1):
        r = np.random.RandomState(seed)
        self.lens, self.ql, self.window, self.sink, self.eight = lens, ql, window, sink, eight
        self.h, self.hkv, self.d, self.bs = h, hkv, d, bs
        self.cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
        t = int(self.cu[-1])
        self.q = torch.from_numpy(r.standard_normal((t, h, d)).astype(np.float32) * std).to(
            torch.bfloat16)
        blocks = [-(-L // bs) for L in lens]
        nb = sum(blocks) + 3
        ids = r.permutation(nb)
        self.table = np.full((len(lens), max(blocks + [1])), empty_entry, np.int32)
        rows = r.standard_normal((2, sum(lens), hkv, d)).astype(np.float32)
        if eight:
            rows = torch.from_numpy(np.clip(rows * 96, -448, 448)).to(torch.float8_e4m3fn)
            pool = torch.full((2, nb, bs, hkv, d), float("nan")).to(torch.float8_e4m3fn)
            s = np.exp(r.standard_normal((2, nb, hkv)) * spread) / 96
            self.scales = torch.from_numpy(s.astype(np.float32))
            # blocks that are not read have scales of anything
            bad = np.full((2, nb, hkv), np.nan, np.float32)
        else:
            rows = torch.from_numpy(rows).to(torch.bfloat16)
            pool = torch.full((2, nb, bs, hkv, d), float("nan"), dtype=torch.bfloat16)
        raw = pool.view(torch.uint8 if eight else torch.int16)
        flat = rows.view(torch.uint8 if eight else torch.int16)
        self.k, self.v = [], []
        at = start = 0
        for i, L in enumerate(lens):
            seen = np.ones(L, bool)
            if window and ql[i]:
                j = np.arange(L)
                seen = (j < sink) | (j > L - ql[i] - window)
            values = rows[:, start:start + L].float().numpy().astype(np.float64)
            for b in range(blocks[i]):
                here = seen[b * bs:(b + 1) * bs]
                if not here.any():
                    continue
                blk = ids[at + b]
                self.table[i, b] = blk
                n = np.nonzero(here)[0]
                raw[:, blk, n] = flat[:, start + b * bs + n]
                if eight:
                    bad[:, blk] = self.scales[:, blk].numpy()
                    values[:, b * bs:(b + 1) * bs] *= bad[:, blk].astype(np.float64)[:, None, :, None]
            self.k.append(values[0])
            self.v.append(values[1])
            at += blocks[i]
            start += L
        if eight:
            self.scales = torch.from_numpy(bad).cuda()
        self.q, self.pool = self.q.cuda(), pool.cuda()
        self.nb = nb

    def call(self, **kw):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw.setdefault("dev_status", st)
        t = self.q.shape[0]
        kw.setdefault("out_lse", torch.full((t, self.h), 7.0, device="cuda"))
        kw.setdefault("out", torch.full((t, self.h, self.d), 7.0, dtype=torch.bfloat16,
                                        device="cuda"))
        args = (i32(self.table), i32(self.cu), i32(self.lens), max(max(self.ql), 1),
                max(max(self.lens), 1))
        if self.eight:
            r = pkv.paged_attention_varlen_fp8(self.q, self.pool, self.scales, *args,
                                               window=self.window, num_sink=self.sink, **kw)
        else:
            r = pkv.paged_attention_varlen_window(self.q, self.pool, *args, self.window,
                                                  num_sink=self.sink, **kw)
        assert st.item() == 0
        return r

    def check(self, out, lse, scale=None):
        d = self.d
        scale = d ** -0.5 if scale is None else scale
        q = f64(self.q)
        want, wl, mag = plain.attention(q, lambda i: self.k[i], lambda i: self.v[i], self.lens,
                                        self.cu, scale, self.window, self.sink)
        most = max(self.lens)
        qn = np.sqrt((q * q).sum(-1)).max()
        kn = max(np.sqrt((k * k).sum(-1)).max() for k in self.k if k.size)
        # a score: a product of D terms in fp32 (a tensor core may truncate, so that
        # a half-ulp counts twice) of at most |q| |k|, its factors' roundings and
        # the exponential's own
        off = (2 * d + 8) * 2.0 ** -24 * qn * kn * scale + 2.0 ** -21
        # a weight's rounding to fp16, in the output and in the sum, and what fp16
        # flushes (2^-25 of the largest weight, times a value of at most vmax)
        vmax = max(np.abs(v).max() for v in self.v if v.size)
        if self.eight:
            vmax = 448 * float(np.nanmax(self.scales.cpu().numpy()))
        err = (2 * off + 2 * FP16_HALF_STEP + most * 2.0 ** -23) * mag + most * 2.0 ** -25 * vmax
        got = f64(out)
        half = BF16_HALF_STEP if out.dtype == torch.bfloat16 else 2.0 ** -24
        assert np.all(np.isfinite(got))
        tol = half * (np.abs(want) + err) + err
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
        lt = off + FP16_HALF_STEP + most * 2.0 ** -24 + 2.0 ** -22 * np.abs(wl)
        assert np.all(np.abs(f64(lse) - wl) <= lt), np.max(np.abs(f64(lse) - wl) / lt)


def case(*a, **kw):
    s = Step(*a, **kw)
    s.check(*s.call())
    return s


BOTH = pytest.mark.parametrize("eight", [False, True])
WINDOWS = [(0, 0), (1, 0), (1, 3), (16, 0), (17, 4), (100, 1), (64, 70), (2000, 5), (2 ** 31 - 1, 9)]


@BOTH
@pytest.mark.parametrize("window,sink", WINDOWS)
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens(eight, window, sink, d):
    lens = [1, 2, 15, 16, 17, 33, 64, 100, 129, 300, 511, 1000]
    case(lens, [1] * len(lens), 8, 2, d, 16, window, sink, eight, seed=window % 97 + sink)


@BOTH
@pytest.mark.parametrize("h,hkv", [(1, 1), (5, 5), (10, 2), (7, 1), (12, 2), (16, 1), (48, 2),
                                   (40, 1), (64, 1), (256, 1), (192, 1)])
def test_single_token_groups(eight, h, hkv):
    case([70, 513, 3], [1, 1, 1], h, hkv, 128, 32, 200, 6, eight, seed=h)
    case([70, 513, 3], [1, 1, 1], h, hkv, 64, 32, 0, 0, eight, seed=h)


@BOTH
@pytest.mark.parametrize("window,sink", [(0, 0), (700, 40), (333, 0)])
@pytest.mark.parametrize("times", [1, 9, 70])
def test_shares(eight, window, sink, times):
    # contexts in one share, cut by several, and many in one
    case([1500, 20, 1, 777] * times, [1, 1, 1, 1] * times, 8, 2, 128, 16, window, sink, eight,
         seed=9)
    # several queries are divided too
    case([1500, 20, 3, 777] * times, [5, 2, 3, 8] * times, 8, 2, 64, 16, window, sink, eight,
         seed=10)


@BOTH
def test_one_long_context(eight):
    # every share cuts the one context; requests without queries before and behind it
    case([40, 20000, 5], [0, 1, 0], 8, 1, 64, 64, 0, 0, eight, seed=11)
    case([20000], [3], 2, 1, 128, 64, 0, 0, eight, seed=12)


@BOTH
@pytest.mark.parametrize("h,hkv,ql", [(8, 2, [2, 8, 1, 0, 5]), (4, 4, [32, 1, 17, 9, 31]),
                                      (10, 2, [6, 1, 2, 0, 5]), (7, 1, [4, 4, 3, 2, 1]),
                                      (32, 2, [2, 2, 1, 2, 0])])
@pytest.mark.parametrize("window,sink", [(0, 0), (3, 2), (150, 17)])
def test_verification_steps(eight, h, hkv, ql, window, sink):
    lens = [a + b for a, b in zip([0, 300, 63, 40, 1000], ql)]
    case(lens, ql, h, hkv, 128, 16, window, sink, eight, seed=h + window)


@BOTH
@pytest.mark.parametrize("window,sink", WINDOWS)
@pytest.mark.parametrize("d", [64, 128])
def test_prompts(eight, window, sink, d):
    case([200, 129, 64, 333, 50], [200, 128, 40, 70, 33], 8, 2, d, 16, window, sink, eight,
         seed=window % 91 + d)


@BOTH
@pytest.mark.parametrize("h,hkv", [(1, 1), (10, 2), (7, 1), (12, 2), (16, 1), (48, 1), (96, 1),
                                   (128, 1), (28, 4)])
def test_prompt_groups(eight, h, hkv):
    # groups that divide 128 and groups that do not; chunks after a long context
    case([500, 260], [90, 260], h, hkv, 128, 64, 120, 5, eight, seed=h)
    case([300, 70], [100, 50], h, hkv, 64, 16, 0, 0, eight, seed=h)


@BOTH
@pytest.mark.parametrize("window,sink,bs", [(0, 0, 16), (300, 4, 64), (64, 130, 256)])
def test_mixed_steps(eight, window, sink, bs):
    lens = [900, 17, 400, 1, 700, 64, 1300, 300]
    ql = [1, 1, 350, 1, 0, 3, 129, 33]
    case(lens, ql, 16, 4, 64, bs, window, sink, eight, seed=bs)
    case(lens, ql, 16, 2, 128, bs, window, sink, eight, seed=bs + 1)


@BOTH
def test_long_context(eight):
    # past the lane-cached ids of several batches of chunks, and tiles far apart
    case([9000, 5000], [1, 2], 8, 2, 128, 16, 0, 0, eight, seed=1)
    case([9000, 5000], [1, 90], 4, 1, 64, 16, 3000, 700, eight, seed=2)
    case([4000], [40], 2, 1, 128, 16, 0, 0, eight, seed=3)


def test_scales_far_apart():
    # scales from 2^-30 to 2^30 in one context: the weights' exponents take them
    for ql in ([1], [60]):
        s = Step([400], ql, 4, 1, 128, 16, 0, 0, True, seed=5)
        r = np.random.RandomState(1)
        used = s.table[0]
        v = np.exp2(r.randint(-30, 31, len(used))).astype(np.float32)
        for b, blk in enumerate(used):
            old = float(s.scales[1, blk, 0])
            s.scales[1, blk] = float(v[b])
            s.v[0][b * 16:(b + 1) * 16] *= float(v[b]) / old
        s.check(*s.call())


def test_zero_scales():
    # a block of zeros kept with a scale of 0 takes part in the sum, not in the output
    s = Step([100], [1], 4, 1, 128, 16, 0, 0, True, seed=6)
    s.scales[1, s.table[0, 2]] = 0.0
    s.v[0][32:48] = 0
    s.check(*s.call())


@BOTH
def test_fp32_output_and_lse(eight):
    s = Step([300, 40, 9], [1, 40, 9], 8, 2, 128, 16, 100, 4, eight, seed=8)
    out = torch.full(s.q.shape, 7.0, device="cuda")
    o, lse = s.call(out=out)
    assert o is out
    s.check(o, lse)
    b, none = s.call(out_lse=None)
    assert none is None and torch.equal(b, out.to(torch.bfloat16))


def test_without_a_window_it_is_the_ordinary_call():
    s = Step([300, 40, 9, 200], [1, 40, 3, 1], 8, 2, 128, 16, 0, 0, False, seed=8)
    out, lse = torch.empty(s.q.shape, device="cuda"), torch.empty(s.q.shape[:2], device="cuda")
    s.call(out=out, out_lse=lse)
    want, wl = pkv.paged_attention_varlen(s.q, s.pool, i32(s.table), i32(s.cu), i32(s.lens), 40, 300,
                                          out_lse=torch.empty_like(lse))
    # each call rounds the weights of its prompts to fp16, by at most 2^-11 of
    # themselves: the ordinary call in the output and in the sum (an output is off by
    # at most 2 x 2^-11 of the largest value, its lse by 2^-11), this one in the
    # output alone (2^-11); fp32 sums of 300 terms and 2^-22 an exponential beside it
    vmax = max(np.abs(v).max() for v in s.v)
    assert np.max(np.abs(f64(out) - f64(want))) <= 3 * FP16_HALF_STEP * vmax + 1e-4
    assert np.max(np.abs(f64(lse) - f64(wl))) <= FP16_HALF_STEP + 1e-4
    # single tokens and short steps (the first query and the last four): 16 bits of
    # fraction in both
    few = [0] + list(range(41, out.shape[0]))
    assert np.max(np.abs(f64(out) - f64(want))[few]) <= 3 * 2.0 ** -16 * vmax + 1e-4


def test_a_cache_of_powers_of_two_is_the_bf16_cache_of_its_values():
    # what an append leaves stands for bf16 numbers: attention over those
    s = Step([300, 140], [1, 140], 8, 2, 128, 16, 0, 0, True, seed=9)
    s.scales = torch.exp2(torch.floor(torch.log2(s.scales)))
    s.scales[~torch.isfinite(s.scales)] = 1.0
    wide = (s.pool.float() * s.scales[:, :, None, :, None]).to(torch.bfloat16)
    out, lse = s.call(out=torch.empty(s.q.shape, device="cuda"))
    want, wl = pkv.paged_attention_varlen(s.q, wide, i32(s.table), i32(s.cu), i32(s.lens), 140, 300,
                                          out_lse=torch.empty_like(lse))
    assert torch.allclose(out, want, atol=2e-3) and torch.allclose(lse, wl, atol=1e-3)


@BOTH
def test_extreme_queries(eight):
    s = Step([40, 40, 40, 40], [1, 1, 40, 1], 2, 1, 64, 16, 0, 0, eight, seed=10)
    s.q[0] *= 1e4      # one key takes everything
    s.q[1] *= 1e-30    # every key the same
    s.q[3] = 0         # the second query of request 2, which sees two keys
    out, lse = s.call()
    got = f64(out)
    assert np.all(np.isfinite(got))
    v = s.v[1]
    assert np.allclose(got[1], v.mean(0), atol=2.0 ** -8 * np.abs(v).max())
    v = s.v[2][:2]
    assert np.allclose(got[3], v.mean(0), atol=2.0 ** -8 * np.abs(v).max())
    scores = f64(s.q[0]) @ s.k[0][:, 0].T
    for a in range(2):
        assert np.allclose(got[0, a], s.v[0][scores[a].argmax(), 0], rtol=2.0 ** -7)


@BOTH
def test_nan_where_it_is_seen(eight):
    # a NaN key or value that a query sees makes its output NaN, and no other's
    for ql in ([1, 1], [40, 40]):
        s = Step([60, 60], ql, 2, 1, 64, 16, 20, 2, eight, seed=11)
        at = int(s.table[0, 59 // 16])
        s.pool.view(torch.uint8 if eight else torch.int16)[0, at, 59 % 16] = 0x7f if eight else 0x7fc0
        out, lse = s.call()
        last = ql[0] - 1
        assert torch.isnan(out[last]).all()
        assert not torch.isnan(out[:last]).any() and not torch.isnan(out[last + 1:]).any()


@BOTH
def test_bad_blocks_and_lengths(eight):
    s = Step([100, 50, 64, 70], [1, 50, 1, 5], 4, 2, 128, 16, 40, 2, eight, seed=12)
    table, lens = s.table.copy(), list(s.lens)
    table[0, 5] = s.nb + 4      # seen by request 0
    lens[3] = 3                 # shorter than its queries
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = s.call()
    kw = dict(out=torch.full_like(out, 7.0), out_lse=torch.full_like(lse, 7.0), dev_status=st)
    good, s.table, s.lens = (s.table, s.lens), table, lens
    s_max = 100
    f = pkv.paged_attention_varlen_fp8 if eight else pkv.paged_attention_varlen_window
    a = (s.q, s.pool) + ((s.scales,) if eight else ()) + (i32(table), i32(s.cu), i32(lens), 50, s_max)
    got, gl = f(*a, **kw, window=40, num_sink=2) if eight else f(*a, 40, **kw, num_sink=2)
    assert st.item() == binding.DEV_BAD_BLOCK | binding.DEV_BAD_LENGTHS
    assert torch.equal(got[1:52], out[1:52]) and torch.equal(gl[1:52], lse[1:52])
    assert torch.all(got[52:] == 7.0) and torch.all(gl[52:] == 7.0)


@BOTH
def test_rows_behind_the_last_request_stay(eight):
    # a padded batch: queries behind the last request's
    s = Step([100, 50], [1, 40], 4, 2, 128, 16, 40, 2, eight, seed=13)
    s.q = torch.cat([s.q, torch.full_like(s.q[:5], float("nan"))])
    buf, out = guarded(s.q.shape, torch.bfloat16)
    out.fill_(7.0)
    lbuf, lse = guarded(s.q.shape[:2], torch.float32)
    lse.fill_(7.0)
    s.call(out=out, out_lse=lse)
    assert torch.all(out[41:] == 7.0) and torch.all(lse[41:] == 7.0)
    s.q = s.q[:41].contiguous()
    s.check(out[:41], lse[:41])
    assert guards_intact(buf, out.numel()) and guards_intact(lbuf, lse.numel())


@BOTH
@pytest.mark.parametrize("ql", [[1, 1, 1], [1, 70, 3]])
def test_streams_workspaces_and_graphs(eight, ql):
    s = Step([900, 300, 40], ql, 8, 2, 128, 16, 200, 4, eight, seed=14)
    want, wl = s.call()
    a = (s.q, s.pool) + ((s.scales,) if eight else ()) + (
        i32(s.table), i32(s.cu), i32(s.lens), max(ql), 900)
    f = pkv.paged_attention_varlen_fp8 if eight else pkv.paged_attention_varlen_window
    w = (lambda **k: f(*a, window=200, num_sink=4, **k)) if eight else (
        lambda **k: f(*a, 200, num_sink=4, **k))
    need = pkv.window_attention_workspace_size(max(ql), 8, 2, 128, 900, 200, 4, eight)
    # a workspace of anything, within guards
    buf, ws = guarded((need,), torch.uint8)
    ws.fill_(0xee)
    got, _ = w(workspace=ws)
    assert torch.equal(got, want) and guards_intact(buf, need)
    # two streams at once, each call with scratch of its own
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [w(stream=side[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o, _ in outs)
    # captured, replayed twice, and beside an eager call
    g = torch.cuda.CUDAGraph()
    lse = torch.empty_like(wl)
    with torch.cuda.graph(g):
        got, _ = w(out_lse=lse)
    for _ in range(2):
        got.fill_(0)
        g.replay()
        again, _ = w()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(lse, wl) and torch.equal(again, want)


@BOTH
def test_same_bits_whatever_the_blocks(eight):
    # the order of the physical blocks changes nothing
    a = Step([900, 300, 40], [1, 70, 3], 8, 2, 128, 16, 200, 4, eight, seed=15)
    want, wl = a.call()
    order = np.random.RandomState(3).permutation(a.nb)
    to = torch.from_numpy(order).cuda()
    pool = torch.empty_like(a.pool)
    kind = torch.uint8 if eight else torch.int16
    pool.view(kind)[:, to] = a.pool.view(kind)
    a.pool = pool
    if eight:
        sc = torch.empty_like(a.scales)
        sc[:, to] = a.scales
        a.scales = sc
    a.table = np.where(a.table >= 0, order[a.table], -1).astype(np.int32)
    got, gl = a.call()
    assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("inter,window", [(False, 0), (True, 60)])
def test_the_operators_together(inter, window):
    # a prompt, then single tokens, through the block manager: normed and rotated
    # into both caches, attended over both
    h, hkv, d, bs, eps = 8, 2, 64, 16, 1e-6
    r = np.random.RandomState(4)
    bm = pkv.BlockManager(40, bs)
    for i in range(3):
        bm.add_seq(i)
    wide = torch.full((2, 40, bs, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    eight = torch.full((2, 40, bs, hkv, d), float("nan"), device="cuda").to(torch.float8_e4m3fn)
    scales = torch.full((2, 40, hkv), float("nan"), device="cuda")
    qw, kw = (torch.from_numpy(r.rand(d).astype(np.float32) + 0.5).cuda() for _ in range(2))
    inv = pkv.rope_frequencies(d)[0].cuda()
    ks, vs = [np.zeros((0, hkv, d))] * 3, [np.zeros((0, hkv, d))] * 3
    for step in range(6):
        new = [70, 1, 33] if step == 0 else [1, 1, 2]
        table, lens, cu, slots, src, dst = bm.build_step([0, 1, 2], new, 12)
        t = int(cu[-1])
        q, k, v = (torch.from_numpy(r.standard_normal((t, n, d)).astype(np.float32)).to(
            torch.bfloat16).cuda() for n in (h, hkv, hkv))
        pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)])
        args = (i32(table), i32(cu), i32(lens), max(new))
        a = pkv.qk_norm_rope_kv_cache_write(q, wide, k, v, i32(pos), i32(slots), inv, qw, kw,
                                            eps=eps, interleaved=inter)
        b = pkv.qk_norm_rope_kv_cache_append_fp8(q, eight, scales, k, v, i32(pos), *args, inv, qw,
                                                 kw, eps=eps, interleaved=inter)
        assert torch.equal(a, b)
        o16, _ = pkv.paged_attention_varlen_window(a, wide, *args, int(max(lens)), window,
                                                   num_sink=2)
        o8, _ = pkv.paged_attention_varlen_fp8(a, eight, scales, *args, int(max(lens)),
                                               window=window, num_sink=2)
        from . import plain_budget
        kt = plain_budget.rope(plain.normed(f64(k), f64(kw), eps), pos, f64(inv), 1.0, inter)[0]
        qt = plain_budget.rope(plain.normed(f64(q), f64(qw), eps), pos, f64(inv), 1.0, inter)[0]
        for i in range(3):
            ks[i] = np.concatenate([ks[i], kt[cu[i]:cu[i + 1]]])
            vs[i] = np.concatenate([vs[i], f64(v)[cu[i]:cu[i + 1]]])
        want, _, mag = plain.attention(qt, lambda i: ks[i], lambda i: vs[i], lens, cu, d ** -0.5,
                                       window, 2)
        # bf16 keys and queries move a score of at most |q| |k| / 8 by 2^-7 of it
        qn, kn = np.sqrt((qt ** 2).sum(-1)).max(), max(np.sqrt((x ** 2).sum(-1)).max() for x in ks)
        off = 2.0 ** -7 * qn * kn * d ** -0.5
        assert np.all(np.abs(f64(o16) - want) <= (np.expm1(2 * off) + 2.0 ** -7) * mag)
        # 8-bit values: half a step of e4m3 on every key and value
        off = (2.0 ** -4 + 2.0 ** -8) * qn * kn * d ** -0.5
        assert np.all(np.abs(f64(o8) - want) <= (np.expm1(2 * off) + 2.0 ** -3) * mag + 1e-2)
        # and in the mean far nearer than that
        assert np.mean(np.abs(f64(o8) - want)) <= 0.06 * np.mean(mag)
    bm.close()
