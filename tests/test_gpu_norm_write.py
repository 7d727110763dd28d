"""The normed rotary write and the writes into the 8-bit cache on the GPU,
against plain 64-bit forms written from their definitions."""
import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv
from paged_kv_cache_varlen_gb300 import binding

from . import plain_budget, plain_cache8 as plain
from .gpu_util import guarded, guards_intact

pytestmark = pytest.mark.gpu

BF16_HALF_STEP = 2.0 ** -8
E4M3_HALF_STEP = 2.0 ** -4


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


def heads(t, h, hkv, d, seed, packed=True, std=1.0):
    qkv = normal((t, (h + 2 * hkv) * d), seed, std)
    q = qkv[:, :h * d].view(t, h, d)
    k = qkv[:, h * d:(h + hkv) * d].view(t, hkv, d)
    v = qkv[:, (h + hkv) * d:].view(t, hkv, d)
    return (q, k, v) if packed else (q.contiguous(), k.contiguous(), v.contiguous())


def weights(d, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.rand((2, d), device="cuda", generator=g) + 0.5
    return w[0].to(dtype), w[1].to(dtype)


def frequencies(rot):
    if rot == 0:
        return None
    f = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    return torch.from_numpy(f).cuda()


def turned(x, weight, eps, offset, pos, inv, factor, inter):
    """The 64-bit result of a norm and a rotation, and its fp32 error's bound."""
    d = x.shape[-1]
    y = plain.normed(f64(x), None if weight is None else f64(weight), eps, offset)
    rel = plain.norm_error(d) if weight is not None else 0.0
    if inv is None:
        return y, rel * np.abs(y)
    want, mag = plain_budget.rope(y, pos, f64(inv), factor, inter)
    # a pair's angle is off by at most 2^-21 rad (its 24 bits of at most half a
    # turn, the function's own few ulp); two products and a sum
    return want, np.where(mag > 0, (2.0 ** -20 + rel) * mag, rel * np.abs(want))


def check_bf16(got, want, err):
    tol = BF16_HALF_STEP * (np.abs(want) + err) + err
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)


# ------------------------------------------------------------- into a bf16 pool
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,h,hkv,d,rot", [
    (1, 32, 8, 128, 128), (7, 4, 2, 64, 64), (65, 32, 8, 128, 64), (33, 16, 2, 64, 48),
    (5, 12, 2, 128, 20), (9, 5, 5, 128, 126), (3, 1, 1, 64, 2), (17, 28, 4, 128, 40),
    (6, 3, 3, 8, 8), (2, 2, 1, 24, 10), (300, 40, 8, 128, 128), (3, 2, 2, 512, 512),
    (4, 3, 1, 96, 96), (5, 2, 2, 80, 32), (2, 1, 1, 512, 30), (6, 8, 2, 128, 0), (1, 1, 1, 8, 0),
    (2500, 3, 1, 64, 32),
])
def test_norm_rope_write(t, h, hkv, d, rot, inter):
    r = np.random.RandomState(t + d)
    q, k, v = heads(t, h, hkv, d, t + rot)
    qw, kw = weights(d, t, torch.float32 if t % 2 else torch.bfloat16)
    inv, eps, offset = frequencies(rot), 1e-5, 1.0 if t % 3 == 0 else 0.0
    bs = 16
    nb = -(-t // bs) + 2
    slots = r.permutation(nb * bs)[:t]
    if t > 3:
        slots[t // 2] = -1
    pos = r.randint(0, 1 << 20, t)
    pool = normal((2, nb, bs, hkv, d), t + 1)
    pool0, st = pool.clone(), status_word()
    got = pkv.qk_norm_rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots), inv, qw, kw, eps=eps,
                                          weight_offset=offset, interleaved=inter, factor=1.25,
                                          dev_status=st)
    check_bf16(f64(got), *turned(q, qw, eps, offset, pos, inv, 1.25, inter))
    rows = f64(pool[0].reshape(-1, hkv, d))[slots[slots >= 0]]
    want, err = turned(k, kw, eps, offset, pos, inv, 1.25, inter)
    check_bf16(rows, want[slots >= 0], err[slots >= 0])
    # values are bit copies; every other slot is as it was
    flat = pool.view(torch.int16).view(2, -1, hkv, d)
    used = torch.from_numpy(slots[slots >= 0]).long().cuda()
    keep = torch.from_numpy(np.nonzero(slots >= 0)[0]).cuda()
    assert torch.equal(flat[1][used], v.contiguous().view(torch.int16)[keep])
    other = torch.ones(flat.shape[1], dtype=torch.bool, device="cuda")
    other[used] = False
    assert torch.equal(flat[:, other], pool0.view(torch.int16).view(2, -1, hkv, d)[:, other])
    assert st.item() == 0


@pytest.mark.parametrize("which", ["q", "k", "neither"])
@pytest.mark.parametrize("inter,rot", [(False, 128), (False, 60), (True, 60)])
def test_without_a_norm_it_is_the_rotary_write(which, inter, rot):
    t, h, hkv, d = 21, 8, 2, 128
    q, k, v = heads(t, h, hkv, d, 3)
    qw, kw = weights(d, 4)
    inv = frequencies(rot)
    pos, slots = i32(np.arange(t) * 977), i32(np.arange(t))
    a, b = normal((2, 2, 16, hkv, d), 5), normal((2, 2, 16, hkv, d), 5)
    x = pkv.qk_norm_rope_kv_cache_write(q, a, k, v, pos, slots, inv, qw if which == "q" else None,
                                        kw if which == "k" else None, interleaved=inter)
    y = pkv.rope_kv_cache_write(q, b, k, v, pos, slots, inv, interleaved=inter)
    # The two form their angles' cosines to an ulp (2^-24) and to pi 2^-25 more, and add
    # the products in other orders (two roundings): of |x| <= 8, sums of two products
    # differ by at most 16 (2^-24 + pi 2^-25 + 2^-24) < 2^-18, which may move a bf16
    # rounding to the next value, a step of 2^-7 at most
    same_q, same_k = [torch.allclose(m.float(), n.float(), rtol=2.0 ** -7, atol=2.0 ** -18)
                      for m, n in ((x, y), (a[0], b[0]))]
    assert same_q == (which != "q") and same_k == (which != "k")
    assert torch.equal(a[1], b[1])


@pytest.mark.parametrize("inter,rot", [(False, 128), (False, 60), (True, 60)])
def test_norm_rope_in_place(inter, rot):
    t, h, hkv, d = 19, 8, 2, 128
    q, k, v = heads(t, h, hkv, d, 5, packed=False)
    qw, kw = weights(d, 6)
    pos, slots = i32(np.arange(t) * 31), i32(np.arange(t)[::-1])
    a, b = normal((2, 2, 16, hkv, d), 5), normal((2, 2, 16, hkv, d), 5)
    want = pkv.qk_norm_rope_kv_cache_write(q, a, k, v, pos, slots, frequencies(rot), qw, kw,
                                           interleaved=inter)
    got = pkv.qk_norm_rope_kv_cache_write(q, b, k, v, pos, slots, frequencies(rot), qw, kw,
                                          interleaved=inter, q_out=q)
    assert got is q and torch.equal(q, want) and torch.equal(a, b)


def test_norm_edges():
    # a head of zeros stays zero with eps, NaN stays in its head, huge values
    # whose squares pass fp32 become zero, bad positions and slots are flagged
    t, h, hkv, d = 6, 2, 1, 64
    q, k, v = heads(t, h, hkv, d, 7, packed=False)
    q[0, 0] = 0
    q[1, 1, 5] = float("nan")
    q[2, 0] = 3e19
    qw, kw = weights(d, 8)
    pool = normal((2, 1, 16, hkv, d), 9)
    pool0, st = pool.clone(), status_word()
    out = torch.full_like(q, 7.0)
    pkv.qk_norm_rope_kv_cache_write(q, pool, k, v, i32([0, 1, 2, -1, 4, 5]), i32([0, 1, 2, 3, 16, 5]),
                                    frequencies(64), qw, kw, q_out=out, dev_status=st)
    assert st.item() == binding.DEV_BAD_POSITION | binding.DEV_BAD_SLOT
    assert torch.all(out[0, 0] == 0) and torch.all(out[2, 0] == 0)
    assert torch.isnan(out[1, 1]).all() and not torch.isnan(out[1, 0]).any()
    assert torch.all(out[3] == 7.0) and not torch.any(out[4] == 7.0)
    assert torch.equal(pool[:, 0, 3:5], pool0[:, 0, 3:5])
    assert torch.equal(pool[:, 0, 6:], pool0[:, 0, 6:])


# ------------------------------------------------------------ into an 8-bit pool
def step(lens, ql, bs, seed, extra=2):
    """Shuffled tables of a step; blocks behind a request's own stay -1."""
    r = np.random.RandomState(seed)
    n = [-(-L // bs) for L in lens]
    nb = sum(n) + extra
    ids = r.permutation(nb)
    table = np.full((len(lens), max(n + [1])), -1, np.int32)
    at = 0
    for i, m in enumerate(n):
        table[i, :m] = ids[at:at + m]
        at += m
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    return table, cu, nb


def pool8(nb, bs, hkv, d, seed):
    x = (normal((2, nb, bs, hkv, d), seed).float() * 100).clamp(-448, 448)
    r = np.random.RandomState(seed)
    s = torch.from_numpy(np.exp2(r.randint(-10, -4, (2, nb, hkv))).astype(np.float32)).cuda()
    return x.to(torch.float8_e4m3fn), s


def values(pool):
    return f64(pool.float())


LENGTHS = [
    ([5], [5], 16), ([1], [1], 16), ([16, 17, 33], [16, 1, 2], 16), ([100, 31, 64], [37, 0, 64], 32),
    ([300, 5, 77, 256], [300, 1, 77, 1], 64), ([511, 520], [300, 17], 256), ([40, 41, 42], [1, 1, 1], 16),
]


@pytest.mark.parametrize("lens,ql,bs", LENGTHS)
@pytest.mark.parametrize("hkv,d", [(8, 128), (1, 64), (3, 64)])
def test_append(lens, ql, bs, hkv, d):
    table, cu, nb = step(lens, ql, bs, sum(lens))
    t = int(cu[-1])
    _, k, v = heads(t, 1, hkv, d, t, std=3.0)
    pool, scales = pool8(nb, bs, hkv, d, t)
    want, ws, _ = plain.append(values(pool), f64(scales), f64(k), f64(v), table, cu, lens)
    st = status_word()
    pkv.kv_cache_append_fp8(pool, scales, k, v, i32(table), i32(cu), i32(lens), max(ql),
                            dev_status=st)
    # nothing but roundings of exact quotients: the same values, and untouched
    # rows, blocks and scales among them
    assert np.array_equal(f64(scales), ws)
    assert np.array_equal(values(pool), want)
    assert st.item() == 0


@pytest.mark.parametrize("inter,rot", [(False, 128), (False, 64), (True, 48), (False, 20), (True, 0)])
@pytest.mark.parametrize("lens,ql,bs", LENGTHS)
def test_norm_rope_append(lens, ql, bs, inter, rot):
    h, hkv, d = 6, 2, 128 if rot != 64 else 64
    table, cu, nb = step(lens, ql, bs, sum(lens))
    t = int(cu[-1])
    q, k, v = heads(t, h, hkv, d, t)
    qw, kw = weights(d, t, torch.float32 if t % 2 else torch.bfloat16)
    inv, pos = frequencies(rot), np.random.RandomState(t).randint(0, 1 << 20, t)
    pool, scales = pool8(nb, bs, hkv, d, t)
    before, sb = values(pool), f64(scales)
    st = status_word()
    out = pkv.qk_norm_rope_kv_cache_append_fp8(
        q, pool, scales, k, v, i32(pos), i32(table), i32(cu), i32(lens), max(ql), inv, qw, kw,
        eps=1e-5, interleaved=inter, factor=1.5, dev_status=st)
    assert st.item() == 0
    check_bf16(f64(out), *turned(q, qw, 1e-5, 0.0, pos, inv, 1.5, inter))
    kt, err = turned(k, kw, 1e-5, 0.0, pos, inv, 1.5, inter)
    want, ws, raw = plain.append(before, sb, kt, f64(v), table, cu, lens)
    got, gs = values(pool), f64(scales)
    # values are not computed with: the same bits
    assert np.array_equal(gs[1], ws[1]) and np.array_equal(got[1], want[1])
    # a key's scale: that of a largest magnitude off by its error
    assert np.all((gs[0] == ws[0]) | (gs[0] == 2 * ws[0]) | (2 * gs[0] == ws[0]))
    assert np.mean(gs[0] == ws[0]) > 0.98
    rows = ~np.isnan(raw[0])
    same = rows | (gs[0] == ws[0])[:, None, :, None]
    assert np.array_equal(got[0][~rows & same], want[0][~rows & same])
    s = gs[0][:, None, :, None]
    # half a step of e4m3 (of a value moved by the error), or of its smallest
    # values; the error in fp32 itself
    worst = np.max(err)
    tol = E4M3_HALF_STEP * (np.abs(raw[0]) + worst) + 2.0 ** -10 * s + worst
    assert np.all(np.abs(got[0] * s - raw[0])[rows] <= np.broadcast_to(tol, rows.shape)[rows])


def test_append_many_steps_of_one_token():
    # a context that grows by one token a step, its magnitudes rising and
    # falling by turns: the same values as the plain form keeps
    hkv, d, bs, n = 2, 64, 16, 40
    table, _, nb = step([n], [n], bs, 1)
    pool, scales = pool8(nb, bs, hkv, d, 2)
    want, ws = values(pool), f64(scales)
    for i in range(n):
        _, k, v = heads(1, 1, hkv, d, 100 + i, std=2.0 ** (i * 7 % 11 - 5))
        want, ws, _ = plain.append(want, ws, f64(k), f64(v), table, [0, 1], [i + 1])
        pkv.kv_cache_append_fp8(pool, scales, k, v, i32(table), i32([0, 1]), i32([i + 1]), 1)
    assert np.array_equal(values(pool), want) and np.array_equal(f64(scales), ws)


def test_append_extreme_values():
    hkv, d, bs = 1, 64, 16
    table, cu, nb = step([16, 16, 16, 3], [16, 16, 16, 2], bs, 1)
    t = int(cu[-1])
    _, k, v = heads(t, 1, hkv, d, 3, packed=False)
    k[:16] = 0  # a block of zeros
    k[16, 0, 3], v[17, 0, 4] = float("inf"), float("-inf")
    v[18, 0, 5] = float("nan")
    k[32:48] = 3.3e38
    v[32:48] = 1e-38
    pool, scales = pool8(nb, bs, hkv, d, 4)
    scales[:, table[3, 0]] = 0.3  # a scale that these writes would not have left
    want, ws, _ = plain.append(values(pool), f64(scales), f64(k), f64(v), table, cu, [16, 16, 16, 3])
    pkv.kv_cache_append_fp8(pool, scales, k, v, i32(table), i32(cu), i32([16, 16, 16, 3]), 16)
    assert np.array_equal(f64(scales), ws)
    assert np.array_equal(values(pool), want, equal_nan=True)
    assert ws[0, table[0, 0], 0] == 2.0 ** -100


def test_append_flags_and_skips():
    hkv, d, bs = 2, 64, 16
    lens, ql = [20, 18, 5, 33], [4, 2, 5, 20]
    table, cu, nb = step(lens, ql, bs, 5)
    t = int(cu[-1])
    q, k, v = heads(t, 4, hkv, d, 6)
    pool, scales = pool8(nb, bs, hkv, d, 7)
    before, sb = values(pool), f64(scales)
    bad = table.copy()
    bad[1, 1] = nb        # request 1's new block is outside the pool
    lens_bad = list(lens)
    lens_bad[2] = 4       # shorter than its queries
    pos = np.arange(t)
    pos[0] = -3           # request 0's first new token
    st, out = status_word(), torch.full((t, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.qk_norm_rope_kv_cache_append_fp8(q, pool, scales, k, v, i32(pos), i32(bad), i32(cu),
                                         i32(lens_bad), 20, None, q_out=out, dev_status=st)
    assert st.item() == (binding.DEV_BAD_BLOCK | binding.DEV_BAD_LENGTHS
                         | binding.DEV_BAD_POSITION)
    got = values(pool)
    blocks = set(range(nb))
    for i, b in ((0, 1), (3, 0), (3, 1), (3, 2)):
        blocks.discard(int(table[i, b]))
    rest = sorted(blocks)
    assert np.array_equal(got[:, rest], before[:, rest])
    assert np.array_equal(f64(scales)[:, rest], sb[:, rest])
    # the token of a bad position is left out, rows and q_out; the others are there
    assert torch.all(out[0] == 7.0) and torch.equal(out[1:6], q[1:6])
    assert torch.all(out[int(cu[2]):int(cu[3])] == 7.0) and torch.equal(out[int(cu[3]):], q[int(cu[3]):])
    row = got[:, table[0, 1], 0] * 1.0
    ratio = sb[:, table[0, 1]] / f64(scales)[:, table[0, 1]]
    assert np.array_equal(row, plain.e4m3(before[:, table[0, 1], 0] * ratio[..., None])) or \
        np.array_equal(row, before[:, table[0, 1], 0])


@pytest.mark.parametrize("b,bs", [(700, 16), (300, 64)])
def test_append_many_requests(b, bs):
    r = np.random.RandomState(b)
    ql = r.choice([0, 1, 1, 1, 2, 17, 50], b)
    lens = ql + r.randint(0, 100, b)
    table, cu, nb = step(lens.tolist(), ql.tolist(), bs, b)
    t = int(cu[-1])
    _, k, v = heads(t, 1, 2, 64, 8)
    pool, scales = pool8(nb, bs, 2, 64, 9)
    want, ws, _ = plain.append(values(pool), f64(scales), f64(k), f64(v), table, cu, lens)
    pkv.kv_cache_append_fp8(pool, scales, k, v, i32(table), i32(cu), i32(lens), 50)
    assert np.array_equal(f64(scales), ws) and np.array_equal(values(pool), want)


def test_guards_around_the_outputs():
    hkv, d, bs = 2, 128, 16
    lens, ql = [30, 16], [9, 16]
    table, cu, nb = step(lens, ql, bs, 5, extra=0)
    q, k, v = heads(25, 4, hkv, d, 6)
    pool, scales = pool8(nb, bs, hkv, d, 7)
    buf, gp = guarded(pool.shape, torch.uint8)
    gp.copy_(pool.view(torch.uint8))
    sbuf, gs = guarded(scales.shape, torch.float32)
    gs.copy_(scales)
    obuf, go = guarded(q.shape, torch.bfloat16)
    pkv.qk_norm_rope_kv_cache_append_fp8(q, gp.view(torch.float8_e4m3fn), gs, k, v,
                                         i32(np.arange(25)), i32(table), i32(cu), i32(lens), 16,
                                         frequencies(128), *weights(d, 1), q_out=go)
    assert guards_intact(buf, pool.numel()) and guards_intact(sbuf, scales.numel())
    assert guards_intact(obuf, q.numel())


def test_streams_and_graphs():
    # on another stream than the current one, and captured and replayed: the
    # same as an ordinary call
    hkv, d, bs = 2, 128, 16
    lens, ql = [30, 16, 50], [9, 16, 1]
    table, cu, nb = step(lens, ql, bs, 5)
    q, k, v = heads(26, 4, hkv, d, 6)
    qw, kw = weights(d, 1)
    tab, cut, ln, pos, inv = i32(table), i32(cu), i32(lens), i32(np.arange(26)), frequencies(128)
    runs = []
    side = torch.cuda.Stream()
    for how in ("plain", "stream", "graph"):
        pool, scales = pool8(nb, bs, hkv, d, 7)
        wide = normal((2, nb, bs, hkv, d), 8)
        torch.cuda.synchronize()

        def call(stream=None):
            a = pkv.qk_norm_rope_kv_cache_append_fp8(q, pool, scales, k, v, pos, tab, cut, ln, 16,
                                                     inv, qw, kw, stream=stream)
            b = pkv.qk_norm_rope_kv_cache_write(q, wide, k, v, pos, pos, inv, qw, kw, stream=stream)
            return a, b

        if how == "stream":
            out = call(side)
            side.synchronize()
        elif how == "graph":
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = call()
            g.replay()
            g.replay()
        else:
            out = call()
        torch.cuda.synchronize()
        runs.append([values(pool), f64(scales), f64(wide), f64(out[0]), f64(out[1])])
    for other in runs[1:]:
        assert all(np.array_equal(a, b) for a, b in zip(runs[0], other))
