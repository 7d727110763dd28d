"""The 8-bit cache's block copies, long requests that are few (their keys are cut
into shares), batches of many requests, and what the Python calls refuse, on the
GPU."""
import os
import re
import textwrap

import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv
from paged_kv_cache_varlen_gb300 import binding

from . import plain_cache8 as plain
from .gpu_util import guarded, guards_intact
from .test_gpu_norm_write import pool8, step, values
from .test_gpu_window import Step, case, f64, i32

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("eight", [False, True])


def _pool(nb, bs, hkv, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool = torch.randint(0, 256, (2, nb, bs, hkv, d), generator=g, device="cuda",
                         dtype=torch.uint8).view(torch.float8_e4m3fn)  # (NaN too)
    return pool, torch.rand((2, nb, hkv), generator=g, device="cuda")


@pytest.mark.parametrize("nb,bs,hkv,d", [(9, 16, 2, 64), (7, 256, 8, 128), (12, 16, 300, 64)])
def test_copied_blocks_keep_their_bits(nb, bs, hkv, d):
    pool, scales = _pool(nb, bs, hkv, d, 1)
    a, b = pool.view(torch.uint8).clone(), scales.clone()
    src, dst = [0, 0, nb - 2], [1, nb - 1, 3]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.copy_blocks_fp8(pool, scales, i32(src), i32(dst), dev_status=st)
    a[:, dst], b[:, dst] = a[:, src], b[:, src]
    assert torch.equal(pool.view(torch.uint8), a) and torch.equal(scales, b) and st.item() == 0
    # a bad id is flagged, the other copies are made
    pkv.copy_blocks_fp8(pool, scales, i32([nb, 2, -1]), i32([2, 4, 0]), dev_status=st)
    a[:, 4], b[:, 4] = a[:, 2], b[:, 2]
    assert torch.equal(pool.view(torch.uint8), a) and torch.equal(scales, b) and st.item() != 0
    pkv.copy_blocks_fp8(pool, scales, i32([]), i32([]))
    with pytest.raises(ValueError):
        pkv.copy_blocks_fp8(pool, scales[:, 1:].contiguous(), i32([0]), i32([1]))
    with pytest.raises(ValueError):
        pkv.copy_blocks_fp8(pool, scales, i32([0, 1]), i32([1]))
    with pytest.raises(TypeError):
        pkv.copy_blocks_fp8(pool.view(torch.uint8), scales, i32([0]), i32([1]))


@pytest.mark.parametrize("bs", [16, 64, 256])
@pytest.mark.parametrize("hkv,d", [(8, 128), (1, 64), (3, 64)])
def test_single_tokens_into_blocks(hkv, d, bs):
    # a token a request at most: rows of their own. Requests without one, first rows of
    # blocks, rows that make the block's scale grow and that do not, tokens of nobody
    r = np.random.RandomState(bs + d)
    ql = r.randint(0, 2, 90)
    lens = r.randint(1, 400, 90)
    lens[:6] = bs + 1, bs, 1, 2 * bs, 17, 16
    table, cu, nb = step(lens.tolist(), ql.tolist(), bs, d)
    t = int(cu[-1])
    g = torch.Generator(device="cuda").manual_seed(bs)
    size = torch.exp2(torch.randint(-6, 6, (t + 3, 1, 1), generator=g, device="cuda").float())
    k, v = ((torch.randn((t + 3, hkv, d), generator=g, device="cuda") * size).to(torch.bfloat16)
            for _ in "kv")
    pool, scales = pool8(nb, bs, hkv, d, bs)
    want, ws, _ = plain.append(values(pool), f64(scales), f64(k), f64(v), table, cu, lens)
    assert 0 < np.mean(ws != f64(scales)) < 0.5
    pkv.kv_cache_append_fp8(pool, scales, k, v, i32(table), i32(cu), i32(lens), 1)
    assert np.array_equal(f64(scales), ws) and np.array_equal(values(pool), want)


def test_single_tokens_that_are_flagged():
    hkv, d, bs = 2, 64, 16
    lens, ql = [20, 18, 5, 33, 9], [1, 1, 1, 1, 1]
    table, cu, nb = step(lens, ql, bs, 5)
    q, k, v = (torch.randn((5, n, d), device="cuda").to(torch.bfloat16) for n in (4, hkv, hkv))
    pool, scales = pool8(nb, bs, hkv, d, 7)
    before, sb = values(pool), f64(scales)
    bad = table.copy()
    bad[1, 1] = nb                                   # a block outside the pool
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((5, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.qk_norm_rope_kv_cache_append_fp8(q, pool, scales, k, v, i32([-1, 1, 2, 3, 4]), i32(bad),
                                         i32(cu), i32([20, 18, 0, 33, 200]), 1, None, q_out=out,
                                         dev_status=st)
    # (200: past the table)
    assert st.item() == (binding.DEV_BAD_BLOCK | binding.DEV_BAD_LENGTHS
                         | binding.DEV_BAD_POSITION)
    skipped = [0, 2, 4]
    assert torch.all(out[skipped] == 7.0) and torch.equal(out[[1, 3]], q[[1, 3]])
    rest = [b for b in range(nb) if b not in (table[0, 1], table[3, 2])]
    assert np.array_equal(values(pool)[:, rest], before[:, rest])
    assert np.array_equal(f64(scales)[:, rest], sb[:, rest])
    # the bad position's block keeps its rows
    assert np.array_equal(values(pool)[:, table[0, 1]], before[:, table[0, 1]])
    # the good token is there
    want, ws, _ = plain.append(before, sb, f64(k[3:4]), f64(v[3:4]), table[3:4], [0, 1], [33])
    assert np.array_equal(values(pool)[:, table[3, 2]], want[:, table[3, 2]])


def test_a_fork_writes_into_copies():
    # two continuations of one prompt: the shared last block is copied with its scale
    # before the child's first token is written
    h, hkv, d, bs = 4, 2, 64, 16
    r = np.random.RandomState(2)
    bm = pkv.BlockManager(20, bs)
    bm.add_seq(0)
    pool = torch.zeros((2, 20, bs, hkv, d), device="cuda").to(torch.float8_e4m3fn)
    scales = torch.zeros((2, 20, hkv), device="cuda")
    ks, vs = {0: np.zeros((0, hkv, d))}, {0: np.zeros((0, hkv, d))}
    for step in range(5):
        if step == 1:
            bm.fork(0, 1)
            ks[1], vs[1] = ks[0], vs[0]
        ids, new = ([0], [37]) if step == 0 else ([0, 1], [1, 1])
        table, lens, cu, _, src, dst = bm.build_step(ids, new, 8)
        if len(src):
            pkv.copy_blocks_fp8(pool, scales, i32(src), i32(dst))
        assert bool(len(src)) == (step == 1)
        t = int(cu[-1])
        q, k, v = (torch.from_numpy(r.standard_normal((t, n, d)).astype(np.float32)).to(
            torch.bfloat16).cuda() for n in (h, hkv, hkv))
        args = (i32(table), i32(cu), i32(lens), max(new))
        pkv.kv_cache_append_fp8(pool, scales, k, v, *args)
        out, _ = pkv.paged_attention_varlen_fp8(q, pool, scales, *args, int(max(lens)))
        for i, s in enumerate(ids):
            ks[s] = np.concatenate([ks[s], f64(k)[cu[i]:cu[i + 1]]])
            vs[s] = np.concatenate([vs[s], f64(v)[cu[i]:cu[i + 1]]])
        want, _, mag = plain.attention(f64(q), lambda i: ks[ids[i]], lambda i: vs[ids[i]], lens, cu,
                                       d ** -0.5)
        qn = np.sqrt((f64(q) ** 2).sum(-1)).max()
        kn = max(np.sqrt((x ** 2).sum(-1)).max() for x in ks.values())
        # half a step of e4m3 on every key and value
        off = (2.0 ** -4 + 2.0 ** -8) * qn * kn * d ** -0.5
        assert np.all(np.abs(f64(out) - want) <= (np.expm1(2 * off) + 2.0 ** -3) * mag + 1e-2)
        assert np.mean(np.abs(f64(out) - want)) <= 0.06 * np.mean(mag)
    bm.close()


# Few items (joined by a grid of their own) and a few dozen (by the CTA that comes
# last); sinks and a window that lie in different pieces, several heads, odd sizes.
CUT = [
    ([5000, 700], [70, 40], 8, 2), ([2500], [300], 7, 1), ([1999, 3, 4001], [33, 3, 65], 12, 4),
    ([3000, 2600], [700, 500], 8, 2), ([1200] * 5 + [900], [290, 1, 200, 310, 1, 77], 16, 4),
]


@BOTH
@pytest.mark.parametrize("window,sink", [(0, 0), (1500, 100), (900, 3)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,ql,h,hkv", CUT)
def test_few_long_requests(eight, lens, ql, h, hkv, d, window, sink):
    s = case(lens, ql, h, hkv, d, 16, window, sink, eight, seed=len(ql) + d)
    # the same bits at every call
    want, wl = s.call()
    for _ in range(3):
        out, lse = s.call()
        assert torch.equal(out, want) and torch.equal(lse, wl)


@BOTH
@pytest.mark.parametrize("lens,ql,h,hkv", [CUT[0], CUT[3]])
def test_few_long_requests_in_graphs(eight, lens, ql, h, hkv):
    s = Step(lens, ql, h, hkv, 128, 16, 0, 0, eight, seed=3)
    want, wl = s.call()
    need = pkv.window_attention_workspace_size(max(ql), h, hkv, 128, max(lens), 0, 0, eight)
    a = (s.q, s.pool) + ((s.scales,) if eight else ()) + (
        i32(s.table), i32(s.cu), i32(s.lens), max(ql), max(lens)) + (() if eight else (0,))
    f = pkv.paged_attention_varlen_fp8 if eight else pkv.paged_attention_varlen_window
    graphs, outs, held = [], [], []
    for i in range(2):  # a workspace each: they run beside one another
        buf, ws = guarded((need,), torch.uint8)
        ws.fill_(0x5a + i)
        out = torch.empty_like(want)
        f(*a, out=out, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f(*a, out=out, workspace=ws)
        graphs.append(g)
        outs.append(out)
        held.append(buf)
    for _ in range(3):
        side = [torch.cuda.Stream() for _ in graphs]
        for g, st, o in zip(graphs, side, outs):
            o.fill_(0)
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    assert all(guards_intact(b, need) for b in held)


@BOTH
@pytest.mark.parametrize("b", [768, 769, 1500])
def test_many_requests_with_prompts_among_them(eight, b):
    r = np.random.RandomState(b)
    ql = np.where(r.rand(b) < 0.03, r.randint(9, 90, b), 1)
    ql[[0, b - 1]] = 40, 70
    lens = ql + r.randint(0, 40, b)
    case(lens.tolist(), ql.tolist(), 8, 2, 64, 16, 50, 3, eight, seed=b)


def test_the_readme_step_over_the_8_bit_cache():
    # the README's blocks, run as they are written there
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md"), encoding="utf-8") as f:
        text = f.read()
    part = text[text.index("over the 8-bit cache and through a window."):]
    blocks = [textwrap.dedent(b) for b in re.findall(r"(?:^    .*\n(?:^\n(?=    ))?)+", part, re.M)]
    r = np.random.RandomState(5)
    s = dict(torch=torch, pkv=pkv, num_blocks=200, num_kv_heads=2, inv_freq=pkv.rope_frequencies(
        128)[0].cuda(), q_norm=torch.ones(128, device="cuda"), k_norm=torch.ones(128, device="cuda"))
    exec(blocks[0], s)
    bm = pkv.BlockManager(200, 16)
    for i in range(2):
        bm.add_seq(i)
    for step in range(3):
        new = [1100, 30] if step == 0 else [1, 1]
        table, lens, cu, _, src, dst = bm.build_step([0, 1], new, 80)
        t = int(cu[-1])
        s.update(table=i32(table), lens=i32(lens), cu=i32(cu), src=i32(src), dst=i32(dst),
                 max_q=max(new), max_len=int(max(lens)), positions=i32(np.concatenate(
                     [np.arange(L - n, L) for L, n in zip(lens, new)])))
        for name, n in (("q", 8), ("k", 2), ("v", 2)):
            s[name] = torch.from_numpy(r.standard_normal((t, n, 128)).astype(np.float32)).to(
                torch.bfloat16).cuda()
        exec(blocks[1], s)
        assert s["out"].shape == (t, 8, 128) and bool(torch.isfinite(s["out"]).all())
        # a request's last row is a mean of its values
        assert 0 < float(s["out"].float().abs().max()) < 5
    bm.close()


@BOTH
@pytest.mark.parametrize("ql", [[1, 1], [40, 1]])
def test_blocks_past_4_gb(eight, ql):
    # the same blocks at the end of a pool of more than 2^32 bytes a half
    hkv, d, bs, nb = 8, 128, 16, 300_000 if eight else 150_000
    s = Step([300, 77], ql, 16, hkv, d, bs, 100, 3, eight, seed=6)
    want, wl = s.call()
    pool = torch.empty((2, nb, bs, hkv, d), dtype=s.pool.dtype, device="cuda")
    kind = torch.uint8 if eight else torch.int16
    pool.view(kind)[:, nb - s.nb:] = s.pool.view(kind)
    s.pool = pool
    if eight:
        scales = torch.empty((2, nb, hkv), device="cuda")
        scales[:, nb - s.nb:] = s.scales
        s.scales = scales
    s.table = np.where(s.table >= 0, s.table + nb - s.nb, -1).astype(np.int32)
    got, gl = s.call()
    assert torch.equal(got, want) and torch.equal(gl, wl)
    # and written there
    t = sum(ql)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((t, 16, d), device="cuda", generator=g).to(torch.bfloat16)
    k, v = (torch.randn((t, hkv, d), device="cuda", generator=g).to(torch.bfloat16) for _ in "kv")
    w = torch.ones(d, device="cuda")
    inv = pkv.rope_frequencies(d)[0].cuda()
    pos = i32(np.arange(t))
    if not eight:
        slots = (nb - 1) * bs + np.arange(t) - 40
        pkv.qk_norm_rope_kv_cache_write(q, s.pool, k, v, pos, i32(slots), inv, w, w)
        rows = s.pool.view(2, -1, hkv, d)[1, torch.from_numpy(slots).cuda()]
        assert torch.equal(rows, v)
        return
    table = np.full((2, 20), -1)
    for i, L in enumerate(s.lens):
        table[i, (L - ql[i]) // bs:(L - 1) // bs + 1] = nb - 1 - 5 * i - np.arange(
            (L - 1) // bs + 1 - (L - ql[i]) // bs)
    small = torch.zeros((2, 10, bs, hkv, d), device="cuda").to(torch.float8_e4m3fn)
    near = torch.zeros((2, 10, hkv), device="cuda")
    s.pool.view(torch.uint8)[:, nb - 10:] = 0
    s.scales[:, nb - 10:] = 0
    for p, sc, tab in ((s.pool, s.scales, table), (small, near, np.where(table < 0, -1, table - (nb - 10)))):
        pkv.qk_norm_rope_kv_cache_append_fp8(q, p, sc, k, v, pos, i32(tab), i32(s.cu), i32(s.lens),
                                             max(ql), inv, w, w)
    assert torch.equal(s.pool.view(torch.uint8)[:, nb - 10:], small.view(torch.uint8))
    assert torch.equal(s.scales[:, nb - 10:], near) and bool((near > 0).any())
    # copied there
    pkv.copy_blocks_fp8(s.pool, s.scales, i32([nb - 1]), i32([nb - 20]))
    assert torch.equal(s.pool.view(torch.uint8)[:, nb - 20], small.view(torch.uint8)[:, 9])
    assert torch.equal(s.scales[:, nb - 20], near[:, 9])


def _inputs():
    q = torch.zeros((4, 8, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    pool, scales = _pool(6, 16, 2, 64, 1)
    return dict(q=q, pool=pool, wide=torch.zeros((2, 6, 16, 2, 64), dtype=torch.bfloat16,
                                                 device="cuda"), scales=scales, k=k, v=k.clone(),
                table=i32([[0, 1], [2, 3]]), cu=i32([0, 1, 4]), lens=i32([5, 20]), pos=i32([4, 17, 18, 19]),
                slots=i32([4, 49, 50, 51]), inv=torch.ones(32, dtype=torch.float64, device="cuda"),
                qw=torch.ones(64, device="cuda"), kw=torch.ones(64, device="cuda"))


def _write(s):
    return pkv.qk_norm_rope_kv_cache_write(s["q"], s["wide"], s["k"], s["v"], s["pos"], s["slots"],
                                           s["inv"], s["qw"], s["kw"])


def _append(s):
    return pkv.kv_cache_append_fp8(s["pool"], s["scales"], s["k"], s["v"], s["table"], s["cu"],
                                   s["lens"], 3)


def _norm_append(s):
    return pkv.qk_norm_rope_kv_cache_append_fp8(
        s["q"], s["pool"], s["scales"], s["k"], s["v"], s["pos"], s["table"], s["cu"], s["lens"], 3,
        s["inv"], s["qw"], s["kw"])


def _window(s):
    return pkv.paged_attention_varlen_window(s["q"], s["wide"], s["table"], s["cu"], s["lens"], 3,
                                             20, 7)


def _fp8(s):
    return pkv.paged_attention_varlen_fp8(s["q"], s["pool"], s["scales"], s["table"], s["cu"],
                                          s["lens"], 3, 20)


CALLS = {"write": (_write, "q wide k v pos slots inv qw kw"),
         "append": (_append, "pool scales k v table cu lens"),
         "norm_append": (_norm_append, "q pool scales k v pos table cu lens inv qw kw"),
         "window": (_window, "q wide table cu lens"),
         "fp8": (_fp8, "q pool scales table cu lens")}


@pytest.mark.parametrize("name", CALLS)
def test_python_refusals(name):
    f, args = CALLS[name]
    f(_inputs())
    torch.cuda.synchronize()
    for a in args.split():
        for change in ("host", "type", "dims", "shape"):
            s = _inputs()
            t = s[a]
            if change == "host":
                s[a] = t.cpu()
            elif change == "type":
                s[a] = t.float().half()
            elif change == "dims":
                s[a] = t[None]
            elif a in ("pool", "wide"):  # a pool of one half
                s[a] = t[:1]
            elif a == "inv":  # more pairs than a head has
                s[a] = t.repeat(2)[:33]
            elif a == "q":  # another head size
                s[a] = t[..., :-8].contiguous()
            elif a in ("table", "cu", "lens", "pos", "slots", "qw", "kw"):
                s[a] = t[:-1]
            else:
                s[a] = t[:, :-1].contiguous()
            with pytest.raises((TypeError, ValueError, pkv.PkvError)):
                f(s)
    torch.cuda.synchronize()
    f(_inputs())  # and nothing is left behind
    torch.cuda.synchronize()
