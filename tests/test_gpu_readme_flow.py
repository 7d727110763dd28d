"""The README's step of requests held inside a budget, run as it is written there
(needs a GPU): the running sums after an eviction of some of the requests are
those of the shortened contexts."""
import os

import numpy as np
import pytest
import torch

import paged_kv_cache_varlen_gb300 as pkv

from . import plain_budget as plain
from .test_gpu_budget import f64, i32, normal

pytestmark = pytest.mark.gpu


def readme_blocks():
    """The indented blocks that follow the README's line about a budget."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md"), encoding="utf-8") as f:
        lines = f.read().split("\n")
    at = next(i for i, s in enumerate(lines) if "held inside a budget" in s)
    blocks, now = [], []
    for s in lines[at + 1:]:
        if s.startswith("    "):
            now.append(s[4:])
        elif s.strip() or not now:
            if now:
                blocks.append("\n".join(now))
                now = []
            if s.startswith("## "):
                break
        else:
            now.append("")
    return blocks


def test_the_readme_flow_goes_on_with_the_cut_sums():
    setup, step = readme_blocks()[:2]
    h, hkv, d, bs, budget, n = 8, 2, 128, 16, 160, 3
    nb = 96
    env = dict(torch=torch, pkv=pkv, manager=pkv.BlockManager(nb, bs), budget=budget,
               max_blocks=32, keep_blocks=budget // bs, ids=[10, 11, 12],
               weights=torch.full((n, hkv, 512), -3.0, device="cuda"),
               pool=torch.zeros((2, nb, bs, hkv, d), dtype=torch.bfloat16, device="cuda"))
    for i in env["ids"]:
        env["manager"].add_seq(i)
    exec(setup, env)
    position = [0] * n
    for number, (new, over) in enumerate([([200, 90, 260], []), ([1, 2, 1], [0, 2]),
                                          ([3, 1, 1], []), ([1, 1, 1], [2])]):
        t = sum(new)
        table, lens, cu, slots, copies, _ = env["manager"].build_step(env["ids"], new, 32)
        assert len(copies) == 0
        pos = np.concatenate([position[i] + np.arange(m) for i, m in enumerate(new)])
        qkv = normal((t, (h + 2 * hkv) * d), 50 + number)
        env.update(q=qkv[:, :h * d].view(t, h, d), k=qkv[:, h * d:(h + hkv) * d].view(t, hkv, d),
                   v=qkv[:, (h + hkv) * d:].view(t, hkv, d), positions=i32(pos), slots=i32(slots),
                   table=i32(table), cu=i32(cu), lens=i32(lens), max_q=max(new),
                   max_len=int(lens.max()), lse=torch.empty((t, h), device="cuda"), over=over)
        before, pool_before = f64(env["weights"]), env["pool"].clone()
        exec(step, env)
        # the keys that the step attended to: the pool before an eviction moved
        # any, with the step's own rows in the slots that it wrote
        rotated, _ = plain.rope(f64(env["k"]), pos, f64(env["inv_freq"]), env["factor"], False)
        rows = f64(pool_before[0].view(-1, hkv, d))
        if not over:
            rows = f64(env["pool"][0].view(-1, hkv, d))
            # (written by the kernel, so rounded as it rounds: one bf16 step at most)
            assert np.all(np.abs(rows[slots] - rotated) <= 2.0 ** -7 * np.abs(rotated) + 1e-4)
        else:
            again = pool_before.clone()
            pkv.rope_kv_cache_write(qkv[:, :h * d].view(t, h, d), again, env["k"], env["v"],
                                    env["positions"], env["slots"], env["inv_freq"],
                                    factor=env["factor"])
            rows = f64(again[0].view(-1, hkv, d))

        def keys(i):
            p = np.arange(lens[i])
            return rows[table[i, p // bs] * bs + p % bs]

        want, bound = plain.key_weights(before, f64(env["q"]), keys,
                                        env["lse"].cpu().double().numpy(), cu, lens,
                                        list(range(n)), None, 1.0, 1.0 / np.sqrt(d), before)
        got = f64(env["weights"])
        for i in range(n):
            for a in range(hkv):
                if i in over:
                    kept = env["kept"][over.index(i), a].cpu().numpy()
                    assert env["manager"].seq_len(env["ids"][i]) == budget
                    w, e, g = want[i, a, kept], bound[i, a, kept], got[i, a, :budget]
                else:
                    w, e, g = want[i, a, :lens[i]], bound[i, a, :lens[i]], got[i, a, :lens[i]]
                assert np.all(np.abs(g - w) <= e)
            position[i] += new[i]
    assert [env["manager"].seq_len(i) for i in env["ids"]] == [164, 94, 160]
