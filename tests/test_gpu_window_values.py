"""Attention through a window over bf16 values that are small, large, or of different
sizes from block to block, within bounds relative to these values."""
import numpy as np
import pytest
import torch

from paged_kv_cache_varlen_gb300 import binding
import paged_kv_cache_varlen_gb300 as pkv

from .test_gpu_window import BF16_HALF_STEP, FP16_HALF_STEP, Step, f64, i32

pytestmark = pytest.mark.gpu


def reference(s):
    """out, lse, the weighted sum of |value|, and the largest weight times the power of
    two that its values are held in, all in 64 bits."""
    q = f64(s.q)
    out, mag, top = (np.zeros(q.shape) for _ in range(3))
    lse = np.zeros(q.shape[:2])
    for i, L in enumerate(s.lens):
        t0, n = int(s.cu[i]), s.ql[i]
        pos, j = (L - n + np.arange(n))[:, None], np.arange(L)[None, :]
        seen = j <= pos
        if s.window:
            seen &= (pos - j < s.window) | (j < s.sink)
        live = seen.any(0)
        for h in range(s.h):
            k, v = (np.where(live[:, None], x[i][:, h // (s.h // s.hkv)], 0.0) for x in (s.k, s.v))
            sc = np.where(seen, q[t0:t0 + n, h] @ k.T * s.d ** -0.5, -np.inf)
            m = sc.max(1, keepdims=True)
            w = np.exp(sc - m)
            total = w.sum(1, keepdims=True)
            w /= total
            out[t0:t0 + n, h], mag[t0:t0 + n, h] = w @ v, w @ np.abs(v)
            lse[t0:t0 + n, h] = (m + np.log(total))[:, 0]
            # the largest value that a key's may be held with: of 64 keys, wherever they
            # begin, sinks beside any others
            size = np.pad(np.abs(v).max(1), 63)
            size = np.lib.stride_tricks.sliding_window_view(size, 127).max(1)
            if s.sink:
                size[:] = size.max()
            # values are held times 2^14 over the largest's binade, 2^64 at most
            held = np.exp2(np.clip(np.floor(np.log2(np.maximum(size, 1e-300))) - 14, -64, 113))
            top[t0:t0 + n, h] = (w * held).max(1)[:, None]
    return out, lse, mag, top


def check(s):
    out, lse = s.call(out=torch.full(s.q.shape, 7.0, device="cuda"))
    want, wl, mag, top = reference(s)
    q, n = f64(s.q), max(s.lens)
    qn = np.sqrt((q * q).sum(-1)).max()
    kn = max(np.sqrt((k * k).sum(-1)).max() for k in s.k)
    # a score's products (a tensor core may truncate), its exponential, and the roundings
    # of a sum with a power's exponent of up to 113 in fp32
    off = (2 * s.d + 8) * 2.0 ** -24 * qn * kn * s.d ** -0.5 + 2.0 ** -21 + 2.0 ** -16
    # fp16 weights, in the output and (not here) in the sum; what they flush: 2^-25 of the
    # largest, times a held value of at most 2^15; a held value's own 2^-25
    err = (2 * off + 2 * FP16_HALF_STEP + n * 2.0 ** -23) * mag + n * (2.0 ** -10 + 2.0 ** -25) * top
    got = f64(out)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= err), np.max(np.abs(got - want) / err)
    # the outputs are not lost: nearly all of what they are
    assert np.abs(got - want).sum() <= 2.0 ** -8 * np.abs(want).sum()
    lt = off + n * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -22 * np.abs(wl)
    assert np.all(np.abs(f64(lse) - wl) <= lt), np.max(np.abs(f64(lse) - wl) / lt)
    # and in bf16, rounded once
    b, _ = s.call()
    assert np.all(np.abs(f64(b) - got) <= BF16_HALF_STEP * np.abs(got) + 1e-40)


def scaled(s, factors):
    """The values of each request's block j times factors[j % len] (powers of two, 0)."""
    for i in range(len(s.lens)):
        for j in range(-(-s.lens[i] // s.bs)):
            f = float(factors[j % len(factors)])
            s.v[i][j * s.bs:(j + 1) * s.bs] *= f
            if s.table[i, j] >= 0:
                s.pool[1, int(s.table[i, j])] *= f
    return s


STEPS = [
    # prompts; few long items (cut); beside single tokens and short steps; single tokens
    ([200, 129, 333], [200, 128, 70], 8, 2), ([1500], [70], 8, 1),
    ([900, 17, 400, 64], [1, 1, 350, 3], 16, 4), ([300, 70], [1, 1], 8, 2),
]
FACTORS = {
    "2^-20": [2.0 ** -20], "2^-40": [2.0 ** -40], "2^-60": [2.0 ** -60], "2^17": [2.0 ** 17],
    "2^60": [2.0 ** 60], "2^110": [2.0 ** 110], "turns": [1.0, 2.0 ** -14, 2.0 ** 9],
    # (values of 64 keys are held together, exact down to 2^-31 of the largest)
    "apart": np.exp2(np.random.RandomState(1).randint(-8, 9, 97)),
    "rises": np.exp2(np.arange(97) - 48.0), "falls": np.exp2(48.0 - np.arange(97)),
    "zeros": [0.0, 2.0 ** -20, 0.0, 0.0],
}


@pytest.mark.parametrize("window,sink", [(0, 0), (100, 20)])
@pytest.mark.parametrize("lens,ql,h,hkv", STEPS)
@pytest.mark.parametrize("name", FACTORS)
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_any_size(lens, ql, h, hkv, name, d, window, sink):
    s = Step(lens, ql, h, hkv, d, 16, window, sink, False, seed=len(ql) + d)
    check(scaled(s, FACTORS[name]))


@pytest.mark.parametrize("bs", [64, 256])
def test_sizes_inside_longer_blocks(bs):
    # 16 keys to 16 keys
    s = Step([700, 300], [90, 300], 4, 2, 128, bs, 250, 3, False, seed=bs)
    r = np.random.RandomState(bs)
    for i in range(2):
        for j in range(-(-s.lens[i] // bs)):
            f = np.repeat(np.exp2(r.randint(-8, 9, bs // 16)), 16)
            rows = s.v[i][j * bs:(j + 1) * bs]
            rows *= f[:len(rows), None, None]
            if s.table[i, j] >= 0:
                s.pool[1, int(s.table[i, j])] *= torch.from_numpy(f).to(
                    torch.bfloat16).cuda()[:, None, None]
    check(s)


@pytest.mark.parametrize("value,flagged", [(65536.0, False), (3.3e38, False), (1e-38, False),
                                           (float("inf"), True), (float("nan"), True)])
def test_prompts_flag_infinite_values_alone(value, flagged):
    s = Step([200, 60], [70, 60], 4, 2, 128, 16, 0, 0, False, seed=3)
    s.pool[1, int(s.table[0, 199 // 16]), 199 % 16, 1, 5] = value
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = pkv.paged_attention_varlen_window(s.q, s.pool, i32(s.table), i32(s.cu), i32(s.lens), 70,
                                               200, 0, dev_status=st)
    assert st.item() == (binding.DEV_V_RANGE if flagged else 0)
    assert torch.isfinite(out[70:]).all()
    if not flagged:
        assert torch.isfinite(out).all()
