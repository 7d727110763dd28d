"""Measured cases of four more operators on the way into and out of the paged
cache: norms of the query and key heads with the rotation and the cache write
in the same pass, the write into a cache held in 8 bits with a scale for each
block of tokens and KV head, the attention that reads that cache, and attention
through a sliding window whose first tokens stay visible.

They are the steps of one layer: ``qk_norm_rope_kv_cache_write`` fills a bf16
pool that ``paged_attention_varlen_window`` reads; the
``..._kv_cache_append_fp8`` calls fill an 8-bit pool that
``paged_attention_varlen_fp8`` reads, through a window too where a layer has one.

``own`` chooses between the plain torch forms below and the library's calls.
Ragged lengths follow from the case alone (``shape`` seeds them), so that
``work`` can count them; every value follows from the seed.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _norm(name, tokens, heads, kv_heads, head_dim, rotary_dim, interleaved, max_pos,
          block_size=16):
    return {"name": name, "op": "norm", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rotary_dim": rotary_dim, "interleaved": interleaved,
            "max_pos": max_pos, "block_size": block_size}


def _append(name, seqs, min_q, max_q, min_len, max_len, heads, kv_heads, head_dim, rotary_dim,
            shape, block_size=16):
    """rotary_dim 0: keys that are rotated already, no queries and no norms."""
    return {"name": name, "op": "append", "seqs": seqs, "min_q": min_q, "max_q": max_q,
            "min_len": min_len, "max_len": max_len, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rotary_dim": rotary_dim, "shape": shape,
            "block_size": block_size}


def _attend(name, bits, seqs, min_q, max_q, min_len, max_len, heads, kv_heads, head_dim, window,
            sink, shape, block_size=16):
    """bits: of a cached value (8: e4m3 and scales, 16: bf16). window 0: every key is seen."""
    return {"name": name, "op": "attend", "bits": bits, "seqs": seqs, "min_q": min_q,
            "max_q": max_q, "min_len": min_len, "max_len": max_len, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "window": window, "sink": sink,
            "shape": shape, "block_size": block_size}


def listed():
    return [
        # one request's next token, far into a context: the smallest call, all latency
        _norm("norm_step_1", 1, 32, 8, 128, 128, False, 131072),
        # an odd-sized chunk, adjacent pairs, three quarters of a 64-wide head rotated
        _norm("norm_part_777", 777, 16, 2, 64, 48, True, 8192),
        # a long prompt
        _norm("norm_prompt_8192", 8192, 32, 8, 128, 128, False, 131072),
        # the decode step of 64 requests: norms, rotation and the 8-bit write of one token each
        _append("append_step_64", 64, 1, 1, 512, 4096, 32, 8, 128, 128, 1),
        # a mixed step of a smaller model that prepares its keys itself: only the 8-bit write
        _append("append_mixed_13", 13, 1, 700, 700, 5000, 16, 4, 64, 0, 2, 32),
        # a long prompt into fresh blocks: the most bytes of a write
        _append("append_prompt_8192", 1, 8192, 8192, 8192, 8192, 32, 8, 128, 128, 3),
        # the decode step of 64 requests over an 8-bit cache (the benchmark's decode shape)
        _attend("fp8_step_64", 8, 64, 1, 1, 512, 4096, 32, 8, 128, 0, 0, 4),
        # decodes over contexts of 32K to 128K tokens: the most bytes
        _attend("fp8_step_long", 8, 8, 1, 1, 32768, 131072, 32, 8, 128, 0, 0, 5),
        # prompt chunks over contexts that are partly cached already: products of 8-bit keys
        _attend("fp8_chunks_2048", 8, 2, 1500, 2048, 4096, 8192, 32, 8, 128, 0, 0, 6),
        # a mixed step of a smaller model, single tokens beside odd-sized chunks, in a window
        _attend("fp8_window_mixed_13", 8, 13, 1, 700, 700, 5000, 16, 4, 64, 513, 5, 7, 32),
        # the decode step of 64 requests whose blocks behind the window were given back
        _attend("window_step_64", 16, 64, 1, 1, 512, 16384, 32, 8, 128, 1024, 4, 8),
        # one whole prompt through a window: the most arithmetic
        _attend("window_prompt_8192", 16, 1, 8192, 8192, 8192, 8192, 32, 8, 128, 1024, 4, 9),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


_HEADS = [(32, 8), (32, 8), (16, 4), (16, 2), (8, 8), (40, 8), (28, 4), (12, 2), (8, 1), (64, 8)]


def draw(rng):
    op = rng.choice(["norm", "append", "fp8", "fp8", "window", "window"])
    heads, kv_heads = rng.choice(_HEADS)
    head_dim = rng.choice([64, 128])
    block_size = rng.choice([16, 16, 32, 64])
    shape = rng.randrange(1 << 20)
    rotary_dim = rng.choice([head_dim, head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)])
    if op == "norm":
        c = _norm("", _log_int(rng, 1, 4096), heads, kv_heads, head_dim, rotary_dim,
                  rng.random() < 0.5, _log_int(rng, 2, 1 << 20), block_size)
    elif op == "append":
        longest = _log_int(rng, 2, 16384)
        max_q = rng.choice([1, _log_int(rng, 1, min(longest, 4096))])
        seqs = _log_int(rng, 1, max(1, min(128, 100000 // longest, 16384 // max_q)))
        c = _append("", seqs, max(1, max_q // 16), max_q, max(max_q, longest // 4), longest, heads,
                    kv_heads, head_dim, rng.choice([0, rotary_dim]), shape, block_size)
    else:
        bits = 8 if op == "fp8" else 16
        window = 0 if op == "fp8" and rng.random() < 0.6 else _log_int(rng, 1, 8192)
        sink = rng.choice([0, 4, rng.randint(1, 70)]) if window else 0
        if rng.random() < 0.5:  # single tokens
            longest = _log_int(rng, 1, 65536)
            seqs = _log_int(rng, 1, max(1, min(256, 300000 // longest)))
            max_q = 1
        else:  # chunks: at most 2^29 scores a head of the padded batch
            longest = _log_int(rng, 2, 8192)
            max_q = _log_int(rng, 1, min(longest, 2048))
            seqs = _log_int(rng, 1, max(1, min(32, (1 << 29) // (longest * max_q * heads))))
        c = _attend("", bits, seqs, max(1, max_q // 16), max_q, max(max_q, longest // 4), longest,
                    heads, kv_heads, head_dim, window, sink, shape, block_size)
    del c["name"]
    return c


def _lengths(case):
    """Context and query lengths of the case's requests (int64 arrays)."""
    r = np.random.RandomState(case["shape"])
    n = case["seqs"]
    lens = r.randint(case["min_len"], case["max_len"] + 1, n).astype(np.int64)
    lens[r.randint(n)] = case["max_len"]
    q = r.randint(case["min_q"], case["max_q"] + 1, n).astype(np.int64)
    if case["max_q"] > 1 and n > 3:  # a mixed step: every third request is a single token
        q[::3] = 1
    q[r.randint(n)] = case["max_q"]
    return np.maximum(lens, q), q


def _hidden(case, lens, q):
    """First key behind the sinks that some query sees, of each request."""
    if not case["window"]:
        return np.zeros_like(lens)
    return np.maximum(0, lens - q - case["window"] + 1)


def work(case):
    h, hkv, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "norm":
        t = case["tokens"]
        return {"bytes": t * ((h + 2 * hkv) * d * 2 * 2 + 8) + case["rotary_dim"] * 4 + 4 * d,
                "flops": t * (h + hkv) * (4 * d + 3 * case["rotary_dim"])}
    lens, q = _lengths(case)
    bs, tokens = case["block_size"], int(q.sum())
    if case["op"] == "append":
        blocks = int((-(-lens // bs) - (lens - q) // bs).sum())
        moved = tokens * 2 * hkv * d * 3 + blocks * (2 * hkv * 4 + 4)
        if not case["rotary_dim"]:
            return {"bytes": moved, "flops": tokens * 2 * hkv * d * 2}
        return {"bytes": moved + tokens * (h * d * 4 + 4) + case["rotary_dim"] * 4 + 4 * d,
                "flops": tokens * ((h + hkv) * (4 * d + 3 * case["rotary_dim"]) + 4 * hkv * d)}
    low = _hidden(case, lens, q)
    keys = int((lens - low + np.minimum(low, case["sink"])).sum())
    pairs = 0
    for L, n in zip(lens.tolist(), q.tolist()):
        seen = np.arange(L - n, L) + 1
        if case["window"]:
            seen = np.minimum(seen, case["window"] + np.clip(seen - case["window"], 0, case["sink"]))
        pairs += int(seen.sum())
    size = case["bits"] // 8
    return {"bytes": keys * hkv * d * 2 * size + (keys // bs * hkv * 8 if size == 1 else 0)
            + tokens * h * (2 * d * 2 + 4),
            "flops": pairs * h * 4 * d}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def _normal(shape, g, std=1.0):
    return torch.randn(shape, device=DEVICE, generator=g, dtype=torch.bfloat16).mul_(std)


def _frequencies(rotary_dim):
    return 500000.0 ** (-np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim)


def _gains(head_dim, g):
    """Weights of the query and key norms: around one, as trained ones are."""
    w = torch.rand((2, head_dim), device=DEVICE, generator=g).mul_(0.6).add_(1.0)
    return w[0].to(torch.bfloat16), w[1].to(torch.bfloat16)


def _table(lens, low, sink, block_size, r):
    """Shuffled block tables; -1 behind a request's blocks and where every key
    of a block is hidden. Also the number of blocks in use."""
    n = -(-lens // block_size)
    b = np.arange(max(1, int(n.max())))[None, :] * block_size
    used = (b < lens[:, None]) & ((b < sink) | (b + block_size > low[:, None]))
    table = np.full(used.shape, -1, dtype=np.int32)
    table[used] = r.permutation(int(used.sum())).astype(np.int32)
    return table, int(used.sum())


def _pool8(blocks, block_size, kv_heads, head_dim, g):
    """An 8-bit pool and its scales, as an earlier step left them."""
    x = torch.randn((2, blocks, block_size, kv_heads, head_dim), device=DEVICE, generator=g,
                    dtype=torch.bfloat16)
    x = x.mul_(96.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    s = torch.randn((2, blocks, kv_heads), device=DEVICE, generator=g).mul_(0.3).exp_()
    return x, s.mul_(1.0 / 96.0)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    return {"norm": _prepare_norm, "append": _prepare_append,
            "attend": _prepare_attend}[case["op"]](case, g, r)


def _projected(case, tokens, g):
    """The projection's output: a token's query, key and value heads in one row."""
    h, hkv, d = case["heads"], case["kv_heads"], case["head_dim"]
    qkv = _normal((tokens, (h + 2 * hkv) * d), g)
    return {"q": qkv[:, :h * d].view(tokens, h, d),
            "k": qkv[:, h * d:(h + hkv) * d].view(tokens, hkv, d),
            "v": qkv[:, (h + hkv) * d:].view(tokens, hkv, d)}


def _prepare_norm(case, g, r):
    t, bs = case["tokens"], case["block_size"]
    nb = -(-t * 5 // (4 * bs)) + 1
    s = _projected(case, t, g)
    q_weight, k_weight = _gains(case["head_dim"], g)
    return {"case": case, **s, "q_weight": q_weight, "k_weight": k_weight,
            "pool": _normal((2, nb, bs, case["kv_heads"], case["head_dim"]), g),
            "positions": _dev(r.randint(0, case["max_pos"], t).astype(np.int32)),
            "slots": _dev(r.permutation(nb * bs)[:t].astype(np.int32)),
            "inv_freq": _dev(_frequencies(case["rotary_dim"]))}


def _prepare_append(case, g, r):
    lens, q = _lengths(case)
    hkv, d, bs = case["kv_heads"], case["head_dim"], case["block_size"]
    cu = np.concatenate([[0], np.cumsum(q)])
    t = int(cu[-1])
    s = _projected(case, t, g)
    q_weight, k_weight = _gains(d, g)
    table, used = _table(lens, np.zeros_like(lens), 0, bs, r)
    pool, scales = _pool8(used + 2, bs, hkv, d, g)
    # scales as the library's own writes leave them: powers of two
    scales = torch.exp2(torch.floor(torch.log2(scales)))
    # a context's tokens sit at their own positions
    where = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, q)])
    return {"case": case, **s, "q_weight": q_weight, "k_weight": k_weight, "pool": pool,
            "scales": scales, "table": _dev(table), "cu": _dev(cu.astype(np.int32)),
            "lens": _dev(lens.astype(np.int32)), "max_q": int(q.max()),
            "positions": _dev(where.astype(np.int32)),
            "inv_freq": _dev(_frequencies(max(2, case["rotary_dim"])))}


def _prepare_attend(case, g, r):
    lens, q = _lengths(case)
    h, hkv, d, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    cu = np.concatenate([[0], np.cumsum(q)])
    table, used = _table(lens, _hidden(case, lens, q), case["sink"], bs, r)
    s = {"case": case, "table": _dev(table), "cu": _dev(cu.astype(np.int32)),
         "lens": _dev(lens.astype(np.int32)), "max_q": int(q.max()), "max_len": int(lens.max()),
         # logits of a standard deviation of about two: a few keys carry most of the weight
         "q": _normal((int(cu[-1]), h, d), g, 2.0),
         "lse": torch.empty((int(cu[-1]), h), dtype=torch.float32, device=DEVICE)}
    if case["bits"] == 8:
        s["pool"], s["scales"] = _pool8(used + 2, bs, hkv, d, g)
    else:
        s["pool"] = _normal((2, used + 2, bs, hkv, d), g)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "append": _own_append, "attend": _own_attend}[op](state)
    return {"norm": _plain_norm, "append": _plain_append, "attend": _plain_attend}[op](state)


def _own_norm(s):
    import paged_kv_cache_varlen_gb300 as pkv

    q_out = pkv.qk_norm_rope_kv_cache_write(
        s["q"], s["pool"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
        s["q_weight"], s["k_weight"], eps=EPS, interleaved=s["case"]["interleaved"])
    return {"q": q_out, "pool": s["pool"]}


def _own_append(s):
    import paged_kv_cache_varlen_gb300 as pkv

    if not s["case"]["rotary_dim"]:
        pkv.kv_cache_append_fp8(s["pool"], s["scales"], s["k"], s["v"], s["table"], s["cu"],
                                s["lens"], s["max_q"])
        return {"pool": s["pool"], "scales": s["scales"]}
    q_out = pkv.qk_norm_rope_kv_cache_append_fp8(
        s["q"], s["pool"], s["scales"], s["k"], s["v"], s["positions"], s["table"], s["cu"],
        s["lens"], s["max_q"], s["inv_freq"], s["q_weight"], s["k_weight"], eps=EPS)
    return {"q": q_out, "pool": s["pool"], "scales": s["scales"]}


def _own_attend(s):
    import paged_kv_cache_varlen_gb300 as pkv

    c = s["case"]
    if c["bits"] == 8:
        out, lse = pkv.paged_attention_varlen_fp8(
            s["q"], s["pool"], s["scales"], s["table"], s["cu"], s["lens"], s["max_q"],
            s["max_len"], window=c["window"], num_sink=c["sink"], out_lse=s["lse"])
    else:
        out, lse = pkv.paged_attention_varlen_window(
            s["q"], s["pool"], s["table"], s["cu"], s["lens"], s["max_q"], s["max_len"],
            c["window"], num_sink=c["sink"], out_lse=s["lse"])
    return {"out": out, "lse": lse}


def _plain_turn(x, weight, s, interleaved):
    """x [T,N,D] normed over each head and rotated, in 32 bits."""
    rot = s["case"]["rotary_dim"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_norm(s):
    c = s["case"]
    slots = s["slots"].long()
    pool = s["pool"].view(2, -1, c["kv_heads"], c["head_dim"])
    pool[0][slots] = _plain_turn(s["k"], s["k_weight"], s, c["interleaved"]).to(torch.bfloat16)
    pool[1][slots] = s["v"]
    q = _plain_turn(s["q"], s["q_weight"], s, c["interleaved"]).to(torch.bfloat16)
    return {"q": q, "pool": s["pool"]}


def _plain_append(s):
    c = s["case"]
    bs, hkv, d = c["block_size"], c["kv_heads"], c["head_dim"]
    k = _plain_turn(s["k"], s["k_weight"], s, False) if c["rotary_dim"] else s["k"].float()
    kv = torch.stack([k, s["v"].float()])
    lens, cu = s["lens"].long(), s["cu"].long()
    t = torch.arange(kv.shape[1], device=DEVICE)
    req = torch.searchsorted(cu, t, right=True) - 1
    start = (lens - (cu[1:] - cu[:-1]))[req]  # tokens that were there before
    pos = start + t - cu[req]
    block = s["table"].long()[req, pos // bs]
    # a block's scale: a power of two that its largest magnitude fits under;
    # a block that held tokens before keeps its own where that is larger
    nb = s["scales"].shape[1]
    most = torch.zeros((2, nb, hkv), device=DEVICE)
    most.index_reduce_(1, block, kv.abs().amax(-1), "amax")
    mantissa, exponent = torch.frexp(most / 448.0)
    need = torch.ldexp(torch.ones_like(most), exponent - (mantissa == 0.5).to(torch.int32))
    need = torch.where(most > 0, need, 0.0).clamp(min=2.0 ** -100)
    first = torch.full((nb,), 1 << 30, device=DEVICE)
    first.index_reduce_(0, block, pos, "amin")
    touched = first < 1 << 30
    before = torch.zeros_like(first).index_copy_(0, block, start) - first // bs * bs
    held = torch.where(touched, before.clamp(min=0), bs)  # rows of the block that stay
    old = s["scales"]
    new = torch.where((held == 0)[None, :, None], need, torch.maximum(old, need))
    new = torch.where(touched[None, :, None], new, old)
    pool = s["pool"].view(torch.uint8)
    again = (s["pool"].float() * (old / new)[:, :, None, :, None]).to(torch.float8_e4m3fn)
    stays = torch.arange(bs, device=DEVICE)[None, :] < held[:, None]
    pool.copy_(torch.where(stays[None, :, :, None, None], again.view(torch.uint8), pool))
    eight = (kv / new[:, block][..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    pool.view(2, -1, hkv, d)[:, block * bs + pos % bs] = eight.view(torch.uint8)
    old.copy_(new)
    if not c["rotary_dim"]:
        return {"pool": s["pool"], "scales": old}
    q = _plain_turn(s["q"], s["q_weight"], s, False).to(torch.bfloat16)
    return {"q": q, "pool": s["pool"], "scales": old}


def _plain_attend(s):
    c = s["case"]
    h, hkv, d = c["heads"], c["kv_heads"], c["head_dim"]
    n, m, grp = s["lens"].shape[0], s["max_q"], h // hkv
    lens, cu = s["lens"].long(), s["cu"].long()
    ql = cu[1:] - cu[:-1]
    table = s["table"].long().clamp(min=0)

    def rows(half):
        x = s["pool"][half]
        if c["bits"] == 8:
            x = x.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
            x *= s["scales"][half][table][:, :, None, :, None]
        else:
            x = x[table].float()
        return x.reshape(n, -1, hkv, d)[:, :s["max_len"]].transpose(1, 2)

    j = torch.arange(m, device=DEVICE)
    at = (cu[:-1, None] + j[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].view(n, m, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, m * grp, d)
    p = torch.matmul(q.float(), rows(0).transpose(2, 3)).view(n, hkv, m, grp, -1)
    p.mul_(1.0 / math.sqrt(d))
    key = torch.arange(p.shape[-1], device=DEVICE)[None, None, :]
    pos = ((lens - ql)[:, None] + j[None, :])[:, :, None]
    seen = key <= pos
    if c["window"]:
        seen = seen & ((key > pos - c["window"]) | (key < c["sink"]))
    p.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = p.amax(-1, keepdim=True)
    total = p.sub_(top).exp_().sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hkv, m * grp, -1), rows(1)).view(n, hkv, m, grp, d) / total
    lse = (top + total.log())[..., 0]
    t = torch.arange(s["q"].shape[0], device=DEVICE)
    req = torch.searchsorted(cu, t, right=True) - 1
    o = o[req, :, t - cu[req]].reshape(-1, h, d).to(torch.bfloat16)
    s["lse"].copy_(lse[req, :, t - cu[req]].reshape(-1, h))
    return {"out": o, "lse": s["lse"]}


# --------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    return {"norm": _exact_norm, "append": _exact_append,
            "attend": _exact_attend}[case["op"]](case, prepare(case, seed))


def _exact_heads(x, weight, case, s):
    rot = case["rotary_dim"]
    x = x.double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / case["head_dim"] + EPS).sqrt() * weight.double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE),
                       s["positions"].double()[:, None, None] * s["inv_freq"])
    if case.get("interleaved"):
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], -1, 2).contiguous())
        y = torch.view_as_real(z * turn).flatten(-2)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _exact_norm(case, s):
    pool = s["pool"].double()
    flat = pool.view(2, -1, case["kv_heads"], case["head_dim"])
    flat[0].index_copy_(0, s["slots"].long(), _exact_heads(s["k"], s["k_weight"], case, s))
    flat[1].index_copy_(0, s["slots"].long(), s["v"].double())
    return {"q": _exact_heads(s["q"], s["q_weight"], case, s), "pool": pool}


def _e4m3(x):
    """The nearest multiple of 2^-3 of the value's binade (not below 2^-6), ties to even."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def _exact_append(case, s):
    bs, rot = case["block_size"], case["rotary_dim"]
    k = _exact_heads(s["k"], s["k_weight"], case, s) if rot else s["k"].double()
    new = np.stack([k.cpu().numpy(), s["v"].double().cpu().numpy()])
    pool, scales = s["pool"].double().cpu().numpy(), s["scales"].double().cpu().numpy()
    table, (lens, ql) = s["table"].cpu().numpy(), _lengths(case)
    t = 0
    for i, (L, n) in enumerate(zip(lens.tolist(), ql.tolist())):
        for b in range((L - n) // bs, (L - 1) // bs + 1):
            id_, first = table[i, b], max(0, L - n - b * bs)
            last = min(bs, L - b * bs)
            x = new[:, t:t + last - first]
            t += last - first
            top = np.abs(x).max((1, 3))
            scale = np.exp2(np.ceil(np.log2(np.maximum(top, 448 * 2.0 ** -100) / 448)))
            if first:
                scale = np.maximum(scale, scales[:, id_])
                ratio = (scales[:, id_] / scale)[:, None, :, None]
                pool[:, id_, :first] = _e4m3(pool[:, id_, :first] * ratio)
            scales[:, id_] = scale
            pool[:, id_, first:last] = _e4m3(x / scale[:, None, :, None])
    out = {"pool": torch.from_numpy(pool), "scales": torch.from_numpy(scales)}
    if rot:
        out["q"] = _exact_heads(s["q"], s["q_weight"], case, s)
    return out


def _exact_attend(case, s):
    lens, ql = _lengths(case)
    h, hkv, d, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    grp = h // hkv
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEVICE)
    start = 0
    for i, (L, n) in enumerate(zip(lens.tolist(), ql.tolist())):
        low = max(0, L - n - case["window"] + 1) if case["window"] else 0
        keys = torch.cat([torch.arange(min(low, case["sink"])), torch.arange(low, L)]).to(DEVICE)
        ids = s["table"][i, keys // bs].long()
        kv = s["pool"].view(torch.uint8 if case["bits"] == 8 else torch.bfloat16)
        kv = kv[:, ids, keys % bs]
        if case["bits"] == 8:
            kv = kv.view(torch.float8_e4m3fn).double() * s["scales"][:, ids].double()[..., None]
        for head in range(hkv):
            k, v = kv[0, :, head].double(), kv[1, :, head].double()
            for j in range(0, n, 512):
                e = min(n, j + 512)
                at = torch.arange(L - n + j, L - n + e, device=DEVICE)[:, None]
                hidden = keys[None, :] > at
                if case["window"]:
                    hidden |= (at - keys[None, :] >= case["window"]) & (keys >= case["sink"])[None, :]
                for a in range(head * grp, (head + 1) * grp):
                    x = (s["q"][start + j:start + e, a].double() @ k.T) / math.sqrt(d)
                    x = x.masked_fill(hidden, -math.inf)
                    lse[start + j:start + e, a] = x.logsumexp(-1)
                    out[start + j:start + e, a] = x.softmax(-1) @ v
        start += n
    return {"out": out, "lse": lse}
