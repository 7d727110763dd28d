"""Measured cases of the cache-budget operators: rotary positions written into
the paged cache, accumulated attention weights of the cached keys, and the
eviction of the keys that carry the least of it.

The operators serve one flow. A step rotates its queries and keys and writes
the keys and values into the paged pool (``rope_kv_cache_write``); after the
attention call, the weight that each cached key received is added to a running
sum (``attention_key_weights``); when a request outgrows its budget, the
heaviest keys are selected per KV head (``evict_select``) and their rows are
moved to fresh blocks (``evict_compact``).

``own`` chooses between the plain torch forms below and the library's calls.
Ragged lengths follow from the case alone (``shape`` seeds them), so that
``work`` can count them; every value follows from the seed.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _rope(name, tokens, heads, kv_heads, head_dim, rotary_dim, interleaved, max_pos, stretch,
          block_size=16):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rotary_dim": rotary_dim, "interleaved": interleaved,
            "max_pos": max_pos, "stretch": stretch, "block_size": block_size}


def _weights(name, seqs, min_q, max_q, min_len, max_len, heads, kv_heads, head_dim, decay, shape,
             block_size=16):
    return {"name": name, "op": "weights", "seqs": seqs, "min_q": min_q, "max_q": max_q,
            "min_len": min_len, "max_len": max_len, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "decay": decay, "shape": shape, "block_size": block_size}


def _select(name, seqs, min_len, max_len, kv_heads, keep, sink, recent, shape):
    return {"name": name, "op": "select", "seqs": seqs, "min_len": min_len, "max_len": max_len,
            "kv_heads": kv_heads, "keep": keep, "sink": sink, "recent": recent, "shape": shape}


def _compact(name, seqs, min_len, max_len, kv_heads, head_dim, keep, shape, block_size=16):
    return {"name": name, "op": "compact", "seqs": seqs, "min_len": min_len, "max_len": max_len,
            "kv_heads": kv_heads, "head_dim": head_dim, "keep": keep, "shape": shape,
            "block_size": block_size}


def listed():
    return [
        # one request's next token, far into a context: the smallest call, all latency
        _rope("rope_step_1", 1, 32, 8, 128, 128, False, 131072, 1.0),
        # the decode step of a batch of 64 requests (the benchmark's decode shape)
        _rope("rope_step_64", 64, 32, 8, 128, 128, False, 4096, 1.0),
        # an odd-sized chunk, adjacent pairs, three quarters of a 64-wide head rotated
        _rope("rope_part_1021", 1021, 16, 2, 64, 48, True, 8192, 1.0),
        # a long prompt at positions stretched eightfold for a long context
        _rope("rope_prompt_8192", 8192, 32, 8, 128, 128, False, 131072, 8.0),
        # the decode step of 64 requests, contexts of 512 to 4096 tokens
        _weights("weights_step_64", 64, 1, 1, 512, 4096, 32, 8, 128, 1.0, 1),
        # a mixed step of a smaller model: single tokens beside odd-sized chunks
        _weights("weights_mixed_13", 13, 1, 700, 700, 5000, 16, 4, 64, 0.97, 2),
        # decodes over contexts of 32K to 128K tokens: the most bytes
        _weights("weights_step_long", 8, 1, 1, 32768, 131072, 32, 8, 128, 1.0, 3),
        # one whole prompt: the most arithmetic
        _weights("weights_prompt_8192", 1, 8192, 8192, 8192, 8192, 32, 8, 128, 1.0, 4),
        # a batch cut back to a budget of 1024 keys a head
        _select("select_64", 64, 1500, 8192, 8, 1024, 4, 128, 5),
        # two very long contexts: few rows, each of them long
        _select("select_long", 2, 100000, 131072, 8, 8192, 16, 1024, 6),
        # one short request of a small model
        _compact("compact_1", 1, 777, 777, 2, 64, 200, 7),
        # the batch of select_64's kind, its kept rows moved to fresh blocks
        _compact("compact_64", 64, 1500, 4096, 8, 128, 1024, 8),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


_HEADS = [(32, 8), (32, 8), (16, 4), (16, 2), (8, 8), (12, 2), (40, 8), (28, 4), (8, 1), (64, 8)]


def draw(rng):
    op = rng.choice(["rope", "weights", "weights", "select", "compact"])
    heads, kv_heads = rng.choice(_HEADS)
    head_dim = rng.choice([64, 128])
    block_size = rng.choice([16, 16, 32, 64])
    shape = rng.randrange(1 << 20)
    if op == "rope":
        rotary_dim = rng.choice([head_dim, head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)])
        c = _rope("", _log_int(rng, 1, 4096), heads, kv_heads, head_dim, rotary_dim,
                  rng.random() < 0.5, _log_int(rng, 2, 1 << 20), rng.choice([1.0, 4.0, 8.0]),
                  block_size)
    elif op == "weights" and rng.random() < 0.5:  # single tokens
        longest = _log_int(rng, 1, 131072)
        seqs = _log_int(rng, 1, max(1, min(256, 500000 // longest)))
        c = _weights("", seqs, 1, 1, max(1, longest // 8), longest, heads, kv_heads, head_dim,
                     rng.choice([1.0, 0.95]), shape, block_size)
    elif op == "weights":  # chunks: at most 2^28 scores a head group of the padded batch
        longest = _log_int(rng, 2, 16384)
        max_q = _log_int(rng, 1, min(longest, 4096))
        seqs = _log_int(rng, 1, max(1, min(32, (1 << 29) // (longest * max_q * heads))))
        c = _weights("", seqs, max(1, max_q // 16), max_q, max(max_q, longest // 4), longest,
                     heads, kv_heads, head_dim, rng.choice([1.0, 0.95]), shape, block_size)
    elif op == "select":
        longest = _log_int(rng, 8, 131072)
        seqs = _log_int(rng, 1, max(1, min(256, 500000 // longest)))
        keep = _log_int(rng, 1, longest)
        c = _select("", seqs, max(1, longest // 6), longest, kv_heads, keep,
                    rng.randint(0, 8), rng.randint(0, keep), shape)
    else:
        longest = _log_int(rng, 2, 32768)
        seqs = _log_int(rng, 1, max(1, min(128, 131072 // longest)))
        c = _compact("", seqs, max(1, longest // 4), longest, kv_heads, head_dim,
                     _log_int(rng, 1, longest), shape, block_size)
    del c["name"]
    return c


def _lengths(case):
    """Context and query lengths of the case's requests (int64 arrays)."""
    r = np.random.RandomState(case["shape"])
    n = case["seqs"]
    lens = r.randint(case["min_len"], case["max_len"] + 1, n).astype(np.int64)
    lens[r.randint(n)] = case["max_len"]
    if case["op"] != "weights":
        return lens, np.ones(n, dtype=np.int64)
    q = r.randint(case["min_q"], case["max_q"] + 1, n).astype(np.int64)
    if case["max_q"] > 1 and n > 3:  # a mixed step: every third request is a single token
        q[::3] = 1
    q[r.randint(n)] = case["max_q"]
    return np.maximum(lens, q), q


def _visible(lens, q):
    """(query, key) pairs that the causal mask leaves."""
    return int(np.sum(q * (lens - q) + q * (q + 1) // 2))


def work(case):
    if case["op"] == "rope":
        t, d = case["tokens"], case["head_dim"]
        h, hkv = case["heads"], case["kv_heads"]
        return {"bytes": t * ((h + 2 * hkv) * d * 2 * 2 + 8) + case["rotary_dim"] * 4,
                "flops": 3 * t * (h + hkv) * case["rotary_dim"]}
    lens, q = _lengths(case)
    hkv = case["kv_heads"]
    if case["op"] == "weights":
        d, h = case["head_dim"], case["heads"]
        keys, queries = int(lens.sum()), int(q.sum())
        return {"bytes": keys * hkv * (2 * d + 4) + (keys - queries) * hkv * 4
                + queries * h * (2 * d + 4),
                "flops": _visible(lens, q) * h * (2 * d + 4)}
    keep = int(np.minimum(lens, case["keep"]).sum())
    if case["op"] == "select":
        return {"bytes": int(lens.sum()) * hkv * 4 + keep * hkv * 8,
                "flops": int(lens.sum()) * hkv}
    return {"bytes": keep * hkv * (4 + 2 * 2 * 2 * case["head_dim"]), "flops": 0}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _frequencies(rotary_dim, stretch):
    """Angle per position of each rotated pair, in radians: base 500000; for a
    stretched context the slow pairs turn `stretch` times slower."""
    f = 500000.0 ** (-np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim)
    if stretch > 1.0:
        turns = 8192.0 * f / (2.0 * math.pi)
        ramp = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = f * (ramp + (1.0 - ramp) / stretch)
    return f


def _tables(lens, block_size, r, first=0):
    """Shuffled block tables of the requests, -1 behind each request's blocks."""
    n = -(-lens // block_size)
    ids = (first + r.permutation(int(n.sum()))).astype(np.int32)
    table = np.full((len(lens), max(1, int(n.max()))), -1, dtype=np.int32)
    table[np.arange(table.shape[1])[None, :] < n[:, None]] = ids
    return table


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    return {"rope": _prepare_rope, "weights": _prepare_weights, "select": _prepare_select,
            "compact": _prepare_compact}[case["op"]](case, g, r)


def _normal(shape, g, std=1.0):
    return torch.randn(shape, device=DEVICE, generator=g, dtype=torch.bfloat16).mul_(std)


def _prepare_rope(case, g, r):
    t, h, hkv, d = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
    bs = case["block_size"]
    nb = -(-t * 5 // (4 * bs)) + 1
    # the projection's output: a token's query, key and value heads in one row
    qkv = _normal((t, (h + 2 * hkv) * d), g)
    return {"case": case,
            "q": qkv[:, :h * d].view(t, h, d), "k": qkv[:, h * d:(h + hkv) * d].view(t, hkv, d),
            "v": qkv[:, (h + hkv) * d:].view(t, hkv, d),
            "pool": _normal((2, nb, bs, hkv, d), g),
            "positions": _dev(r.randint(0, case["max_pos"], t).astype(np.int32)),
            "slots": _dev(r.permutation(nb * bs)[:t].astype(np.int32)),
            "inv_freq": _dev(_frequencies(case["rotary_dim"], case["stretch"])),
            "factor": 0.1 * math.log(case["stretch"]) + 1.0}


def _prepare_weights(case, g, r):
    lens, q = _lengths(case)
    h, hkv, d, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    grp, n, scale = h // hkv, len(lens), 1.0 / math.sqrt(case["head_dim"])
    cu = np.concatenate([[0], np.cumsum(q)])
    table = _tables(lens, bs, r)
    nb = int((table >= 0).sum()) + 2
    pool = _normal((2, nb, bs, hkv, d), g)
    # logits of a standard deviation of about two: a few keys carry most of the weight
    qs = _normal((int(cu[-1]), h, d), g, 2.0)
    ids = _dev(table)
    lse = torch.empty((int(cu[-1]), h), dtype=torch.float32, device=DEVICE)
    for i in range(n):  # the log-sum-exp that the attention call returned
        L, ql = int(lens[i]), int(q[i])
        k = pool[0][ids[i, :-(-L // bs)].long()].reshape(-1, hkv, d)[:L].float().permute(1, 2, 0)
        for j in range(0, ql, 1024):
            m = min(1024, ql - j)
            rows = qs[cu[i] + j:cu[i] + j + m].float().view(m, hkv, grp, d).permute(1, 0, 2, 3)
            s = torch.matmul(rows.reshape(hkv, m * grp, d), k).view(hkv, m, grp, L).mul_(scale)
            if ql > 1:
                pos = torch.arange(L - ql + j, L - ql + j + m, device=DEVICE)
                s.masked_fill_(torch.arange(L, device=DEVICE)[None, None, None, :]
                               > pos[None, :, None, None], -math.inf)
            lse[cu[i] + j:cu[i] + j + m] = torch.logsumexp(s, -1).permute(1, 0, 2).reshape(m, h)
    shape = (n, hkv, case["max_len"])
    return {"case": case, "q": qs, "pool": pool, "lse": lse, "table": ids,
            "cu": _dev(cu.astype(np.int32)), "lens": _dev(lens.astype(np.int32)),
            "max_q": int(q.max()), "max_len": int(lens.max()), "scale": scale,
            "rows": _dev(r.permutation(n).astype(np.int32)),
            "weights": torch.rand(shape, device=DEVICE, generator=g),
            "out": torch.zeros(shape, device=DEVICE)}


def _prepare_select(case, g, r):
    lens, _ = _lengths(case)
    n, hkv, m = len(lens), case["kv_heads"], case["max_len"]
    # accumulated weights: a long tail, and keys that never received any (ties)
    w = torch.randn((n, hkv, m), device=DEVICE, generator=g).mul_(2.0).exp_()
    w[torch.rand((n, hkv, m), device=DEVICE, generator=g) < 0.05] = 0.0
    return {"case": case, "weights": w, "lens": _dev(lens.astype(np.int32)),
            "keep": _dev(np.minimum(lens, case["keep"]).astype(np.int32)),
            "max_len": int(lens.max()), "max_keep": int(min(lens.max(), case["keep"])),
            "rows": _dev(r.permutation(n).astype(np.int32)),
            "kept": torch.full((n, hkv, int(min(lens.max(), case["keep"]))), -1,
                               dtype=torch.int32, device=DEVICE),
            "out": torch.zeros((n, hkv, m), device=DEVICE)}


def _prepare_compact(case, g, r):
    lens, _ = _lengths(case)
    keep = np.minimum(lens, case["keep"])
    n, hkv, d, bs = len(lens), case["kv_heads"], case["head_dim"], case["block_size"]
    src = _tables(lens, bs, r)
    used = int((src >= 0).sum())
    dst = _tables(keep, bs, r, first=used)
    nb = used + int((dst >= 0).sum())
    # a head's kept keys: a random subset of its context, in order
    m = int(keep.max())
    at = torch.rand((n, hkv, int(lens.max())), device=DEVICE, generator=g)
    idx = torch.arange(at.shape[2], device=DEVICE)
    at = torch.where(idx[None, None, :] < _dev(lens)[:, None, None], at, 2.0)
    order = at.argsort(-1)[:, :, :m]
    order = torch.where(idx[None, None, :m] < _dev(keep)[:, None, None], order, 1 << 30)
    kept = order.sort(-1).values.to(torch.int32)
    return {"case": case, "pool": _normal((2, nb, bs, hkv, d), g), "src": _dev(src),
            "dst": _dev(dst), "kept": kept, "keep": _dev(keep.astype(np.int32))}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "weights": _own_weights, "select": _own_select,
                "compact": _own_compact}[op](state)
    return {"rope": _plain_rope, "weights": _plain_weights, "select": _plain_select,
            "compact": _plain_compact}[op](state)


def _own_rope(s):
    import paged_kv_cache_varlen_gb300 as pkv

    q_out = pkv.rope_kv_cache_write(s["q"], s["pool"], s["k"], s["v"], s["positions"], s["slots"],
                                    s["inv_freq"], interleaved=s["case"]["interleaved"],
                                    factor=s["factor"])
    return {"q": q_out, "pool": s["pool"]}


def _own_weights(s):
    import paged_kv_cache_varlen_gb300 as pkv

    out = pkv.attention_key_weights(s["q"], s["pool"], s["lse"], s["table"], s["cu"], s["lens"],
                                    s["max_q"], s["max_len"], s["weights"], out=s["out"],
                                    weight_rows=s["rows"], decay=s["case"]["decay"],
                                    scale=s["scale"])
    return {"weights": out}


def _own_select(s):
    import paged_kv_cache_varlen_gb300 as pkv

    kept, out = pkv.evict_select(s["weights"], s["lens"], s["keep"], s["max_len"], s["max_keep"],
                                 num_sink=s["case"]["sink"], num_recent=s["case"]["recent"],
                                 weight_rows=s["rows"], kept=s["kept"], weights_out=s["out"])
    return {"kept": kept, "weights": out}


def _own_compact(s):
    import paged_kv_cache_varlen_gb300 as pkv

    pkv.evict_compact(s["pool"], s["src"], s["dst"], s["kept"], s["keep"])
    return {"pool": s["pool"]}


def _plain_rope(s):
    c, q, k = s["case"], s["q"], s["k"]
    rot = c["rotary_dim"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos = (angle.cos() * s["factor"]).float()[:, None, :]
    sin = (angle.sin() * s["factor"]).float()[:, None, :]

    def turn(x):
        y = x.float()
        if c["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return y.to(x.dtype)

    slots = s["slots"].long()
    pool = s["pool"].view(2, -1, c["kv_heads"], c["head_dim"])
    pool[0][slots] = turn(k)
    pool[1][slots] = s["v"]
    return {"q": turn(q), "pool": s["pool"]}


def _plain_weights(s):
    c = s["case"]
    h, hkv, d = c["heads"], c["kv_heads"], c["head_dim"]
    n, m, grp = s["lens"].shape[0], s["max_q"], h // hkv
    lens, cu = s["lens"].long(), s["cu"].long()
    ql = cu[1:] - cu[:-1]
    k = s["pool"][0][s["table"].long().clamp(min=0)].reshape(n, -1, hkv, d)[:, :s["max_len"]]
    j = torch.arange(m, device=DEVICE)
    at = (cu[:-1, None] + j[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].view(n, m, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, m * grp, d)
    lse = s["lse"][at].view(n, m, hkv, grp).permute(0, 2, 1, 3)
    p = torch.matmul(q.float(), k.float().permute(0, 2, 3, 1)).view(n, hkv, m, grp, -1)
    p = p.mul_(s["scale"]).sub_(lse[..., None]).exp_()
    key = torch.arange(p.shape[-1], device=DEVICE)
    seen = ((key[None, None, :] <= (lens - ql)[:, None, None] + j[None, :, None])
            & (j[None, :, None] < ql[:, None, None]))
    total = p.masked_fill_(~seen[:, None, :, None, :], 0.0).sum((2, 3))
    rows = s["rows"].long()
    old = s["weights"][rows][..., :p.shape[-1]]
    new = torch.where(key < (lens - ql)[:, None, None], c["decay"] * old, 0.0) + total
    out = s["out"]
    out[rows, :, :p.shape[-1]] = torch.where(key < lens[:, None, None], new,
                                             out[rows, :, :p.shape[-1]])
    return {"weights": out}


def _plain_select(s):
    c = s["case"]
    lens, keep, rows = s["lens"].long(), s["keep"].long(), s["rows"].long()
    w = s["weights"][rows][..., :s["max_len"]]
    i = torch.arange(w.shape[-1], device=DEVICE)
    L, n = lens[:, None, None], keep[:, None, None]
    recent = n.clamp(max=c["recent"])
    sink = (n - recent).clamp(max=c["sink"])
    order = torch.where(i >= L - recent, math.inf, w)
    order = torch.where(i < sink, math.inf, order)
    order = torch.where(i >= L, -math.inf, order)
    first = order.sort(dim=-1, descending=True, stable=True).indices  # ties: lowest index first
    rank = torch.empty_like(first).scatter_(-1, first, i.expand_as(first).contiguous())
    picked = torch.where(rank < n, i, w.shape[-1]).sort(-1).values[..., :s["max_keep"]]
    j = torch.arange(s["max_keep"], device=DEVICE)
    s["kept"].copy_(torch.where(j < n, picked.to(torch.int32), s["kept"]))
    values = w.gather(-1, picked.clamp(max=w.shape[-1] - 1))
    out = s["out"]
    out[rows, :, :s["max_keep"]] = torch.where(j < n, values, out[rows, :, :s["max_keep"]])
    return {"kept": s["kept"], "weights": out}


def _plain_compact(s):
    c, bs = s["case"], s["case"]["block_size"]
    n, hkv, m = s["kept"].shape
    # behind a request's last kept key the last one is copied again
    j = torch.minimum(torch.arange(m, device=DEVICE)[None, :], s["keep"].long()[:, None] - 1)
    kept = s["kept"].long().gather(-1, j[:, None, :].expand(n, hkv, m))
    req = torch.arange(n, device=DEVICE)[:, None, None]
    from_ = s["src"].long()[req, kept // bs] * bs + kept % bs
    to = (s["dst"].long()[req, j[:, None, :] // bs] * bs + j[:, None, :] % bs).expand(n, hkv, m)
    head = torch.arange(hkv, device=DEVICE)[None, :, None]
    pool = s["pool"].view(2, -1, hkv, c["head_dim"])
    pool[:, to, head] = pool[:, from_, head]
    return {"pool": s["pool"]}


# --------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    return {"rope": _exact_rope, "weights": _exact_weights, "select": _exact_select,
            "compact": _exact_compact}[case["op"]](case, prepare(case, seed))


def _exact_rope(case, s):
    rot = case["rotary_dim"]
    turn = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device=DEVICE),
                       s["positions"].double()[:, None, None] * s["inv_freq"])

    def rotated(x):
        x = x.double()
        if case["interleaved"]:
            z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], -1, 2).contiguous())
            y = torch.view_as_real(z * turn).flatten(-2)
        else:
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous())
            z = z * turn
            y = torch.cat([z.real, z.imag], -1)
        return torch.cat([y, x[..., rot:]], -1)

    pool = s["pool"].double()
    flat = pool.view(2, -1, case["kv_heads"], case["head_dim"])
    flat[0].index_copy_(0, s["slots"].long(), rotated(s["k"]))
    flat[1].index_copy_(0, s["slots"].long(), s["v"].double())
    return {"q": rotated(s["q"]), "pool": pool}


def _exact_weights(case, s):
    lens, ql = _lengths(case)
    if _visible(lens, ql) * case["heads"] * case["head_dim"] > 2 ** 39:
        return None  # 64-bit products of this many pairs take too long
    h, hkv, d, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    out, rows = s["out"].double(), s["rows"].tolist()
    start = 0
    for i, (L, n) in enumerate(zip(lens.tolist(), ql.tolist())):
        blocks = s["table"][i, :(L + bs - 1) // bs].long()
        keys = s["pool"][0].index_select(0, blocks).flatten(0, 1)[:L].double()
        for head in range(hkv):
            total = s["weights"][rows[i], head, :L].double() * case["decay"]
            total[L - n:] = 0.0
            kt = keys[:, head].T.contiguous()
            for j in range(0, n, 512):
                e = min(n, j + 512)
                last = torch.arange(L - n + j, L - n + e, device=DEVICE)[:, None]
                hidden = torch.arange(L, device=DEVICE)[None, :] > last
                for a in range(head * (h // hkv), (head + 1) * (h // hkv)):
                    x = s["q"][start + j:start + e, a].double() @ kt * s["scale"]
                    x = (x - s["lse"][start + j:start + e, a, None].double()).exp()
                    total += x.masked_fill(hidden, 0.0).sum(0)
            out[rows[i], head, :L] = total
        start += n
    return {"weights": out}


def _exact_select(case, s):
    kept, out = s["kept"].cpu().numpy().copy(), s["out"].double().cpu().numpy()
    w, lens = s["weights"].double().cpu().numpy(), s["lens"].tolist()
    rows, keep = s["rows"].tolist(), s["keep"].tolist()
    for i, (L, n) in enumerate(zip(lens, keep)):
        recent = min(n, case["recent"])
        sink = min(n - recent, case["sink"])
        for head in range(case["kv_heads"]):
            x = w[rows[i], head, :L]
            middle = np.arange(sink, L - recent)
            heavy = middle[np.lexsort((middle, -x[middle]))][:n - sink - recent]
            ids = np.sort(np.concatenate([np.arange(sink), heavy, np.arange(L - recent, L)]))
            kept[i, head, :n] = ids
            out[rows[i], head, :n] = x[ids]
    return {"kept": torch.from_numpy(kept), "weights": torch.from_numpy(out)}


def _exact_compact(case, s):
    bs, keep = case["block_size"], s["keep"].tolist()
    pool = s["pool"].double()
    rows = pool.view(2, -1, case["kv_heads"], case["head_dim"])
    for i, n in enumerate(keep):
        ids = torch.arange(n, device=DEVICE)
        to = s["dst"][i, ids // bs].long() * bs + ids % bs
        for head in range(case["kv_heads"]):
            ids = s["kept"][i, head, :n].long()
            rows[:, to, head] = rows[:, s["src"][i, ids // bs].long() * bs + ids % bs, head]
    return {"pool": pool}
