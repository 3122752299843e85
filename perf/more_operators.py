"""Cases, plain forms and exact values of the operators around shared contexts and bounded caches.

The operators:

* norm and rotation of queries and keys with a position on several axes (time, height, width): pair p of
  a head is turned by position[axis of p] * frequency[p]; forward, and forward with backward;
* attention of a batch whose sequences share a prefix: a query sees every prefix row and, of its own
  sequence's tokens, itself and the `window` before it; for prompts, and for single tokens over caches;
* a cache of slots with accumulated attention weights: the weights that a prompt's queries gave each key,
  one decoding step that adds its own (w <- decay w + sum of the key head's query heads' probabilities),
  and the eviction that keeps `keep` slots: those of the first `sinks` and of the newest `recent`
  tokens, then the ones of most weight (ties: the lower slot). The kept rows at or past slot `keep` fill the
  freed slots below it, both in ascending order; rows at or past `keep` stay as they were.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # queries and keys of one decoding step at far positions of a video: 8 sequences, 16 heads of 128
        # over 4 key heads, time, height and width on a third of the pairs each; a call of microseconds
        {"name": "axes_step", "op": "axes", "batch": 8, "tokens": 1, "heads": 16, "kv_heads": 4, "dim": 128, "rotary": 128,
         "axes": 3, "mixed": False, "interleaved": False, "train": False, "first": 60000},
        # the 8K training shape (4 x 8192 tokens, 12 heads of 64), forward and backward
        {"name": "axes_train_8k", "op": "axes", "batch": 4, "tokens": 8192, "heads": 12, "kv_heads": 12, "dim": 64,
         "rotary": 64, "axes": 3, "mixed": False, "interleaved": False, "train": True, "first": 0},
        # one token for each of four chats behind a short common instruction
        {"name": "prefix_decode_short", "op": "prefix_decode", "batch": 4, "prefix": 1000, "capacity": 256, "len_lo": 1,
         "len_hi": 200, "heads": 12, "kv_heads": 12, "dim": 64, "window": 255},
        # one token for each of 64 sequences that share a document of 32768 tokens
        {"name": "prefix_decode_batch", "op": "prefix_decode", "batch": 64, "prefix": 32768, "capacity": 1024, "len_lo": 1,
         "len_hi": 1000, "heads": 16, "kv_heads": 4, "dim": 128, "window": 1023},
        # 32 short questions to a document of 16384 tokens
        {"name": "prefix_questions", "op": "prefix", "batch": 32, "prefix": 16384, "tokens": 37, "heads": 16, "kv_heads": 4,
         "dim": 128, "window": 36},
        # the last 8192 tokens of a 64K prompt whose first part is there already
        {"name": "prefix_chunk", "op": "prefix", "batch": 1, "prefix": 57344, "tokens": 8192, "heads": 16, "kv_heads": 4,
         "dim": 128, "window": 4095},
        # the weights that the last 64 queries of a 32K prompt give its keys
        {"name": "weights_last", "op": "weights", "batch": 1, "tokens": 32768, "heads": 16, "kv_heads": 4, "dim": 128,
         "window": 32767, "sinks": 0, "first": 32704},
        # and the weights of all queries of two 8K prompts
        {"name": "weights_prompt", "op": "weights", "batch": 2, "tokens": 8192, "heads": 16, "kv_heads": 4, "dim": 128,
         "window": 8191, "sinks": 0, "first": 0},
        # a decoding step (its row appended, attention, weights) of one sequence
        {"name": "scored_one", "op": "scored", "batch": 1, "capacity": 1024, "len_lo": 700, "len_hi": 700, "heads": 12,
         "kv_heads": 12, "dim": 64, "decay": 1.0},
        # and of 64 sequences with caches of 4096 slots
        {"name": "scored_batch", "op": "scored", "batch": 64, "capacity": 4096, "len_lo": 2049, "len_hi": 4096, "heads": 16,
         "kv_heads": 4, "dim": 128, "decay": 0.99},
        # the row that leaves each full cache in every step of 64 sequences
        {"name": "evict_step", "op": "evict", "batch": 64, "capacity": 4104, "len_lo": 4097, "len_hi": 4097, "kv_heads": 4,
         "dim": 128, "keep": 4096, "sinks": 4, "recent": 512},
        # caches of 32 sequences cut to 4096 slots after long prompts
        {"name": "evict_prompt", "op": "evict", "batch": 32, "capacity": 8192, "len_lo": 5001, "len_hi": 8192, "kv_heads": 4,
         "dim": 128, "keep": 4096, "sinks": 4, "recent": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8, 12])
    return kv * rng.choice([1, 1, 2, 4] if kv <= 8 else [1]), kv


def draw(rng):
    op = rng.choice(["axes", "prefix", "prefix_decode", "weights", "scored", "evict"])
    dim = rng.choice([32, 64, 128])
    heads, kv = _heads(rng)
    case = {"op": op, "dim": dim, "kv_heads": kv}
    if op == "axes":
        tokens = _log(rng, 1, 16384)
        case.update(batch=max(1, min(rng.choice([1, 2, 3, 8]), 32768 // tokens)), tokens=tokens, heads=heads,
                    rotary=rng.choice([dim, dim, dim // 2]), axes=rng.randint(1, 4), mixed=rng.random() < 0.4,
                    interleaved=rng.random() < 0.3, train=rng.random() < 0.5, first=_log(rng, 1, 500000))
    elif op == "prefix":
        tokens = _log(rng, 1, 8192)
        case.update(batch=max(1, min(rng.choice([1, 2, 5, 16, 32]), 16384 // tokens)), tokens=tokens, heads=heads,
                    prefix=_log(rng, 1, 32768), window=rng.choice([tokens - 1, _log(rng, 1, 4096) - 1]))
    elif op == "prefix_decode":
        capacity = _log(rng, 1, 4096)
        hi = rng.randint(1, capacity)
        case.update(batch=rng.choice([1, 2, 5, 16, 64]), prefix=_log(rng, 1, 65536), capacity=capacity, heads=heads,
                    len_lo=rng.randint(0, hi), len_hi=hi, window=rng.choice([capacity - 1, _log(rng, 1, 4096) - 1]))
    elif op == "weights":
        tokens = _log(rng, 1, 16384)
        case.update(batch=max(1, min(rng.choice([1, 2, 3]), 16384 // tokens)), tokens=tokens, heads=heads,
                    window=rng.choice([tokens - 1, _log(rng, 1, 4096) - 1]),
                    sinks=rng.choice([0, 1, 4, 16, rng.randrange(129)]),
                    first=rng.choice([0, max(0, tokens - _log(rng, 1, 512)), rng.randrange(tokens)]))
    elif op == "scored":
        capacity = _log(rng, 8, 16384)
        hi = rng.randint(1, capacity)
        case.update(batch=rng.choice([1, 2, 5, 16, 32]), capacity=capacity, len_lo=rng.randint(1, hi), len_hi=hi, heads=heads,
                    decay=rng.choice([1.0, 1.0, round(rng.uniform(0.9, 1.0), 4)]))
    else:
        capacity = _log(rng, 8, 16384)
        hi = rng.randint(1, capacity)
        keep = rng.randint(1, hi)
        sinks = min(keep, rng.choice([0, 1, 4, 16]))
        case.update(batch=rng.choice([1, 2, 5, 16, 32]), capacity=capacity, len_lo=rng.randint(0, hi), len_hi=hi, keep=keep,
                    sinks=sinks, recent=rng.randint(0, keep - sinks))
    return case


def _lengths(case):
    """Slots of each sequence, spread over [len_lo, len_hi]."""
    b, lo, hi = case["batch"], case["len_lo"], case["len_hi"]
    return [hi if b == 1 else lo + (hi - lo) * ((7 * s) % b) // max(1, b - 1) for s in range(b)]


def _causal_edges(n, window, sinks=0, first=0):
    """Keys that queries first .. n - 1 see: j <= i and (i - j <= window or j < sinks)."""
    near = [min(i + 1, window + 1) for i in range(first, n)]
    return sum(x + min(sinks, i + 1 - x) for i, x in zip(range(first, n), near))


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    def bf16(*shape):
        return normal(*shape).to(torch.bfloat16)

    st = dict(case)
    op, d, hk, b = case["op"], case["dim"], case["kv_heads"], case["batch"]
    if op == "axes":
        n, h, a, half = case["tokens"], case["heads"], case["axes"], case["rotary"] // 2
        packed = bf16(b, n, h + 2 * hk, d)                # one projection's output: queries, keys, values
        st.update(q=packed[:, :, :h], k=packed[:, :, h:h + hk], q_weight=1.0 + 0.1 * normal(d),
                  k_weight=1.0 + 0.1 * normal(d), inv_freq=10000.0 ** (-np.arange(half) * 2.0 / case["rotary"]))
        # one run of pairs per axis, or axis after axis in turn
        st["pair_axes"] = [p % a if case["mixed"] else p * a // half for p in range(half)]
        # frames of 16 x 16 patches: time, height and width, a fourth axis counts frames backwards
        i = torch.arange(n, device="cuda")
        grid = torch.stack([i // 256, i % 256 // 16, i % 16, -(i // 256)], -1)[:, :a]
        start = torch.randint(0, 1000, (b, 1, a), generator=gen, device="cuda")
        start[:, :, 0] += case["first"]
        st["positions"] = (start + grid).to(torch.int32).contiguous()
        if case["train"]:
            st.update(d_q=bf16(b, n, h, d), d_k=bf16(b, n, hk, d))
    elif op == "prefix":
        n, h = case["tokens"], case["heads"]
        st.update(q=bf16(b, n, h, d), k_prefix=bf16(1, case["prefix"], hk, d), v_prefix=bf16(1, case["prefix"], hk, d),
                  k=bf16(b, n, hk, d), v=bf16(b, n, hk, d))
    elif op == "prefix_decode":
        cap = case["capacity"]
        st.update(q=bf16(b, 1, case["heads"], d), k_prefix=bf16(1, case["prefix"], hk, d),
                  v_prefix=bf16(1, case["prefix"], hk, d), k=bf16(b, cap, hk, d), v=bf16(b, cap, hk, d),
                  lengths=torch.tensor(_lengths(case), dtype=torch.int32, device="cuda"))
    elif op == "weights":
        n, h = case["tokens"], case["heads"]
        st.update(q=bf16(b, n, h, d), k=bf16(b, n, hk, d))
        st["lse"] = _lse(st)                              # as the forward left it
    else:
        cap = case["capacity"]
        lengths = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        slot = torch.arange(cap, device="cuda")
        used = slot < lengths[:, None, None]              # [b, 1, cap]
        # heavy-tailed weights; positions with gaps, in an order that earlier evictions have mixed
        weights = (2.0 * normal(b, hk, cap)).exp_() * used
        tokens = torch.randint(1, 4, (b, hk, cap), generator=gen, device="cuda").cumsum(-1) - 1
        order = torch.where(used, torch.rand(b, hk, cap, generator=gen, device="cuda"), 2.0 + slot / cap).argsort(-1)
        positions = tokens.gather(-1, order).to(torch.int32).contiguous()
        st.update(k=bf16(b, cap, hk, d), v=bf16(b, cap, hk, d), weights=weights, positions=positions, lengths=lengths,
                  weights_out=torch.zeros_like(weights), positions_out=torch.zeros_like(positions))
        if op == "scored":
            st.update(q=bf16(b, 1, case["heads"], d), k_new=bf16(b, 1, hk, d), v_new=bf16(b, 1, hk, d),
                      start=lengths - 1, token=torch.full((b,), 3 * cap, dtype=torch.int32, device="cuda"))
        else:
            st["lengths_out"] = torch.zeros_like(lengths)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _run_own(st)
    return {"axes": _plain_axes, "prefix": _plain_prefix, "prefix_decode": _plain_prefix_decode, "weights": _plain_weights,
            "scored": _plain_scored, "evict": _plain_evict}[st["op"]](st)


def _run_own(st):
    import content_adaptive_sparse_gb300 as sa
    op = st["op"]
    if op == "axes":
        args = (st["q_weight"], st["k_weight"], st["inv_freq"], st["pair_axes"], st["positions"], 1e-6, st["interleaved"])
        q_out, k_out = sa.qk_norm_rope_axes_fwd(st["q"], st["k"], *args)
        out = {"q_out": q_out, "k_out": k_out}
        if st["train"]:
            grads = sa.qk_norm_rope_axes_bwd(st["q"], st["k"], st["d_q"], st["d_k"], *args)
            out.update(zip(("dq", "dk", "dq_weight", "dk_weight"), grads))
        return out
    if op == "prefix":
        o, lse = sa.prefix_attn_fwd(st["q"], st["k_prefix"], st["v_prefix"], st["k"], st["v"], st["window"])
        return {"o": o, "lse": lse}
    if op == "prefix_decode":
        o, lse = sa.prefix_attn_decode(st["q"], st["k_prefix"], st["v_prefix"], st["k"], st["v"], st["lengths"], st["window"])
        return {"o": o, "lse": lse}
    if op == "weights":
        return {"weights": sa.sink_attn_weights(st["q"], st["k"], st["lse"], st["window"], st["sinks"], st["first"])}
    cache = sa.ScoredCache(st["k"], st["v"], st["weights"], st["positions"])
    if op == "scored":
        sa.scored_append(cache, st["k_new"], st["v_new"], st["start"], st["token"])
        o, lse = sa.scored_attn_decode(st["q"], cache, st["lengths"], st["decay"], st["weights_out"])
        return {"o": o, "lse": lse, "weights": st["weights_out"]}
    w, p, n = sa.scored_evict(cache, st["lengths"], st["keep"], st["sinks"], st["recent"], st["weights_out"],
                              st["positions_out"], st["lengths_out"])
    return {"k": st["k"], "v": st["v"], "weights": w, "positions": p, "lengths": n}


# ------------------------------------------------------------------ plain forms (32 bits)

def _rotate(x, cos, sin, rotary, interleaved):
    """x [b, n, heads, d] with its first `rotary` elements turned pair by pair."""
    if interleaved:
        lo, hi = x[..., 0:rotary:2], x[..., 1:rotary:2]
        rot = torch.stack((lo * cos - hi * sin, hi * cos + lo * sin), dim=-1).flatten(-2)
    else:
        lo, hi = x[..., :rotary // 2], x[..., rotary // 2:rotary]
        rot = torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), dim=-1)
    return torch.cat((rot, x[..., rotary:]), dim=-1)


def _plain_axes(st):
    freq = torch.tensor(st["inv_freq"], dtype=torch.float64, device="cuda")
    axes = torch.tensor(st["pair_axes"], device="cuda")
    angle = (st["positions"].double()[..., axes] * freq)[:, :, None, :]      # far positions: 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    rotary, inter = st["rotary"], st["interleaved"]

    def forward(x, w):
        x = x.float()
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        return _rotate(x * rstd * w, cos, sin, rotary, inter).to(torch.bfloat16)

    def backward(x, w, dy):
        x = x.float()
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        xh = x * rstd
        g = _rotate(dy.float(), cos, -sin, rotary, inter)
        gw = g * w
        dx = rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True))
        return dx.to(torch.bfloat16), (g * xh).sum((0, 1, 2))

    out = {"q_out": forward(st["q"], st["q_weight"]), "k_out": forward(st["k"], st["k_weight"])}
    if st["train"]:
        out["dq"], out["dq_weight"] = backward(st["q"], st["q_weight"], st["d_q"])
        out["dk"], out["dk_weight"] = backward(st["k"], st["k_weight"], st["d_k"])
    return out


def _softmax(s):
    """exp(s - max) in place of s, its sums and the log of the sum of exp(s); rows without a key give zeros."""
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total == 0, 1.0, total), top + total.log()


def _plain_prefix(st):
    """Blocks of queries against the prefix and the band of own keys that their windows reach."""
    q, window = st["q"], st["window"]
    b, n, h, d = q.shape
    hk, np_ = st["kv_heads"], st["prefix"]
    g, scale = h // hk, 1.0 / math.sqrt(d)
    kp, vp = (st[x][0].float().transpose(0, 1) for x in ("k_prefix", "v_prefix"))            # [hk, prefix, d]
    o = torch.empty_like(q)
    lse = torch.empty(b, h, n, dtype=torch.float32, device="cuda")
    for i0 in range(0, n, 512):
        i1 = min(n, i0 + 512)
        j0 = max(0, i0 - window)
        i, j = torch.arange(i0, i1, device="cuda")[:, None], torch.arange(j0, i1, device="cuda")
        hidden = ((j > i) | (i - j > window)).repeat_interleave(g, 0)
        step = max(1, 2048 // (i1 - i0))
        for s0 in range(0, b, step):
            s1 = min(b, s0 + step)
            m = s1 - s0
            # rows (query, head of the group) of every key head
            rows = q[s0:s1, i0:i1].float().view(m, i1 - i0, hk, g, d).transpose(1, 2).reshape(m, hk, -1, d)
            own_k, own_v = (x[s0:s1, j0:i1].float().transpose(1, 2) for x in (st["k"], st["v"]))
            score = torch.cat((rows @ kp.mT, (rows @ own_k.mT).masked_fill_(hidden, -math.inf)), -1).mul_(scale)
            p, total, logs = _softmax(score)
            out = (p[..., :np_] @ vp + p[..., np_:] @ own_v) / total
            o[s0:s1, i0:i1] = out.view(m, hk, i1 - i0, g, d).transpose(1, 2).reshape(m, i1 - i0, h, d).to(q.dtype)
            lse[s0:s1, :, i0:i1] = logs.view(m, hk, i1 - i0, g).transpose(2, 3).reshape(m, h, i1 - i0)
    return {"o": o, "lse": lse}


def _plain_prefix_decode(st):
    q, window, n = st["q"], st["window"], st["lengths"].long()
    b, _, h, d = q.shape
    hk, np_ = st["kv_heads"], st["prefix"]
    g, scale = h // hk, 1.0 / math.sqrt(d)
    rows = q.float().view(b, hk, g, d)
    kp, vp = (st[x][0].float().transpose(0, 1) for x in ("k_prefix", "v_prefix"))
    k, v = (st[x].float().transpose(1, 2) for x in ("k", "v"))                               # [b, hk, capacity, d]
    j = torch.arange(st["capacity"], device="cuda")
    hidden = (j >= n[:, None]) | (n[:, None] - 1 - j > window)
    mine = (rows @ k.mT).masked_fill_(hidden[:, None, None], -math.inf)
    folded = rows.permute(1, 0, 2, 3).reshape(hk, b * g, d)
    common = (folded @ kp.mT).view(hk, b, g, np_).transpose(0, 1)
    p, total, lse = _softmax(torch.cat((common, mine), -1).mul_(scale))
    far = p[..., :np_].transpose(0, 1).reshape(hk, b * g, np_) @ vp
    out = (far.view(hk, b, g, d).transpose(0, 1) + p[..., np_:] @ v) / total
    return {"o": out.reshape(b, 1, h, d).to(q.dtype), "lse": lse.reshape(b, h, 1)}


def _sink_scores(st, i0, i1, s):
    """Scores [hk, g * queries, keys] of queries i0 .. i1 - 1 of sequence s over the keys j < i1, hidden ones -inf."""
    q, k = st["q"][s, i0:i1], st["k"][s, :i1]
    hk, d = st["kv_heads"], st["dim"]
    rows = q.float().view(i1 - i0, hk, -1, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
    i, j = torch.arange(i0, i1, device="cuda")[:, None], torch.arange(i1, device="cuda")
    hidden = (j > i) | ((i - j > st["window"]) & (j >= st["sinks"]))
    score = (rows @ k.float().permute(1, 2, 0)).mul_(1.0 / math.sqrt(d))
    return score.view(hk, -1, i1 - i0, i1).masked_fill_(hidden, -math.inf)


def _blocks(st):
    b, n = st["q"].shape[:2]
    for s in range(b):
        for i0 in range(st["first"], n, 1024):
            yield s, i0, min(n, i0 + 1024)


def _lse(st):
    """lse [b, h, n] of the queries from `first` on (zeros before it)."""
    b, n, h, _ = st["q"].shape
    lse = torch.zeros(b, h, n, dtype=torch.float32, device="cuda")
    for s, i0, i1 in _blocks(st):
        lse[s, :, i0:i1] = _sink_scores(st, i0, i1, s).logsumexp(-1).view(h, i1 - i0)
    return lse


def _plain_weights(st):
    b, n, h, _ = st["q"].shape
    hk = st["kv_heads"]
    out = torch.zeros(b, hk, n, dtype=torch.float32, device="cuda")
    for s, i0, i1 in _blocks(st):
        score = _sink_scores(st, i0, i1, s)
        lse = st["lse"][s, :, i0:i1].reshape(hk, -1, i1 - i0, 1)
        out[s, :, :i1] += score.sub_(lse).exp_().sum((1, 2))
    return {"weights": out}


def _plain_scored(st):
    q, n = st["q"], st["lengths"].long()
    b, _, h, d = q.shape
    hk, cap = st["kv_heads"], st["capacity"]
    at = torch.arange(b, device="cuda"), st["start"].long()
    st["k"][at] = st["k_new"][:, 0]
    st["v"][at] = st["v_new"][:, 0]
    st["weights"][at[0], :, at[1]] = 0.0
    st["positions"][at[0], :, at[1]] = st["token"][:, None]
    k, v = (st[x].float().transpose(1, 2) for x in ("k", "v"))
    seen = torch.arange(cap, device="cuda") < n[:, None]                                     # [b, cap]
    score = (q.float().view(b, hk, h // hk, d) @ k.mT).mul_(1.0 / math.sqrt(d))
    p, total, lse = _softmax(score.masked_fill_(~seen[:, None, None], -math.inf))
    p = p.div_(total)
    new = st["decay"] * st["weights"] + p.sum(2)
    st["weights_out"].copy_(torch.where(seen[:, None], new, st["weights_out"]))
    return {"o": (p @ v).view(b, 1, h, d).to(q.dtype), "lse": lse.view(b, h, 1), "weights": st["weights_out"]}


def _plain_evict(st):
    w, pos, n = st["weights"], st["positions"], st["lengths"].long()
    b, hk, cap = w.shape
    keep = st["keep"]
    slot = torch.arange(cap, device="cuda")
    used = slot < n[:, None, None]
    newest = torch.where(used, pos, -1).amax(-1, keepdim=True)
    safe = (pos < st["sinks"]) | (pos > newest - st["recent"])
    rank = torch.where(used, torch.where(safe, math.inf, w), -1.0)
    best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.zeros_like(used.expand_as(w)).scatter_(-1, best, True) & used
    # the e-th kept row at or past `keep` goes to the e-th freed slot below it
    hole = ~kept & (slot < keep) & used
    mover = kept & (slot >= keep)
    s, head, src = mover.nonzero(as_tuple=True)
    _, _, dst = hole.nonzero(as_tuple=True)               # as many per (sequence, head), in the same order
    # (a sequence of `keep` slots or fewer has neither)
    st["k"][s, dst, head] = st["k"][s, src, head]
    st["v"][s, dst, head] = st["v"][s, src, head]
    left = used & (slot < keep)
    st["weights_out"].copy_(torch.where(left, w, st["weights_out"]))
    st["positions_out"].copy_(torch.where(left, pos, st["positions_out"]))
    st["weights_out"][s, head, dst] = w[s, head, src]
    st["positions_out"][s, head, dst] = pos[s, head, src]
    st["lengths_out"].copy_(n.clamp(max=keep))
    return {"k": st["k"], "v": st["v"], "weights": st["weights_out"], "positions": st["positions_out"],
            "lengths": st["lengths_out"]}


# ------------------------------------------------------------------ work

def work(case):
    op, b, hk, d = case["op"], case["batch"], case["kv_heads"], case["dim"]
    if op == "axes":
        rows = b * case["tokens"] * (case["heads"] + hk)
        passes = 5 if case["train"] else 2                # x, y; with gradients x, dy and dx too
        return {"bytes": rows * d * 2 * passes + b * case["tokens"] * case["axes"] * 4, "flops": rows * d * 4 * passes}
    if op == "evict":
        moved = read = left = 0
        for n in _lengths(case):
            read += 8 * n * hk
            left += 8 * min(n, case["keep"]) * hk
            # of n - keep evicted rows, those below `keep`, were each as likely to go
            moved += (n - case["keep"]) * case["keep"] / n * hk if n > case["keep"] else 0
        return {"bytes": read + left + 2 * moved * 4 * d, "flops": read / 8}
    h = case["heads"]
    if op == "weights":
        seen = b * h * _causal_edges(case["tokens"], case["window"], case["sinks"], case["first"])
        late = case["tokens"] - case["first"]
        return {"bytes": b * (late * h * (2 * d + 4) + case["tokens"] * hk * (2 * d + 4)), "flops": seen * (2 * d + 2)}
    if op == "prefix":
        n = case["tokens"]
        edges = b * h * (n * case["prefix"] + _causal_edges(n, case["window"]))
        return {"bytes": (case["prefix"] + b * n) * hk * 4 * d + b * n * h * (4 * d + 4), "flops": 4 * d * edges}
    if op == "prefix_decode":
        seen = sum(min(n, case["window"] + 1) for n in _lengths(case))
        return {"bytes": (case["prefix"] + seen) * hk * 4 * d + b * h * (4 * d + 4),
                "flops": 4 * d * h * (b * case["prefix"] + seen)}
    seen = sum(_lengths(case))
    return {"bytes": seen * hk * (4 * d + 8) + b * (h * (4 * d + 4) + hk * 8 * d), "flops": (4 * d + 2) * h * seen}


# ------------------------------------------------------------------ exact values (64 bits)

def exact(case, seed):
    st = prepare(case, seed)
    return {"axes": _exact_axes, "prefix": _exact_prefix, "prefix_decode": _exact_prefix_decode, "weights": _exact_weights,
            "scored": _exact_scored, "evict": _exact_evict}[case["op"]](st)


def _exact_axes(st):
    rotary, half = st["rotary"], st["rotary"] // 2
    pair = torch.arange(half, device="cuda")
    lo, hi = (2 * pair, 2 * pair + 1) if st["interleaved"] else (pair, pair + half)
    per_pair = torch.stack([st["positions"][:, :, a] for a in st["pair_axes"]], -1).double()
    angle = (per_pair * torch.tensor(st["inv_freq"], device="cuda"))[:, :, None]
    turn = torch.polar(torch.ones_like(angle), angle)     # each pair as a complex number

    def formula(x, w):
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        z = torch.complex(y[..., lo], y[..., hi]) * turn
        return y.index_copy(-1, lo, z.real).index_copy(-1, hi, z.imag)

    out = {}
    for name, x, w, dy in (("q", st["q"], st["q_weight"], st.get("d_q")), ("k", st["k"], st["k_weight"], st.get("d_k"))):
        x, w = x.double().requires_grad_(), w.double().requires_grad_()
        y = formula(x, w)
        out[name + "_out"] = y.detach()
        if st["train"]:
            out["d" + name], out["d%s_weight" % name] = torch.autograd.grad(y, (x, w), dy.double())
    return out


def _exact_prefix(st):
    b, n, h, d = st["q"].shape
    g = h // st["kv_heads"]
    o = torch.empty(b, n, h, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(b, h, n, dtype=torch.float64, device="cuda")
    at = torch.arange(n, device="cuda")
    for head in range(h):
        kp, vp = st["k_prefix"][0, :, head // g].double(), st["v_prefix"][0, :, head // g].double()
        for s in range(b):
            keys = torch.cat((kp, st["k"][s, :, head // g].double()))
            values = torch.cat((vp, st["v"][s, :, head // g].double()))
            for i0 in range(0, n, 2048):
                i = at[i0:i0 + 2048, None]
                see = torch.cat((torch.ones(len(i), len(kp), dtype=torch.bool, device="cuda"),
                                 (at <= i) & (i - at <= st["window"])), 1)
                score = torch.where(see, st["q"][s, i0:i0 + 2048, head].double() @ keys.T / math.sqrt(d), -math.inf)
                lse[s, head, i0:i0 + 2048] = score.logsumexp(-1)
                o[s, i0:i0 + 2048, head] = score.softmax(-1) @ values
    return {"o": o, "lse": lse}


def _exact_prefix_decode(st):
    b, _, h, d = st["q"].shape
    g = h // st["kv_heads"]
    o, lse = torch.empty(b, 1, h, d, dtype=torch.float64, device="cuda"), torch.empty(b, h, 1, dtype=torch.float64, device="cuda")
    for hk in range(st["kv_heads"]):
        kp, vp = st["k_prefix"][0, :, hk].double(), st["v_prefix"][0, :, hk].double()
        mine = slice(hk * g, hk * g + g)
        for s, n in enumerate(_lengths(st)):
            near = slice(max(0, n - 1 - st["window"]), n)
            keys = torch.cat((kp, st["k"][s, near, hk].double()))
            values = torch.cat((vp, st["v"][s, near, hk].double()))
            score = st["q"][s, 0, mine].double() @ keys.T / math.sqrt(d)
            o[s, 0, mine] = score.softmax(-1) @ values
            lse[s, mine, 0] = score.logsumexp(-1)
    return {"o": o, "lse": lse}


def _exact_weights(st):
    b, n, h, d = st["q"].shape
    g = h // st["kv_heads"]
    out = torch.zeros(b, st["kv_heads"], n, dtype=torch.float64, device="cuda")
    j = torch.arange(n, device="cuda")
    for s in range(b):
        for head in range(h):
            k = st["k"][s, :, head // g].double()
            for i0 in range(st["first"], n, 2048):
                i = j[i0:i0 + 2048, None]
                see = (i >= j) & ((i - j <= st["window"]) | (j < st["sinks"]))
                log_p = st["q"][s, i0:i0 + 2048, head].double() @ k.T / math.sqrt(d) - st["lse"][s, head, i0:i0 + 2048, None].double()
                out[s, head // g] += torch.where(see, log_p.exp(), 0.0).sum(0)
    return {"weights": out}


def _exact_scored(st):
    b, _, h, d = st["q"].shape
    hk = st["kv_heads"]
    g = h // hk
    o, lse = torch.empty(b, 1, h, d, dtype=torch.float64, device="cuda"), torch.empty(b, h, 1, dtype=torch.float64, device="cuda")
    weights = torch.zeros(b, hk, st["capacity"], dtype=torch.float64, device="cuda")
    for s, n in enumerate(_lengths(st)):
        for head in range(hk):
            k = torch.cat((st["k"][s, :n - 1, head], st["k_new"][s, :, head])).double()
            v = torch.cat((st["v"][s, :n - 1, head], st["v_new"][s, :, head])).double()
            mine = slice(head * g, head * g + g)
            score = st["q"][s, 0, mine].double() @ k.T / math.sqrt(d)
            p = score.softmax(-1)
            o[s, 0, mine] = p @ v
            lse[s, mine, 0] = score.logsumexp(-1)
            old = st["weights"][s, head, :n].double()
            old[n - 1] = 0.0
            weights[s, head, :n] = st["decay"] * old + p.sum(0)
    return {"o": o, "lse": lse, "weights": weights}


def _exact_evict(st):
    """Row by row on the host: the protected slots, then slots in falling order of weight."""
    keep = st["keep"]
    k, v = st["k"].double(), st["v"].double()
    w, p = np.zeros(st["weights"].shape), np.zeros(st["positions"].shape, dtype=np.int32)
    all_w, all_p = st["weights"].cpu().numpy(), st["positions"].cpu().numpy()
    for s, n in enumerate(_lengths(st)):
        for head in range(st["kv_heads"]):
            wh, ph = all_w[s, head, :n].astype(np.float64), all_p[s, head, :n]
            at = np.arange(n)
            if n > keep:
                safe = (ph < st["sinks"]) | (ph > ph.max() - st["recent"])
                chosen = set(np.lexsort((at, -wh, ~safe))[:keep].tolist())
                free = [x for x in range(keep) if x not in chosen]
                far = sorted(x for x in chosen if x >= keep)
                at = np.arange(keep)
                at[free] = far
                f, m = torch.tensor(free, device="cuda"), torch.tensor(far, device="cuda")
                if free:
                    k[s, f, head], v[s, f, head] = k[s, m, head], v[s, m, head]
            w[s, head, :len(at)], p[s, head, :len(at)] = wh[at], ph[at]
    lengths = torch.tensor([min(n, keep) for n in _lengths(st)], dtype=torch.int32, device="cuda")
    return {"k": k, "v": v, "weights": torch.from_numpy(w).cuda(), "positions": torch.from_numpy(p).cuda(), "lengths": lengths}
