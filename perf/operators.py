"""Cases, plain forms and exact values of the streaming-attention operators.

The operators: per-head RMS norms of queries and keys with the position rotation (forward and
backward), causal attention over a token window and a few first tokens that stay visible
("sinks"; forward, and forward with backward), its single-token form over a bf16 cache and over
a cache held in 4 bits, and the 4-bit cache's writing and reading.

Graph of the attention: query i sees key j iff j <= i and (i - j <= window or j < sinks).
With a cache of `length` tokens the query is token length - 1.

4-bit rows: each run of 32 elements of a (token, head) row has one bf16 scale s = amax / 7 and
codes round(x / s) in -7 .. 7, stored + 8. Little-endian 32-bit word t * (d / 32) + c of a row
holds elements 32 c + 8 t + u, u = 0 .. 7, element u = 4 p + i at bit 8 p + 4 (i // 2) + 16 (i % 2).
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # queries and keys of one decoding step: 8 sequences at far positions, 16 heads of 128
        # over 4 key heads; a call of microseconds
        {"name": "norm_rope_step", "op": "norm_rope", "batch": 8, "tokens": 1, "heads": 16, "kv_heads": 4, "dim": 128,
         "rotary": 128, "interleaved": False, "train": False, "first": 60000},
        # the 8K training shape (4 x 8192 tokens, 12 heads of 64), forward and backward
        {"name": "norm_rope_train_8k", "op": "norm_rope", "batch": 4, "tokens": 8192, "heads": 12, "kv_heads": 12,
         "dim": 64, "rotary": 64, "interleaved": False, "train": True, "first": 0},
        # a long prompt: one sequence of 65536 tokens, 16 heads of 128 over 4 key heads
        {"name": "sink_fwd_64k", "op": "sink", "batch": 1, "tokens": 65536, "heads": 16, "kv_heads": 4, "dim": 128,
         "window": 4095, "sinks": 4, "train": False},
        # a short ragged prompt, heads of 32
        {"name": "sink_fwd_ragged", "op": "sink", "batch": 3, "tokens": 997, "heads": 8, "kv_heads": 2, "dim": 32,
         "window": 200, "sinks": 17, "train": False},
        # a training step's attention at the 8K shape, short window
        {"name": "sink_train_8k", "op": "sink", "batch": 4, "tokens": 8192, "heads": 12, "kv_heads": 12, "dim": 64,
         "window": 511, "sinks": 4, "train": True},
        # and of a 16K sequence with 16 heads of 128 that share 4 key heads, ragged length
        {"name": "sink_train_16k", "op": "sink", "batch": 1, "tokens": 16321, "heads": 16, "kv_heads": 4, "dim": 128,
         "window": 2047, "sinks": 4, "train": True},
        # one token for one short sequence
        {"name": "decode_one", "op": "decode", "batch": 1, "capacity": 1024, "len_lo": 700, "len_hi": 700, "heads": 12,
         "kv_heads": 12, "dim": 64, "window": 511, "sinks": 4},
        # one token for each of 64 sequences of 1000 .. 16000 tokens, window 4096
        {"name": "decode_batch", "op": "decode", "batch": 64, "capacity": 16384, "len_lo": 1000, "len_hi": 16000,
         "heads": 16, "kv_heads": 4, "dim": 128, "window": 4095, "sinks": 4},
        # the same two over a cache in 4 bits: one sequence, and 32 long ones read almost whole
        {"name": "decode4_one", "op": "decode4", "batch": 1, "capacity": 2048, "len_lo": 1500, "len_hi": 1500,
         "heads": 16, "kv_heads": 4, "dim": 128, "window": 1023, "sinks": 4},
        {"name": "decode4_batch", "op": "decode4", "batch": 32, "capacity": 32768, "len_lo": 9001, "len_hi": 32768,
         "heads": 16, "kv_heads": 4, "dim": 128, "window": 16383, "sinks": 4},
        # writing the keys and values of one step of 64 sequences to the 4-bit cache, and back
        {"name": "cache4_step", "op": "cache4", "batch": 64, "tokens": 1, "capacity": 4096, "kv_heads": 4, "dim": 128,
         "first": 777},
        # and of a 16K prompt
        {"name": "cache4_prompt", "op": "cache4", "batch": 2, "tokens": 16384, "capacity": 32768, "kv_heads": 8,
         "dim": 128, "first": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8, 12])
    return kv * rng.choice([1, 1, 2, 4] if kv <= 8 else [1]), kv


def draw(rng):
    op = rng.choice(["norm_rope", "sink", "sink", "decode", "decode4", "cache4"])
    dim = rng.choice([32, 64, 128])
    heads, kv = _heads(rng)
    case = {"op": op, "dim": dim, "kv_heads": kv}
    if op == "norm_rope":
        tokens = _log(rng, 1, 16384)
        case.update(batch=max(1, min(rng.choice([1, 2, 3, 8]), 32768 // tokens)), tokens=tokens, heads=heads,
                    rotary=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.3, train=rng.random() < 0.5,
                    first=_log(rng, 1, 500000))
    elif op == "sink":
        tokens = _log(rng, 1, 16384)
        case.update(batch=max(1, min(rng.choice([1, 2, 3]), 24576 // tokens)), tokens=tokens, heads=heads,
                    window=_log(rng, 1, 4096) - 1, sinks=rng.choice([0, 1, 4, 16, rng.randrange(129)]),
                    train=rng.random() < 0.5)
    elif op in ("decode", "decode4"):
        capacity = -(-_log(rng, 16, 32768) // 8) * 8
        hi = rng.randint(1, capacity)
        case.update(batch=rng.choice([1, 2, 5, 16, 32]), capacity=capacity, len_lo=rng.randint(1, hi), len_hi=hi,
                    heads=heads, window=_log(rng, 1, 16384) - 1, sinks=rng.choice([0, 1, 4, 16, rng.randrange(129)]))
    else:
        tokens = _log(rng, 1, 8192)
        first = rng.randrange(4096)
        case.update(batch=rng.choice([1, 2, 5]), tokens=tokens, capacity=-(-(first + tokens) // 8) * 8 + 8 * rng.randrange(8), first=first)
    return case


def _lengths(case):
    """Tokens of each sequence of a decoding case, spread over [len_lo, len_hi]."""
    b, lo, hi = case["batch"], case["len_lo"], case["len_hi"]
    return [hi if b == 1 else lo + (hi - lo) * ((7 * s) % b) // max(1, b - 1) for s in range(b)]


def _seen(length, window, sinks):
    """Keys that token length - 1 sees."""
    near = min(length, window + 1)
    return near + min(sinks, length - near)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    def bf16(*shape):
        return normal(*shape).to(torch.bfloat16)

    st = dict(case)
    d, hk, b = case["dim"], case["kv_heads"], case["batch"]
    if case["op"] == "norm_rope":
        n, h = case["tokens"], case["heads"]
        packed = bf16(b, n, h + 2 * hk, d)                # one projection's output: queries, keys, values
        st.update(q=packed[:, :, :h], k=packed[:, :, h:h + hk], q_weight=1.0 + 0.1 * normal(d),
                  k_weight=1.0 + 0.1 * normal(d), inv_freq=10000.0 ** (-np.arange(case["rotary"] // 2) * 2.0 / case["rotary"]))
        start = case["first"] + torch.randint(0, 1000, (b, 1), generator=gen, device="cuda")
        st["positions"] = (start + torch.arange(n, device="cuda")).to(torch.int32)
        if case["train"]:
            st.update(d_q=bf16(b, n, h, d), d_k=bf16(b, n, hk, d))
    elif case["op"] == "sink":
        n, h = case["tokens"], case["heads"]
        st.update(q=bf16(b, n, h, d), k=bf16(b, n, hk, d), v=bf16(b, n, hk, d))
        if case["train"]:
            st["d_o"] = bf16(b, n, h, d)
    elif case["op"] == "cache4":
        n, cap = case["tokens"], case["capacity"]
        st.update(k=bf16(b, n, hk, d), v=bf16(b, n, hk, d))
        st["start"] = torch.full((b,), case["first"], dtype=torch.int32, device="cuda")
        st["cache"] = _empty_cache(b, cap, hk, d)
    else:
        cap = case["capacity"]
        st["q"] = bf16(b, 1, case["heads"], d)
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        if case["op"] == "decode":
            st.update(k=bf16(b, cap, hk, d), v=bf16(b, cap, hk, d))
        else:
            cache = _empty_cache(b, cap, hk, d)
            for codes, scales in (cache[:2], cache[2:]):   # filled as a run of the model left it
                scales.copy_(0.25 + 0.2 * torch.rand(scales.shape, generator=gen, device="cuda"))
                # codes 1 .. 15 in both nibbles of a byte, whatever element they belong to
                for _ in range(2):
                    codes.mul_(16).add_((normal(*codes.shape) * 2.4).round_().clamp_(-7, 7).add_(8).to(torch.uint8))
            st["cache"] = cache
    return st


def _empty_cache(b, cap, hk, d):
    """k_codes, k_scales, v_codes, v_scales."""
    def rows():
        return [torch.zeros(b, hk, cap, d // 2, dtype=torch.uint8, device="cuda"),
                torch.zeros(b, hk, cap, d // 32, dtype=torch.bfloat16, device="cuda")]
    return tuple(rows() + rows())


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "norm_rope":
        return _plain_norm_rope(st)
    if st["op"] == "sink":
        return _plain_sink(st)
    if st["op"] == "cache4":
        return {"k": _plain_roundtrip(st["k"]), "v": _plain_roundtrip(st["v"])}
    if st["op"] == "decode":
        k, v = st["k"].permute(0, 2, 1, 3), st["v"].permute(0, 2, 1, 3)
        return _plain_decode(st, lambda i: _rows(k, i).float(), lambda i: _rows(v, i).float())
    kc, ks, vc, vs = st["cache"]
    return _plain_decode(st, lambda i: _plain_values(_rows(kc, i), _rows(ks, i)),
                         lambda i: _plain_values(_rows(vc, i), _rows(vs, i)))


def _run_own(st):
    import content_adaptive_sparse_gb300 as sa
    if st["op"] == "norm_rope":
        args = (st["q_weight"], st["k_weight"], st["inv_freq"], st["positions"], 1e-6, st["interleaved"])
        q_out, k_out = sa.qk_norm_rope_fwd(st["q"], st["k"], *args)
        out = {"q_out": q_out, "k_out": k_out}
        if st["train"]:
            grads = sa.qk_norm_rope_bwd(st["q"], st["k"], st["d_q"], st["d_k"], *args)
            out.update(zip(("dq", "dk", "dq_weight", "dk_weight"), grads))
        return out
    if st["op"] == "sink":
        q, k, v, w, s = st["q"], st["k"], st["v"], st["window"], st["sinks"]
        o, lse = sa.sink_attn_fwd(q, k, v, w, s)
        out = {"o": o, "lse": lse}
        if st["train"]:
            out.update(zip(("dq", "dk", "dv"), sa.sink_attn_bwd(q, k, v, o, lse, st["d_o"], w, s)))
        return out
    if st["op"] == "cache4":
        cache = sa.Cache4(*st["cache"])
        sa.cache4_append(cache, st["k"], st["v"], st["start"])
        k, v = sa.cache4_read(cache, st["start"], st["tokens"])
        return {"k": k, "v": v}
    if st["op"] == "decode":
        o, lse = sa.sink_attn_decode(st["q"], st["k"], st["v"], st["lengths"], st["window"], st["sinks"])
    else:
        o, lse = sa.sink_attn_decode_cache4(st["q"], sa.Cache4(*st["cache"]), st["lengths"], st["window"], st["sinks"])
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------ plain forms (32 bits)

def _rotate(x, cos, sin, rotary, interleaved):
    """x [b, n, heads, d] with its first `rotary` elements rotated pair by pair."""
    if interleaved:
        lo, hi = x[..., 0:rotary:2], x[..., 1:rotary:2]
        rot = torch.stack((lo * cos - hi * sin, hi * cos + lo * sin), dim=-1).flatten(-2)
    else:
        lo, hi = x[..., :rotary // 2], x[..., rotary // 2:rotary]
        rot = torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), dim=-1)
    return torch.cat((rot, x[..., rotary:]), dim=-1)


def _plain_norm_rope(st):
    freq = torch.tensor(st["inv_freq"], dtype=torch.float64, device="cuda")
    angle = (st["positions"].double()[..., None] * freq)[:, :, None, :]     # far positions: 64 bits
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


def _plain_sink(st):
    """Blocks of queries against the band of keys that the block's window reaches, plus the sinks."""
    q, k, v, window, sinks = st["q"], st["k"], st["v"], st["window"], st["sinks"]
    b, n, h, d = q.shape
    hk = k.shape[2]
    g = h // hk
    c = min(512, n)
    nb = -(-n // c)
    reach = min(window, (nb - 1) * c)
    scale = 1.0 / math.sqrt(d)
    first = torch.arange(nb, device="cuda")[:, None] * c
    near = first - reach + torch.arange(reach + c, device="cuda")            # [nb, reach + c]
    far = torch.arange(min(sinks, n), device="cuda").expand(nb, -1)
    far = torch.where(far < first - reach, far, -1)                          # sinks that the band does not hold
    key = torch.cat((far, near), dim=1)                                      # [nb, L]
    query = first + torch.arange(c, device="cuda")                           # [nb, c]
    i, j = query[:, :, None], key[:, None, :]
    seen = (j >= 0) & (j <= i) & (i < n) & ((i - j <= window) | (j < sinks))  # [nb, c, L]
    at = key.clamp(0, n - 1)

    def queries(x):                                                          # [b, nb, hk, g * c, d] in 32 bits
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, nb * c - n))
        return x.view(b, nb, c, hk, g, d).permute(0, 1, 3, 4, 2, 5).reshape(b, nb, hk, g * c, d)

    def back(x):
        x = x.view(b, nb, hk, g, c, d).permute(0, 1, 4, 2, 3, 5).reshape(b, nb * c, h, d)
        return x[:, :n]

    def keys(x):                                                             # [b, nb, hk, L, d]
        return x.float()[:, at].permute(0, 1, 3, 2, 4)

    qb, kb, vb = queries(q), keys(k), keys(v)
    hidden = ~seen.repeat(1, g, 1)[None, :, None]
    s = (qb @ kb.transpose(-1, -2)).mul_(scale).masked_fill_(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = top + total.log()
    p.div_(torch.where(total == 0, 1.0, total))
    ob = p @ vb
    o = back(ob).to(torch.bfloat16)
    out = {"o": o, "lse": lse.view(b, nb, hk, g, c).permute(0, 2, 3, 1, 4).reshape(b, h, nb * c)[:, :, :n].contiguous()}
    if st["train"]:
        gb = queries(st["d_o"])
        dv = p.transpose(-1, -2) @ gb
        ds = (gb @ vb.transpose(-1, -2)).sub_((gb * ob).sum(-1, keepdim=True)).mul_(p)
        out["dq"] = back((ds @ kb).mul_(scale)).to(torch.bfloat16)
        dk = (ds.transpose(-1, -2) @ qb).mul_(scale)

        def gather(x):                                                       # sums the blocks' rows of each key
            rows = x.permute(0, 1, 3, 2, 4).reshape(b, -1, hk, d)
            return torch.zeros(b, n, hk, d, device="cuda").index_add_(1, at.flatten(), rows).to(torch.bfloat16)

        out["dk"], out["dv"] = gather(dk), gather(dv)
    return out


def _rows(x, at):
    """Rows at [b, L] of a [b, kv_heads, capacity, row] tensor."""
    b, hk, cap, r = x.shape
    return x.gather(2, at[:, None, :, None].expand(b, hk, at.shape[1], r))


def _plain_decode(st, k_rows, v_rows):
    q, lengths, window, sinks = st["q"], st["lengths"].long(), st["window"], st["sinks"]
    b, _, h, d = q.shape
    hk, cap = st["kv_heads"], st["capacity"]
    near = min(window + 1, cap)
    lo = (lengths - near).clamp(min=0)[:, None]
    j = torch.cat((lo + torch.arange(near, device="cuda"), torch.arange(min(sinks, cap), device="cuda").expand(b, -1)), 1)
    seen = j < lengths[:, None]
    seen[:, near:] &= j[:, near:] < lo                                       # sinks that the window does not hold
    at = j.clamp(0, cap - 1)
    qg = q.float().view(b, hk, h // hk, d)
    s = (qg @ k_rows(at).transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).masked_fill_(~seen[:, None, None, :], -math.inf)
    lse = s.logsumexp(-1, keepdim=True)
    o = (s.sub_(lse).exp_() @ v_rows(at)).view(b, 1, h, d).to(torch.bfloat16)
    return {"o": o, "lse": lse.view(b, h, 1)}


def _plain_roundtrip(x):
    runs = x.float().unflatten(-1, (-1, 32))
    scale = (runs.abs().amax(-1, keepdim=True) / 7.0).to(torch.bfloat16).float()
    codes = (runs / torch.where(scale == 0, 1.0, scale)).round().clamp(-7, 7)
    return (codes * scale).flatten(-2).to(torch.bfloat16)


def _order(d):
    """For element e of a row: its byte, and its nibble in it."""
    e = torch.arange(d, device="cuda")
    c, t, u = e // 32, e % 32 // 8, e % 8
    bit = 8 * (u // 4) + 4 * (u % 4 // 2) + 16 * (u % 2)
    return 4 * (t * (d // 32) + c) + bit // 8, bit % 8


def _plain_values(codes, scales):
    """Rows [..., d / 2] of codes and their scales [..., d / 32] as 32-bit numbers."""
    at, shift = _order(2 * codes.shape[-1])
    values = ((codes[..., at] >> shift.to(torch.uint8)) & 15).float().sub_(8.0)
    return (values.unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


# ------------------------------------------------------------------ work

def work(case):
    b, hk, d = case["batch"], case["kv_heads"], case["dim"]
    if case["op"] == "norm_rope":
        rows = b * case["tokens"] * (case["heads"] + hk)
        passes = 5 if case["train"] else 2                # x, y; with gradients x, dy and dx too
        return {"bytes": rows * d * 2 * passes + b * case["tokens"] * 4, "flops": rows * d * 8 * passes / 2}
    if case["op"] == "sink":
        n, h, w, s = case["tokens"], case["heads"], case["window"], case["sinks"]
        edges = b * h * sum(_seen(i + 1, w, s) for i in range(n))
        bytes_q, bytes_k = b * n * h * d * 2, b * n * hk * d * 2
        if case["train"]:                                 # q, o, d_o, dq; k, v, dk, dv; lse
            return {"bytes": 4 * bytes_q + 4 * bytes_k + b * h * n * 4, "flops": 14 * edges * d}
        return {"bytes": 2 * bytes_q + 2 * bytes_k + b * h * n * 4, "flops": 4 * edges * d}
    if case["op"] == "cache4":
        values = 2 * b * case["tokens"] * hk * d          # read in bf16, 4.5 bits written and read, bf16 written
        return {"bytes": values * (2 + 2 + 2 * 4.5 / 8), "flops": values * 4}
    seen = sum(_seen(length, case["window"], case["sinks"]) for length in _lengths(case))
    row = d * 2 if case["op"] == "decode" else d // 2 + d // 16
    return {"bytes": 2 * seen * hk * row + 2 * b * case["heads"] * d * 2, "flops": 4 * seen * case["heads"] * d}


# ------------------------------------------------------------------ exact values (64 bits)

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "sink": _exact_sink, "decode": _exact_decode, "decode4": _exact_decode,
            "cache4": _exact_cache4}[case["op"]](st)


def _exact_norm_rope(st):
    rotary, half = st["rotary"], st["rotary"] // 2
    pair = torch.arange(half, device="cuda")
    lo, hi = (2 * pair, 2 * pair + 1) if st["interleaved"] else (pair, pair + half)
    angle = st["positions"].double()[:, :, None, None] * torch.tensor(st["inv_freq"], device="cuda")
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


def _exact_sink(st):
    b, n, h, d = st["q"].shape
    hk, window, sinks = st["kv_heads"], st["window"], st["sinks"]
    g, dev = h // hk, "cuda"
    out = {"o": torch.empty(b, n, h, d, dtype=torch.float64, device=dev),
           "lse": torch.empty(b, h, n, dtype=torch.float64, device=dev)}
    if st["train"]:
        out["dq"] = torch.empty_like(out["o"])
        out["dk"] = torch.zeros(b, n, hk, d, dtype=torch.float64, device=dev)
        out["dv"] = torch.zeros_like(out["dk"])
    for q0 in range(0, n, 1024):
        q1 = min(n, q0 + 1024)
        reach = max(0, q0 - window)
        at = torch.cat((torch.arange(min(sinks, reach), device=dev), torch.arange(reach, q1, device=dev)))
        i, j = torch.arange(q0, q1, device=dev)[:, None], at[None, :]
        bias = torch.zeros(q1 - q0, len(at), dtype=torch.float64, device=dev)
        bias[(j > i) | ((i - j > window) & (j >= sinks))] = -math.inf
        for s in range(b):
            for head in range(hk):
                mine = slice(head * g, head * g + g)
                q = st["q"][s, q0:q1, mine].double().transpose(0, 1).requires_grad_()     # [g, queries, d]
                k = st["k"][s, at, head].double().requires_grad_()
                v = st["v"][s, at, head].double().requires_grad_()
                with torch.set_grad_enabled(bool(st["train"])):
                    score = q @ k.T / math.sqrt(d) + bias
                    o = torch.softmax(score, -1) @ v
                out["o"][s, q0:q1, mine] = o.detach().transpose(0, 1)
                out["lse"][s, mine, q0:q1] = score.detach().logsumexp(-1)
                if st["train"]:
                    dq, dk, dv = torch.autograd.grad(o, (q, k, v), st["d_o"][s, q0:q1, mine].double().transpose(0, 1))
                    out["dq"][s, q0:q1, mine] = dq.transpose(0, 1)
                    out["dk"][s, at, head] += dk
                    out["dv"][s, at, head] += dv
    return out


def _exact_rows(codes, scales, at):
    """Values of the 4-bit rows `at` of one (sequence, head), from the layout's definition."""
    words = codes[at].contiguous().view(torch.int32).long()                  # [rows, d / 8]
    d = 8 * words.shape[1]
    x = torch.empty(len(at), d, dtype=torch.float64, device=codes.device)
    for c in range(d // 32):
        for t in range(4):
            for u in range(8):
                p, i = divmod(u, 4)
                code = (words[:, t * (d // 32) + c] >> (8 * p + 4 * (i // 2) + 16 * (i % 2))) & 15
                x[:, 32 * c + 8 * t + u] = (code - 8) * scales[at, c].double()
    return x


def _exact_decode(st):
    q = st["q"].double()
    b, _, h, d = q.shape
    hk = st["kv_heads"]
    g = h // hk
    o, lse = torch.empty_like(q), torch.empty(b, h, 1, dtype=torch.float64, device=q.device)
    for s, length in enumerate(_lengths(st)):
        j = torch.arange(length, device=q.device)
        at = j[(length - 1 - j <= st["window"]) | (j < st["sinks"])]
        for head in range(hk):
            if st["op"] == "decode":
                k, v = st["k"][s, at, head].double(), st["v"][s, at, head].double()
            else:
                kc, ks, vc, vs = (x[s, head] for x in st["cache"])
                k, v = _exact_rows(kc, ks, at), _exact_rows(vc, vs, at)
            mine = slice(head * g, head * g + g)
            score = q[s, 0, mine] @ k.T / math.sqrt(d)
            o[s, 0, mine] = torch.softmax(score, -1) @ v
            lse[s, mine, 0] = score.logsumexp(-1)
    return {"o": o, "lse": lse}


def _exact_cache4(st):
    out = {}
    for name in ("k", "v"):
        x = st[name].double().view(*st[name].shape[:-1], -1, 32)
        scale = (x.abs().max(-1).values / 7).to(torch.bfloat16).double()[..., None]
        code = torch.where(scale > 0, x / scale, 0.0).round().clamp(-7, 7)
        out[name] = (code * scale).view(st[name].shape)
    return out
