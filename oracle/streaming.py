"""float64 forms of the streaming-attention calls, with elementwise error bounds.

Written from the definitions (dense masks, one head at a time); no code is shared with the CUDA
path. Where a kernel must round inside a sum (P and dS to bf16 for the tensor cores, O to bf16
before D), the function also returns the sum of the magnitudes that such a rounding scales, so
that a test can bound the kernel's error element by element: a bf16 rounding is off by at most
2^-8 of its value.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8          # half a bf16 step, relative


def sink_mask(n: int, window: int, sinks: int) -> np.ndarray:
    """[n, n] bool: query i sees key j."""
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    return (j <= i) & ((i - j <= window) | (j < sinks))


def _softmax(s, seen):
    s = np.where(seen, s, -np.inf)
    top = s.max(-1, keepdims=True)
    top = np.where(np.isneginf(top), 0.0, top)
    e = np.exp(s - top)
    total = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (top + np.log(total))[..., 0]
    return e / np.where(total == 0, 1.0, total), lse


def sink_attention(q, k, v, window, sinks, scale=None):
    """o [b, n, h, d], lse [b, h, n] and the bound of |o_kernel - o|."""
    b, n, h, d = q.shape
    g = h // k.shape[2]
    c = d ** -0.5 if scale is None else scale
    seen = sink_mask(n, window, sinks)
    o, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((b, h, n))
    for s in range(b):
        for e in range(h):
            p, lse[s, e] = _softmax(q[s, :, e] @ k[s, :, e // g].T * c, seen)
            o[s, :, e] = p @ v[s, :, e // g]
            mag[s, :, e] = p @ np.abs(v[s, :, e // g])
    return o, lse, 1.02 * U * (np.abs(o) + mag) + 1e-6


def sink_attention_backward(q, k, v, d_o, window, sinks, scale=None, rounded_o=True):
    """(dq, dk, dv) and their bounds; rounded_o: D may be formed from the rounded O."""
    b, n, h, d = q.shape
    hk = k.shape[2]
    g = h // hk
    c = d ** -0.5 if scale is None else scale
    seen = sink_mask(n, window, sinks)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)
    bq, bk, bv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)
    for s in range(b):
        for e in range(h):
            qq, kk, vv, gg = q[s, :, e], k[s, :, e // g], v[s, :, e // g], d_o[s, :, e]
            p, _ = _softmax(qq @ kk.T * c, seen)
            o = p @ vv
            ds = p * (gg @ vv.T - (gg * o).sum(-1, keepdims=True))
            dq[s, :, e] = c * ds @ kk
            dk[s, :, e // g] += c * ds.T @ qq
            dv[s, :, e // g] += p.T @ gg
            # D is formed from the rounded O (off by U (|o| + p |v|)); dS and P are rounded
            off = (np.abs(gg) * (np.abs(o) + p @ np.abs(vv))).sum(-1, keepdims=True)
            worst = np.abs(ds) + (p * off if rounded_o else 0.0)
            bq[s, :, e] = c * worst @ np.abs(kk)
            bk[s, :, e // g] += c * worst.T @ np.abs(qq)
            bv[s, :, e // g] += p.T @ np.abs(gg)
    bounds = [1.05 * U * (np.abs(x) + y) + 2e-5 for x, y in ((dq, bq), (dk, bk), (dv, bv))]
    return (dq, dk, dv), bounds


def sink_decode(q, k, v, lengths, window, sinks, scale=None):
    """q [b, 1, h, d] at token length - 1 over cache rows k, v [b, capacity, hk, d]; o, lse [b, h, 1], bound
    (P once rounded)."""
    b, _, h, d = q.shape
    g = h // k.shape[2]
    c = d ** -0.5 if scale is None else scale
    o, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((b, h, 1), -np.inf)
    for s in range(b):
        n = int(min(max(lengths[s], 0), k.shape[1]))
        j = np.arange(n)
        j = j[(n - 1 - j <= window) | (j < sinks)]
        for e in range(h if n else 0):
            p, l = _softmax(q[s, 0, e] @ k[s, j, e // g].T * c, np.ones(len(j), bool))
            o[s, 0, e] = p @ v[s, j, e // g]
            mag[s, 0, e] = p @ np.abs(v[s, j, e // g])
            lse[s, e, 0] = l
    return o, lse, 1.02 * U * (np.abs(o) + mag) + 1e-6


def _pairs(rotary, interleaved):
    p = np.arange(rotary // 2)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + rotary // 2)


def norm_rope(x, w, positions, inv_freq, eps, interleaved):
    """x [b, n, h, d], positions [b, n]; y and the bound of the kernel's error (one bf16 rounding; fp32
    sums, products and angles below 4e-6 of the magnitudes that they combine)."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    out, mag = y.copy(), np.abs(y)
    a, c = _pairs(2 * len(inv_freq), interleaved)
    t = positions[:, :, None, None].astype(np.float64) * np.asarray(inv_freq)
    out[..., a] = y[..., a] * np.cos(t) - y[..., c] * np.sin(t)
    out[..., c] = y[..., c] * np.cos(t) + y[..., a] * np.sin(t)
    both = mag[..., a] + mag[..., c]
    mag[..., a] = both
    mag[..., c] = both
    return out, 1.01 * U * np.abs(out) + 4e-6 * mag


def norm_rope_backward(x, w, dy, positions, inv_freq, eps, interleaved):
    """(dx, dw) and their bounds (dw: fp32 sums)."""
    d = x.shape[-1]
    g = dy.copy()
    a, c = _pairs(2 * len(inv_freq), interleaved)
    t = positions[:, :, None, None].astype(np.float64) * np.asarray(inv_freq)
    g[..., a] = dy[..., a] * np.cos(t) + dy[..., c] * np.sin(t)
    g[..., c] = dy[..., c] * np.cos(t) - dy[..., a] * np.sin(t)
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * rstd
    dx = rstd * (g * w - xh * (g * w * xh).mean(-1, keepdims=True))
    dw = (g * xh).sum((0, 1, 2))
    size = np.abs(dy).max(-1, keepdims=True) * np.abs(w).max() * rstd * (2 + np.abs(xh) * np.abs(xh).mean(-1, keepdims=True) * 2)
    # the sum of g xh: angles and factors are off by 2e-6 of |dy| |xh|, the sums by 64 roundings of 2^-24
    turn = np.abs(dy)
    both = turn[..., a] + turn[..., c]
    turn[..., a] = both
    turn[..., c] = both
    return (dx, dw), (1.01 * U * np.abs(dx) + 8e-6 * size, 1e-5 * (turn * np.abs(xh)).sum((0, 1, 2)) + 1e-30)


# ------------------------------------------------------------------ 4-bit rows

def bf16_round(x):
    """Nearest bf16 (ties to even) of float64 values, as float64."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))      # 8 significant bits; subnormals from 2^-126 on
    return np.where(np.isfinite(x), np.rint(x / step) * step, x)


def quantise(x):
    """codes (-7 .. 7) and scales [..., d / 32] of rows x [..., d]."""
    runs = x.reshape(*x.shape[:-1], -1, 32)
    scale = bf16_round(np.abs(runs).max(-1) / 7)
    with np.errstate(divide="ignore", invalid="ignore"):
        codes = np.where(scale[..., None] > 0, np.clip(np.rint(runs / scale[..., None]), -7, 7), 0)
    return codes.reshape(x.shape).astype(np.int64), scale


def values(codes, scales):
    return codes * np.repeat(scales, 32, axis=-1)


def pack(codes):
    """uint8 [..., d / 2] of codes [..., d], element by element from the layout's definition."""
    d = codes.shape[-1]
    out = np.zeros(codes.shape[:-1] + (d // 8,), dtype=np.uint32)
    for e in range(d):
        c, t, u = e // 32, e % 32 // 8, e % 8
        p, i = divmod(u, 4)
        out[..., t * (d // 32) + c] |= (codes[..., e] + 8).astype(np.uint32) << np.uint32(8 * p + 4 * (i // 2) + 16 * (i % 2))
    return out.astype("<u4").view(np.uint8)
