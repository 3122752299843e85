"""float64 forms of the calls around shared prefixes and caches with accumulated weights, with elementwise
error bounds as in oracle/streaming.py (a bf16 rounding is off by at most 2^-8 of its value). Written from the
definitions; no code is shared with the CUDA path."""
from __future__ import annotations

import numpy as np

from .streaming import U, _softmax, sink_mask

# A probability in fp32: scores of |s| <= about 20 and LSE are each off by less than 1e-4 (see the LSE tolerance of
# the streaming tests)
P_REL = 2e-4


def prefix_attention(q, k_prefix, v_prefix, k, v, window, scale=None):
    """o [b, n, h, d], lse [b, h, n] and the bound of |o_kernel - o| (P once rounded, and o)."""
    b, n, h, d = q.shape
    g = h // k.shape[2]
    c = d ** -0.5 if scale is None else scale
    pre = k_prefix.shape[1]
    seen = np.concatenate((np.ones((n, pre), bool), sink_mask(n, window, 0)), 1)
    o, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((b, h, n))
    for s in range(b):
        for e in range(h):
            keys = np.concatenate((k_prefix[0, :, e // g], k[s, :, e // g]))
            values = np.concatenate((v_prefix[0, :, e // g], v[s, :, e // g]))
            p, lse[s, e] = _softmax(q[s, :, e] @ keys.T * c, seen)
            o[s, :, e] = p @ values
            mag[s, :, e] = p @ np.abs(values)
    return o, lse, 1.02 * U * (np.abs(o) + mag) + 1e-6


def prefix_decode(q, k_prefix, v_prefix, k, v, lengths, window, scale=None):
    """q [b, 1, h, d] at own token length - 1; o, lse [b, h, 1], bound."""
    b, _, h, d = q.shape
    g = h // k.shape[2]
    c = d ** -0.5 if scale is None else scale
    o, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((b, h, 1), -np.inf)
    for s in range(b):
        n = int(min(max(lengths[s], 0), k.shape[1]))
        near = slice(max(0, n - 1 - window), n)
        for e in range(h):
            keys = np.concatenate((k_prefix[0, :, e // g], k[s, near, e // g]))
            values = np.concatenate((v_prefix[0, :, e // g], v[s, near, e // g]))
            if len(keys) == 0:
                continue
            p, lse[s, e, 0] = _softmax(q[s, 0, e] @ keys.T * c, np.ones(len(keys), bool))
            o[s, 0, e] = p @ values
            mag[s, 0, e] = p @ np.abs(values)
    return o, lse, 1.02 * U * (np.abs(o) + mag) + 1e-6


def scored_decode(q, k, v, lengths, weights, decay, scale=None):
    """o, lse, the bound of o; weights [b, hk, capacity] after the step and their bound."""
    b, _, h, d = q.shape
    hk = k.shape[2]
    g = h // hk
    c = d ** -0.5 if scale is None else scale
    o, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((b, h, 1), -np.inf)
    out, off = weights.copy(), np.zeros(weights.shape)
    for s in range(b):
        n = int(min(max(lengths[s], 0), k.shape[1]))
        for e in range(h if n else 0):
            p, lse[s, e, 0] = _softmax(q[s, 0, e] @ k[s, :n, e // g].T * c, np.ones(n, bool))
            o[s, 0, e] = p @ v[s, :n, e // g]
            mag[s, 0, e] = p @ np.abs(v[s, :n, e // g])
            if e % g == 0:
                out[s, e // g, :n] *= decay
                off[s, e // g, :n] = 2.0 ** -22 * np.abs(out[s, e // g, :n]) + 1e-30
            out[s, e // g, :n] += p
            off[s, e // g, :n] += P_REL * p
    return o, lse, 1.02 * U * (np.abs(o) + mag) + 1e-6, out, off


def sink_weights(q, k, lse, window, sinks, first, scale=None):
    """Weights [b, hk, n] that queries first .. give the keys under `lse`, and their bound."""
    b, n, h, d = q.shape
    hk = k.shape[2]
    g = h // hk
    c = d ** -0.5 if scale is None else scale
    seen = sink_mask(n, window, sinks)[first:]
    out = np.zeros((b, hk, n))
    for s in range(b):
        for e in range(h):
            x = q[s, first:, e] @ k[s, :, e // g].T * c - lse[s, e, first:, None]
            out[s, e // g] += np.exp(np.where(seen, x, -np.inf)).sum(0)
    return out, P_REL * out + 1e-30


def evict(k, v, weights, positions, lengths, keep, sinks, recent):
    """The cache after an eviction: copies of k, v, weights, positions and the lengths (rows past them as before)."""
    k, v, w, p = k.copy(), v.copy(), weights.copy(), positions.copy()
    b, hk, cap = w.shape
    out = [min(max(int(n), 0), cap) for n in lengths]
    for s, n in enumerate(out):
        for e in range(hk if n > keep else 0):
            newest = max(int(x) for x in p[s, e, :n])

            def rank(j):
                x = float(w[s, e, j])
                safe = p[s, e, j] < sinks or int(p[s, e, j]) > newest - recent
                return (0 if safe else 1 if x != x else 2, 0.0 if safe or x != x else -x, j)

            kept = set(sorted(range(n), key=rank)[:keep])
            free = [j for j in range(keep) if j not in kept]
            far = [j for j in range(keep, n) if j in kept]
            for to, at in zip(free, far):
                k[s, to, e], v[s, to, e] = k[s, at, e], v[s, at, e]
                w[s, e, to], p[s, e, to] = w[s, e, at], p[s, e, at]
    return k, v, w, p, [min(n, keep) for n in out]
