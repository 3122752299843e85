"""Shared contexts and bounded caches: the calls around a prefix that a batch shares and around a cache of
slots with accumulated attention weights (binding of sa_api.h's parts of these names; re-exported by the
package).

``sa_*`` functions carry the C ABI's names and write into tensors that the caller gives; the others
allocate their outputs (and workspace) and make one call. Argument checks are those of the streaming
calls: ``ValueError`` for types, shapes, strides and devices of tensors, ``SAError`` for the library's own
refusals.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

from . import streaming as _s
from .streaming import _F32, _I32, _P, _S3, _check, _dense, _device, _flat, _int, _lib, _like, _rows, _stream, _workspace

_SIZE = ctypes.c_size_t
_NO_ROWS = _S3(0, 0, 0)


def declare(lib) -> None:
    """Argument types of this module's entry points (called once, when the library is loaded)."""
    signatures = {
        "sa_prefix_attn_fwd_workspace_size": [_I32] * 7 + [_P],
        "sa_prefix_attn_fwd": [_P] * 5 + [_S3] * 6 + [_I32] * 7 + [_F32, _P, _P, _P, _SIZE, _P],
        "sa_prefix_attn_decode_workspace_size": [_I32] * 5 + [_P],
        "sa_prefix_attn_decode": [_P] * 5 + [_S3] * 6 + [_I32] * 6 + [_P, _I32, _F32, _P, _P, _P, _SIZE, _P],
        "sa_scored_append": [_P, _P, _S3, _S3] + [_I32] * 5 + [_P] * 4 + [_S3, _S3, _P, _P, _P],
        "sa_scored_attn_decode_workspace_size": [_I32] * 4 + [_P],
        "sa_scored_attn_decode": [_P] * 3 + [_S3] * 4 + [_I32] * 5 + [_P, _F32, _F32] + [_P] * 5 + [_SIZE, _P],
        "sa_scored_evict": [_P, _P, _S3, _S3] + [_I32] * 7 + [_P] * 7,
        "sa_sink_attn_weights_workspace_size": [_P],
        "sa_sink_attn_weights": [_P] * 3 + [_S3, _S3] + [_I32] * 8 + [_F32, _P, _P, _SIZE, _P],
    }
    for name, types in signatures.items():
        fn = getattr(lib, name)
        fn.argtypes = types
        fn.restype = ctypes.c_int


def _size_of(name: str, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(name, getattr(_lib(), name)(*map(_int, args), ctypes.byref(out)))
    return int(out.value)


def _scale(softmax_scale, d: int) -> float:
    return d ** -0.5 if softmax_scale is None else float(softmax_scale)


def _bytes(size: int, like):
    return _s.torch.empty(size, dtype=_s.torch.uint8, device=like.device)


# A decoding step is a few microseconds of GPU work, so what the checks of its tensors' shapes and strides come to
# (sizes, stride arrays, workspace) is kept by these, in the `_plan` functions below; each call looks at types and
# devices.

def _layouts(**tensors) -> list:
    """Stride arrays of bf16 rows given as name=(shape, strides), or the ValueError that names one of them."""
    out = []
    for name, (shape, strides) in tensors.items():
        if len(shape) != 4:
            raise ValueError(f"{name}: expected a bfloat16 [batch, tokens, heads, head_dim] tensor")
        if strides[3] != 1:
            raise ValueError(f"{name}: head_dim must be contiguous")
        layout = _s._layout(strides, shape)
        if type(layout) is str:
            raise ValueError(f"{name}: {layout}")
        out.append(layout)
    return out


def _blame(dev: int, **tensors):
    """Raises for the tensor that is not bf16 rows on the current device."""
    for name, t in tensors.items():
        if t.dtype is not _s._BF16:
            raise ValueError(f"{name}: expected a bfloat16 [batch, tokens, heads, head_dim] tensor")
        if t.get_device() != dev:
            _s._elsewhere(name)


def _expect(name: str, shape, want):
    if shape != want:
        raise ValueError(f"{name}: expected shape {tuple(want)}, got {tuple(shape)}")


def _cache_dims(name: str, shape):
    if len(shape) != 4:
        raise ValueError(f"{name}: expected a bfloat16 [batch, capacity, kv_heads, head_dim] tensor")
    return shape


# ------------------------------------------------------------------ attention behind a shared prefix

def _prefix(k_prefix, v_prefix, kv_heads: int, d: int, dev: int):
    """Addresses and strides of the prefix's rows, and their number."""
    if len(k_prefix.shape) != 4 or k_prefix.shape[0] != 1 or k_prefix.shape[2] != kv_heads or k_prefix.shape[3] != d:
        raise ValueError(f"k_prefix: expected a [1, prefix tokens, {kv_heads}, {d}] tensor, got {tuple(k_prefix.shape)}")
    if k_prefix.shape[1] == 0 and v_prefix.shape == k_prefix.shape and k_prefix.dtype == v_prefix.dtype == _s._BF16:
        return (0, 0), (_NO_ROWS, _NO_ROWS), 0           # an empty tensor's strides may be anything
    return (k_prefix.data_ptr(), v_prefix.data_ptr()), (
        _rows("k_prefix", k_prefix, dev), _rows("v_prefix", v_prefix, dev, k_prefix.shape)), k_prefix.shape[1]


def sa_prefix_attn_fwd_workspace_size(batch: int, n_tokens: int, prefix_tokens: int, heads: int, kv_heads: int,
                                      head_dim: int, window: int) -> int:
    return _size_of("sa_prefix_attn_fwd_workspace_size", batch, n_tokens, prefix_tokens, heads, kv_heads, head_dim, window)


def sa_prefix_attn_decode_workspace_size(batch: int, prefix_tokens: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return _size_of("sa_prefix_attn_decode_workspace_size", batch, prefix_tokens, heads, kv_heads, head_dim)


_fwd_bytes = functools.lru_cache(maxsize=64)(sa_prefix_attn_fwd_workspace_size)


def sa_prefix_attn_fwd(q, k_prefix, v_prefix, k, v, window: int, o, lse, workspace, softmax_scale: float | None = None,
                       stream=None) -> None:
    """``k_prefix``, ``v_prefix``: bf16 [1, prefix tokens, kv_heads, head_dim]; ``k``, ``v``: the rows of q's tokens."""
    dev = _device()
    strides = _rows("q", q, dev), _rows("k", k, dev), _rows("v", v, dev, k.shape)
    _s._same_sequence(q, k)
    b, n, h, d = q.shape
    hk = k.shape[2]
    pre, pre_strides, p = _prefix(k_prefix, v_prefix, hk, d, dev)
    _check("sa_prefix_attn_fwd", _lib().sa_prefix_attn_fwd(
        q.data_ptr(), *pre, k.data_ptr(), v.data_ptr(), strides[0], *pre_strides, *strides[1:], _rows("o", o, dev, q.shape),
        b, n, p, h, hk, d, _int(window), _scale(softmax_scale, d), o.data_ptr(),
        _flat("lse", lse, _s.torch.float32, (b, h, n), dev), *_workspace(workspace, dev), _stream(stream, dev)))


def prefix_attn_fwd(q, k_prefix, v_prefix, k, v, window: int, softmax_scale: float | None = None):
    """Returns (o, lse): every query sees the whole prefix and, of its own sequence, itself and the
    `window` tokens before it."""
    dev = _device()
    strides = _rows("q", q, dev), _rows("k", k, dev), _rows("v", v, dev, k.shape)
    _s._same_sequence(q, k)
    b, n, h, d = q.shape
    hk = k.shape[2]
    pre, pre_strides, p = _prefix(k_prefix, v_prefix, hk, d, dev)
    size = _fwd_bytes(b, n, p, h, hk, d, window)
    o = _like(q)
    lse = _s.torch.empty((b, h, n), dtype=_s.torch.float32, device=q.device)
    ws = _bytes(size, q)
    _check("sa_prefix_attn_fwd", _lib().sa_prefix_attn_fwd(
        q.data_ptr(), *pre, k.data_ptr(), v.data_ptr(), strides[0], *pre_strides, *strides[1:], _dense(q.shape), b, n, p, h,
        hk, d, _int(window), _scale(softmax_scale, d), o.data_ptr(), lse.data_ptr(), ws.data_ptr(), size, _stream(None, dev)))
    return o, lse


def _one_token(shape, b: int, d: int) -> int:
    if len(shape) != 4 or shape[0] != b or shape[1] != 1 or shape[3] != d:
        raise ValueError("q: expected one token per sequence, [batch, 1, heads, head_dim]")
    return shape[2]


@functools.lru_cache(maxsize=256)
def _decode_plan(q, q_st, kp, kp_st, vp, vp_st, k, k_st, v, v_st):
    """Sizes, the inputs' strides, o's where it is allocated here, and the workspace's bytes."""
    b, cap, hk, d = _cache_dims("k_cache", k)
    h = _one_token(q, b, d)
    _expect("v_cache", v, k)
    if len(kp) != 4 or kp[0] != 1 or kp[2:] != (hk, d):
        raise ValueError(f"k_prefix: expected a [1, prefix tokens, {hk}, {d}] tensor, got {tuple(kp)}")
    _expect("v_prefix", vp, kp)
    qs, ks, vs = _layouts(q=(q, q_st), k_cache=(k, k_st), v_cache=(v, v_st))
    # (an empty tensor's strides may be anything)
    kps, vps = _layouts(k_prefix=(kp, kp_st), v_prefix=(vp, vp_st)) if kp[1] else (_NO_ROWS, _NO_ROWS)
    return (b, kp[1], cap, h, hk, d), (qs, kps, vps, ks, vs), _dense(q), \
        sa_prefix_attn_decode_workspace_size(b, kp[1], h, hk, d), (b,), d ** -0.5


def _decode_call(q, k_prefix, v_prefix, k_cache, v_cache, lengths, dev):
    if not (q.dtype is k_prefix.dtype is v_prefix.dtype is k_cache.dtype is v_cache.dtype is _s._BF16 and
            q.get_device() == k_prefix.get_device() == v_prefix.get_device() == k_cache.get_device() ==
            v_cache.get_device() == dev):
        _blame(dev, q=q, k_prefix=k_prefix, v_prefix=v_prefix, k_cache=k_cache, v_cache=v_cache)
    plan = _decode_plan(q.shape, q.stride(), k_prefix.shape, k_prefix.stride(), v_prefix.shape, v_prefix.stride(),
                        k_cache.shape, k_cache.stride(), v_cache.shape, v_cache.stride())
    return plan, (q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()), \
        _flat("lengths", lengths, _s.torch.int32, plan[4], dev)


def sa_prefix_attn_decode(q, k_prefix, v_prefix, k_cache, v_cache, lengths, window: int, o, lse, workspace,
                          softmax_scale: float | None = None, stream=None) -> None:
    """``lengths``: int32 [batch] on the device, own tokens in each cache with the query's own key."""
    dev = _device()
    (sizes, strides, _, _, _, scale), inputs, n = _decode_call(q, k_prefix, v_prefix, k_cache, v_cache, lengths, dev)
    _check("sa_prefix_attn_decode", _lib().sa_prefix_attn_decode(
        *inputs, *strides, _rows("o", o, dev, q.shape), *sizes, n, _int(window),
        scale if softmax_scale is None else float(softmax_scale), o.data_ptr(),
        _flat("lse", lse, _s.torch.float32, (sizes[0], sizes[3], 1), dev), *_workspace(workspace, dev), _stream(stream, dev)))


def prefix_attn_decode(q, k_prefix, v_prefix, k_cache, v_cache, lengths, window: int, softmax_scale: float | None = None):
    """One token per sequence behind a shared prefix; returns (o [batch, 1, heads, head_dim], lse)."""
    dev = _device()
    (sizes, strides, os, size, _, scale), inputs, n = _decode_call(q, k_prefix, v_prefix, k_cache, v_cache, lengths, dev)
    o, lse = _s._token_outputs(q)
    ws = _bytes(size, q)
    _check("sa_prefix_attn_decode", _lib().sa_prefix_attn_decode(
        *inputs, *strides, os, *sizes, n, _int(window), scale if softmax_scale is None else float(softmax_scale),
        o.data_ptr(), lse.data_ptr(), ws.data_ptr(), size, _stream(None, dev)))
    return o, lse


# ------------------------------------------------------------------ a cache of slots with accumulated weights

class ScoredCache(NamedTuple):
    """Keys and values bfloat16 [batch, capacity, kv_heads, head_dim], with the attention weight that each
    row has gathered (fp32) and its token (int32), both [batch, kv_heads, capacity]."""
    k: object
    v: object
    weights: object
    positions: object


def scored_alloc(batch: int, capacity: int, kv_heads: int, head_dim: int, device="cuda") -> ScoredCache:
    """An empty cache (rows are undefined until they are appended)."""
    import torch
    rows = [torch.empty((batch, capacity, kv_heads, head_dim), dtype=torch.bfloat16, device=device) for _ in range(2)]
    return ScoredCache(*rows, torch.zeros((batch, kv_heads, capacity), dtype=torch.float32, device=device),
                       torch.zeros((batch, kv_heads, capacity), dtype=torch.int32, device=device))


@functools.lru_cache(maxsize=256)
def _cache_plan(k, k_st, v, v_st):
    """Sizes and strides of a cache's rows, and its weights' shape."""
    b, cap, hk, d = _cache_dims("k", k)
    _expect("v", v, k)
    return (b, hk, d, cap), tuple(_layouts(k=(k, k_st), v=(v, v_st))), (b, hk, cap), (b,)


def _scored(cache, dev):
    """Plan and addresses of a cache."""
    k, v, w, pos = cache
    if not (k.dtype is v.dtype is _s._BF16 and k.get_device() == v.get_device() == dev):
        _blame(dev, k=k, v=v)
    plan = _cache_plan(k.shape, k.stride(), v.shape, v.stride())
    return plan, (k.data_ptr(), v.data_ptr()), _flat("weights", w, _s.torch.float32, plan[2], dev), \
        _flat("positions", pos, _s.torch.int32, plan[2], dev)


def sa_scored_append(cache: ScoredCache, k, v, start=None, tokens=None, stream=None) -> None:
    """Writes rows start[s] .. start[s] + n - 1 of every sequence with weight 0 and the positions tokens[s] ..
    (``start``, ``tokens``: int32 [batch] on the device; None: slot 0, and the slots' own numbers; a
    sequence with a negative start is left out)."""
    dev = _device()
    ((b, hk, d, cap), strides, _, batch), rows, w, pos = _scored(cache, dev)
    shape = k.shape
    ks, vs = _rows("k", k, dev), _rows("v", v, dev, shape)
    if shape[0] != b or shape[2] != hk or shape[3] != d:
        raise ValueError(f"k: expected rows of the cache's shape {(b, shape[1], hk, d)}, got {tuple(shape)}")
    i32 = _s.torch.int32
    _check("sa_scored_append", _lib().sa_scored_append(
        k.data_ptr(), v.data_ptr(), ks, vs, b, shape[1], hk, d, cap, _flat("start", start, i32, batch, dev),
        _flat("tokens", tokens, i32, batch, dev), *rows, *strides, w, pos, _stream(stream, dev)))


def scored_append(cache: ScoredCache, k, v, start=None, tokens=None) -> None:
    sa_scored_append(cache, k, v, start, tokens)


def sa_scored_attn_decode_workspace_size(batch: int, capacity: int, heads: int, kv_heads: int) -> int:
    return _size_of("sa_scored_attn_decode_workspace_size", batch, capacity, heads, kv_heads)


@functools.lru_cache(maxsize=256)
def _scored_plan(q, q_st, k, k_st, v, v_st):
    b, cap, hk, d = _cache_dims("k", k)
    h = _one_token(q, b, d)
    _expect("v", v, k)
    return (b, cap, h, hk, d), tuple(_layouts(q=(q, q_st), k=(k, k_st), v=(v, v_st))), _dense(q), \
        sa_scored_attn_decode_workspace_size(b, cap, h, hk), (b,), (b, hk, cap), d ** -0.5


def _scored_call(q, cache, lengths, weights_out, dev):
    k, v, w, _ = cache
    if not (q.dtype is k.dtype is v.dtype is _s._BF16 and q.get_device() == k.get_device() == v.get_device() == dev):
        _blame(dev, q=q, k=k, v=v)
    plan = _scored_plan(q.shape, q.stride(), k.shape, k.stride(), v.shape, v.stride())
    f32 = _s.torch.float32
    at = _flat("weights", w, f32, plan[5], dev)
    return plan, (q.data_ptr(), k.data_ptr(), v.data_ptr()), _flat("lengths", lengths, _s.torch.int32, plan[4], dev), \
        (at, at if weights_out is None else _flat("weights_out", weights_out, f32, plan[5], dev))


def sa_scored_attn_decode(q, cache: ScoredCache, lengths, o, lse, workspace, decay: float = 1.0, weights_out=None,
                          softmax_scale: float | None = None, stream=None) -> None:
    dev = _device()
    (sizes, strides, _, _, _, _, scale), inputs, n, weights = _scored_call(q, cache, lengths, weights_out, dev)
    _check("sa_scored_attn_decode", _lib().sa_scored_attn_decode(
        *inputs, *strides, _rows("o", o, dev, q.shape), *sizes, n, scale if softmax_scale is None else float(softmax_scale),
        float(decay), *weights, o.data_ptr(), _flat("lse", lse, _s.torch.float32, (sizes[0], sizes[2], 1), dev),
        *_workspace(workspace, dev), _stream(stream, dev)))


def scored_attn_decode(q, cache: ScoredCache, lengths, decay: float = 1.0, weights_out=None,
                       softmax_scale: float | None = None):
    """One token per sequence over the first lengths[s] slots; returns (o [batch, 1, heads, head_dim], lse).
    Every slot's weight becomes decay * weight + the sum of its probabilities over the query heads of its key
    head, in place or in ``weights_out``."""
    dev = _device()
    (sizes, strides, os, size, _, _, scale), inputs, n, weights = _scored_call(q, cache, lengths, weights_out, dev)
    o, lse = _s._token_outputs(q)
    ws = _bytes(size, q)
    _check("sa_scored_attn_decode", _lib().sa_scored_attn_decode(
        *inputs, *strides, os, *sizes, n, scale if softmax_scale is None else float(softmax_scale), float(decay), *weights,
        o.data_ptr(), lse.data_ptr(), ws.data_ptr(), size, _stream(None, dev)))
    return o, lse


def sa_scored_evict(cache: ScoredCache, lengths, keep: int, sinks: int, recent: int, weights_out, positions_out, lengths_out,
                    stream=None) -> None:
    dev = _device()
    ((b, hk, d, cap), strides, shape, batch), rows, w, pos = _scored(cache, dev)
    i32 = _s.torch.int32
    _check("sa_scored_evict", _lib().sa_scored_evict(
        *rows, *strides, b, hk, d, cap, _int(keep), _int(sinks), _int(recent), w, pos, _flat("lengths", lengths, i32, batch, dev),
        _flat("weights_out", weights_out, _s.torch.float32, shape, dev), _flat("positions_out", positions_out, i32, shape, dev),
        _flat("lengths_out", lengths_out, i32, batch, dev), _stream(stream, dev)))


def scored_evict(cache: ScoredCache, lengths, keep: int, sinks: int, recent: int, weights_out=None, positions_out=None,
                 lengths_out=None):
    """Leaves at most `keep` slots per sequence: those of the first `sinks` and the newest `recent` tokens, then the
    ones of most weight. Rows move within the cache; weights, positions and lengths are changed in
    place where no output is given. Returns (weights, positions, lengths)."""
    out = (cache[2] if weights_out is None else weights_out, cache[3] if positions_out is None else positions_out,
           lengths if lengths_out is None else lengths_out)
    sa_scored_evict(cache, lengths, keep, sinks, recent, *out)
    return out


def sa_sink_attn_weights_workspace_size() -> int:
    return _size_of("sa_sink_attn_weights_workspace_size")


def sa_sink_attn_weights(q, k, lse, window: int, sinks: int, weights, workspace, first_query: int = 0,
                         softmax_scale: float | None = None, stream=None) -> None:
    dev = _device()
    qs, ks = _rows("q", q, dev), _rows("k", k, dev)
    _s._same_sequence(q, k)
    b, n, h, d = q.shape
    hk, f32 = k.shape[2], _s.torch.float32
    _check("sa_sink_attn_weights", _lib().sa_sink_attn_weights(
        q.data_ptr(), k.data_ptr(), _flat("lse", lse, f32, (b, h, n), dev), qs, ks, b, n, h, hk, d, _int(window), _int(sinks),
        _int(first_query), _scale(softmax_scale, d), _flat("weights", weights, f32, (b, hk, n), dev),
        *_workspace(workspace, dev), _stream(stream, dev)))


def sink_attn_weights(q, k, lse, window: int, sinks: int, first_query: int = 0, softmax_scale: float | None = None):
    """The attention weight that each key gathers from queries first_query .. of sink_attn_fwd (with its lse),
    summed over them and over the query heads of its key head: fp32 [batch, kv_heads, tokens]."""
    at = _device()
    _rows("q", q, at)
    _rows("k", k, at)
    weights = _s.torch.empty((k.shape[0], k.shape[2], k.shape[1]), dtype=_s.torch.float32, device=k.device)
    sa_sink_attn_weights(q, k, lse, window, sinks, weights, _bytes(sa_sink_attn_weights_workspace_size(), q), first_query,
                         softmax_scale)
    return weights


NAMES = [
    "sa_prefix_attn_fwd", "sa_prefix_attn_fwd_workspace_size", "sa_prefix_attn_decode", "sa_prefix_attn_decode_workspace_size",
    "sa_scored_append", "sa_scored_attn_decode", "sa_scored_attn_decode_workspace_size", "sa_scored_evict",
    "sa_sink_attn_weights", "sa_sink_attn_weights_workspace_size",
    "prefix_attn_fwd", "prefix_attn_decode", "scored_alloc", "scored_append", "scored_attn_decode", "scored_evict",
    "sink_attn_weights", "ScoredCache",
]
__all__ = NAMES
