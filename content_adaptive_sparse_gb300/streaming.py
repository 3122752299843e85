"""Streaming attention: the calls around the sink-window graph (binding of sa_api.h's
"streaming attention" part; re-exported by the package).

Query i sees key j iff j <= i and (i - j <= window or j < sinks). ``sa_*`` functions carry the
C ABI's names and write into tensors that the caller gives; the others allocate their outputs
(and workspace) and make one call. Like the rest of the package this only marshals arguments: it
checks what the C side cannot see (types, shapes and devices of tensors) and raises ``ValueError``,
while the library's own refusals raise ``SAError``.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import numpy as np

_P, _I32, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
_S3 = ctypes.c_int64 * 3


def declare(lib) -> None:
    """Argument types of this module's entry points (called once, when the library is loaded)."""
    sizes = [_I32] * 5
    rope = [_P, _P, _F32, _P, _I32, _I32, _P]          # weights, eps, frequencies, rotary, interleaved, positions
    sink = [_I32] * 7 + [_F32]                         # batch, tokens, heads, kv_heads, dim, window, sinks; scale
    decode = [_I32] * 5 + [_P, _I32, _I32, _F32, _P, _P, _P]
    signatures = {
        "sa_qk_norm_rope_fwd": [_P, _P, _S3, _S3] + sizes + rope + [_P, _P, _S3, _S3, _P],
        "sa_qk_norm_rope_bwd_workspace_size": [_I32, _P],
        "sa_qk_norm_rope_bwd": [_P] * 4 + [_S3] * 4 + sizes + rope + [_P, _P, _S3, _S3, _P, _P, _P, ctypes.c_size_t, _P],
        "sa_sink_attn_fwd": [_P] * 3 + [_S3] * 4 + sink + [_P, _P, _P],
        "sa_sink_attn_bwd_workspace_size": [_I32] * 7 + [_P],
        "sa_sink_attn_bwd": [_P] * 6 + [_S3] * 5 + sink + [_P] * 3 + [_S3] * 3 + [_P, ctypes.c_size_t, _P],
        "sa_sink_attn_decode": [_P] * 3 + [_S3] * 4 + decode,
        "sa_sink_attn_decode_cache4": [_P] * 5 + [_S3] * 2 + decode,
        "sa_cache4_append": [_P, _P, _S3, _S3] + sizes + [_P] * 6,
        "sa_cache4_read": [_P] * 4 + sizes + [_P, _P, _P, _S3, _S3, _P],
    }
    for name, types in signatures.items():
        fn = getattr(lib, name)
        fn.argtypes = types
        fn.restype = ctypes.c_int


def _lib():
    from . import load_library
    return load_library()


def _check(name: str, code: int) -> None:
    if code != 0:
        from . import SAError
        raise SAError(name, code)


# ------------------------------------------------------------------ argument checks

def _rows(name: str, t, shape=None) -> _S3:
    """Strides of a bf16 [batch, tokens, heads, head_dim] tensor on the current device."""
    import torch
    if t.dtype is not torch.bfloat16 or t.dim() != 4:
        raise ValueError(f"{name}: expected a bfloat16 [batch, tokens, heads, head_dim] tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"{name}: head_dim must be contiguous")
    _on_device(name, t)
    return _S3(st[0], st[1], st[2])


def _sizes(name: str, t):
    if t.dim() != 4:
        raise ValueError(f"{name}: expected a bfloat16 [batch, tokens, heads, head_dim] tensor")
    return t.shape


def _on_device(name: str, t) -> None:
    import torch
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: expected a tensor on the current CUDA device")


def _flat(name: str, t, dtype, shape) -> int:
    """Address of a contiguous tensor of this type and shape (0 for None)."""
    if t is None:              # a null pointer: refused by the library where the argument is needed
        return 0
    if t.dtype is not dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)}")
    _on_device(name, t)
    return t.data_ptr()


def _kv(k, v, shape=None) -> tuple[_S3, _S3]:
    return _rows("k", k, shape), _rows("v", v, k.shape)


def _same_sequence(q, k) -> None:
    if k.shape[0] != q.shape[0] or k.shape[1] != q.shape[1] or k.shape[3] != q.shape[3]:
        raise ValueError("q and k must agree in batch, tokens and head_dim")


def _scale(softmax_scale, d: int) -> float:
    return d ** -0.5 if softmax_scale is None else float(softmax_scale)


def _stream(stream) -> int:
    import torch
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _workspace(ws) -> tuple[int, int]:
    _on_device("workspace", ws)
    if not ws.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    return ws.data_ptr(), ws.numel() * ws.element_size()


# ------------------------------------------------------------------ norm and rotation of queries and keys

def _rope_args(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved):
    import torch
    qs, ks = _rows("q", q), _rows("k", k)
    _same_sequence(q, k)
    b, n, h, d = q.shape
    freq = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if freq.ndim != 1:
        raise ValueError("inv_freq: expected one frequency per rotated pair")
    tail = (_flat("q_weight", q_weight, torch.float32, (d,)), _flat("k_weight", k_weight, torch.float32, (d,)),
            float(eps), freq.ctypes.data if freq.size else 0, 2 * freq.size, int(bool(interleaved)),
            _flat("positions", positions, torch.int32, (b, n)))
    return qs, ks, (b, n, h, k.shape[2], d) + tail, freq        # freq: kept alive until the call returns


def sa_qk_norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out, eps: float = 1e-6,
                        interleaved: bool = False, stream=None) -> None:
    """RMS norm and rotation of q and k into q_out and k_out (which may be q and k). ``inv_freq``:
    host sequence of one frequency per rotated pair, radians per position; weights (fp32 [head_dim])
    and ``positions`` (int32 [batch, tokens]) may be None."""
    qs, ks, args, freq = _rope_args(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved)
    _check("sa_qk_norm_rope_fwd", _lib().sa_qk_norm_rope_fwd(
        q.data_ptr(), k.data_ptr(), qs, ks, *args, q_out.data_ptr(), k_out.data_ptr(), _rows("q_out", q_out, q.shape),
        _rows("k_out", k_out, k.shape), _stream(stream)))


def sa_qk_norm_rope_bwd_workspace_size(head_dim: int) -> int:
    out = ctypes.c_size_t(0)
    _check("sa_qk_norm_rope_bwd_workspace_size", _lib().sa_qk_norm_rope_bwd_workspace_size(head_dim, ctypes.byref(out)))
    return int(out.value)


def sa_qk_norm_rope_bwd(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, positions, dq, dk, dq_weight, dk_weight,
                        workspace, eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """Gradients of sa_qk_norm_rope_fwd; the weights' (fp32 [head_dim]) may be None."""
    import torch
    qs, ks, args, freq = _rope_args(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved)
    d = q.shape[3]
    ws, ws_bytes = _workspace(workspace)
    _check("sa_qk_norm_rope_bwd", _lib().sa_qk_norm_rope_bwd(
        q.data_ptr(), k.data_ptr(), d_q_out.data_ptr(), d_k_out.data_ptr(), qs, ks, _rows("d_q_out", d_q_out, q.shape),
        _rows("d_k_out", d_k_out, k.shape), *args, dq.data_ptr(), dk.data_ptr(), _rows("dq", dq, q.shape),
        _rows("dk", dk, k.shape), _flat("dq_weight", dq_weight, torch.float32, (d,)),
        _flat("dk_weight", dk_weight, torch.float32, (d,)), ws, ws_bytes, _stream(stream)))


def qk_norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, positions=None, eps: float = 1e-6, interleaved: bool = False):
    """Returns (q_out, k_out), contiguous."""
    import torch
    q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=k.device)
    sa_qk_norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out, eps, interleaved)
    return q_out, k_out


def qk_norm_rope_bwd(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, positions=None, eps: float = 1e-6,
                     interleaved: bool = False):
    """Returns (dq, dk, dq_weight, dk_weight); a weight given as None has the gradient None."""
    import torch
    d, dev = q.shape[-1], q.device
    dq, dk = torch.empty(q.shape, dtype=torch.bfloat16, device=dev), torch.empty(k.shape, dtype=torch.bfloat16, device=dev)
    dqw = None if q_weight is None else torch.empty(d, dtype=torch.float32, device=dev)
    dkw = None if k_weight is None else torch.empty(d, dtype=torch.float32, device=dev)
    ws = torch.empty(sa_qk_norm_rope_bwd_workspace_size(d), dtype=torch.uint8, device=dev)
    sa_qk_norm_rope_bwd(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, positions, dq, dk, dqw, dkw, ws, eps,
                        interleaved)
    return dq, dk, dqw, dkw


# ------------------------------------------------------------------ sink-window attention

def sa_sink_attn_fwd(q, k, v, window: int, sinks: int, o, lse, softmax_scale: float | None = None, stream=None) -> None:
    import torch
    qs, (ks, vs) = _rows("q", q), _kv(k, v)
    _same_sequence(q, k)
    b, n, h, d = q.shape
    _check("sa_sink_attn_fwd", _lib().sa_sink_attn_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, _rows("o", o, q.shape), b, n, h, k.shape[2], d, window, sinks,
        _scale(softmax_scale, d), o.data_ptr(), _flat("lse", lse, torch.float32, (b, h, n)), _stream(stream)))


def sa_sink_attn_bwd_workspace_size(batch: int, n_tokens: int, heads: int, kv_heads: int, head_dim: int, window: int,
                                    sinks: int) -> int:
    out = ctypes.c_size_t(0)
    _check("sa_sink_attn_bwd_workspace_size", _lib().sa_sink_attn_bwd_workspace_size(
        batch, n_tokens, heads, kv_heads, head_dim, window, sinks, ctypes.byref(out)))
    return int(out.value)


def sa_sink_attn_bwd(q, k, v, o, d_o, lse, window: int, sinks: int, dq, dk, dv, workspace,
                     softmax_scale: float | None = None, stream=None) -> None:
    import torch
    qs, (ks, vs) = _rows("q", q), _kv(k, v)
    _same_sequence(q, k)
    b, n, h, d = q.shape
    ws, ws_bytes = _workspace(workspace)
    _check("sa_sink_attn_bwd", _lib().sa_sink_attn_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), d_o.data_ptr(),
        _flat("lse", lse, torch.float32, (b, h, n)), qs, ks, vs, _rows("o", o, q.shape), _rows("d_o", d_o, q.shape), b, n, h,
        k.shape[2], d, window, sinks, _scale(softmax_scale, d), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
        _rows("dq", dq, q.shape), _rows("dk", dk, k.shape), _rows("dv", dv, k.shape), ws, ws_bytes, _stream(stream)))


def sink_attn_fwd(q, k, v, window: int, sinks: int, softmax_scale: float | None = None):
    """Returns (o, lse): causal attention over the `window` keys before each query, itself and the
    first `sinks` tokens."""
    import torch
    b, n, h, d = _sizes("q", q)
    o = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((b, h, n), dtype=torch.float32, device=q.device)
    sa_sink_attn_fwd(q, k, v, window, sinks, o, lse, softmax_scale)
    return o, lse


def sink_attn_bwd(q, k, v, o, lse, d_o, window: int, sinks: int, softmax_scale: float | None = None):
    """Returns (dq, dk, dv) from sink_attn_fwd's inputs and outputs."""
    import torch
    b, n, h, d = _sizes("q", q)
    dev = q.device
    dq = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
    dk, dv = torch.empty(k.shape, dtype=torch.bfloat16, device=dev), torch.empty(v.shape, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(sa_sink_attn_bwd_workspace_size(b, n, h, k.shape[2], d, window, sinks), dtype=torch.uint8, device=dev)
    sa_sink_attn_bwd(q, k, v, o, d_o, lse, window, sinks, dq, dk, dv, ws, softmax_scale)
    return dq, dk, dv


# ------------------------------------------------------------------ single tokens over a cache

class Cache4(NamedTuple):
    """Keys and values in 4 bits (layout: sa_api.h): codes uint8 [batch, kv_heads, capacity,
    head_dim / 2], scales bfloat16 [batch, kv_heads, capacity, head_dim / 32]."""
    k_codes: object
    k_scales: object
    v_codes: object
    v_scales: object


def cache4_alloc(batch: int, capacity: int, kv_heads: int, head_dim: int, device="cuda") -> Cache4:
    """An empty cache (rows are undefined until they are appended); capacity a multiple of 8."""
    import torch
    if capacity % 8 != 0 or head_dim % 32 != 0:
        raise ValueError("capacity must be a multiple of 8, head_dim of 32")

    def rows():
        return (torch.empty((batch, kv_heads, capacity, head_dim // 2), dtype=torch.uint8, device=device),
                torch.empty((batch, kv_heads, capacity, head_dim // 32), dtype=torch.bfloat16, device=device))
    return Cache4(*rows(), *rows())


def _cache4(cache) -> tuple[tuple[int, int, int, int], tuple[int, int, int, int]]:
    """Addresses of a cache's four tensors and (batch, kv_heads, capacity, head_dim)."""
    import torch
    kc, ks, vc, vs = cache
    if kc.dim() != 4:
        raise ValueError("cache: expected codes of shape [batch, kv_heads, capacity, head_dim / 2]")
    b, hk, cap, half = kc.shape
    scales = (b, hk, cap, half // 16)
    at = (_flat("k_codes", kc, torch.uint8, kc.shape), _flat("k_scales", ks, torch.bfloat16, scales),
          _flat("v_codes", vc, torch.uint8, kc.shape), _flat("v_scales", vs, torch.bfloat16, scales))
    return at, (b, hk, cap, 2 * half)


def sa_cache4_append(cache: Cache4, k, v, start=None, stream=None) -> None:
    """Writes rows start[s] .. start[s] + n - 1 of every sequence (``start``: int32 [batch] on the
    device, None for 0; a negative one leaves its sequence out)."""
    import torch
    at, (b, hk, cap, d) = _cache4(cache)
    ks, vs = _kv(k, v, (b, k.shape[1], hk, d))
    _check("sa_cache4_append", _lib().sa_cache4_append(
        k.data_ptr(), v.data_ptr(), ks, vs, b, k.shape[1], hk, d, cap, _flat("start", start, torch.int32, (b,)), *at,
        _stream(stream)))


def sa_cache4_read(cache: Cache4, start, k, v, stream=None) -> None:
    """Reads rows start[s] .. start[s] + n - 1 of every sequence into k and v."""
    import torch
    at, (b, hk, cap, d) = _cache4(cache)
    ks, vs = _kv(k, v, (b, k.shape[1], hk, d))
    _check("sa_cache4_read", _lib().sa_cache4_read(
        *at, b, k.shape[1], hk, d, cap, _flat("start", start, torch.int32, (b,)), k.data_ptr(), v.data_ptr(), ks, vs,
        _stream(stream)))


def cache4_append(cache: Cache4, k, v, start=None) -> None:
    sa_cache4_append(cache, k, v, start)


def cache4_read(cache: Cache4, start, n_tokens: int):
    """Returns (k, v), bfloat16 [batch, n_tokens, kv_heads, head_dim]."""
    import torch
    b, hk, _, half = cache[0].shape
    k = torch.empty((b, n_tokens, hk, 2 * half), dtype=torch.bfloat16, device=cache[0].device)
    v = torch.empty_like(k)
    sa_cache4_read(cache, start, k, v)
    return k, v


def _token(q, b: int, d: int) -> _S3:
    st = _rows("q", q)
    if q.shape[0] != b or q.shape[1] != 1 or q.shape[3] != d:
        raise ValueError("q: expected one token per sequence, [batch, 1, heads, head_dim]")
    return st


def sa_sink_attn_decode(q, k_cache, v_cache, lengths, window: int, sinks: int, o, lse,
                        softmax_scale: float | None = None, stream=None) -> None:
    """``lengths``: int32 [batch] on the device, tokens in each cache with the query's own key."""
    import torch
    ks, vs = _kv(k_cache, v_cache)
    b, cap, hk, d = k_cache.shape
    qs = _token(q, b, d)
    h = q.shape[2]
    _check("sa_sink_attn_decode", _lib().sa_sink_attn_decode(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), qs, ks, vs, _rows("o", o, q.shape), b, cap, h, hk, d,
        _flat("lengths", lengths, torch.int32, (b,)), window, sinks, _scale(softmax_scale, d), o.data_ptr(),
        _flat("lse", lse, torch.float32, (b, h, 1)), _stream(stream)))


def sa_sink_attn_decode_cache4(q, cache: Cache4, lengths, window: int, sinks: int, o, lse,
                               softmax_scale: float | None = None, stream=None) -> None:
    import torch
    at, (b, hk, cap, d) = _cache4(cache)
    qs = _token(q, b, d)
    h = q.shape[2]
    _check("sa_sink_attn_decode_cache4", _lib().sa_sink_attn_decode_cache4(
        q.data_ptr(), *at, qs, _rows("o", o, q.shape), b, cap, h, hk, d,
        _flat("lengths", lengths, torch.int32, (b,)), window, sinks, _scale(softmax_scale, d), o.data_ptr(),
        _flat("lse", lse, torch.float32, (b, h, 1)), _stream(stream)))


def _token_outputs(q):
    import torch
    b, _, h, d = _sizes("q", q)
    return (torch.empty((b, 1, h, d), dtype=torch.bfloat16, device=q.device),
            torch.empty((b, h, 1), dtype=torch.float32, device=q.device))


def sink_attn_decode(q, k_cache, v_cache, lengths, window: int, sinks: int, softmax_scale: float | None = None):
    """One token per sequence over a bf16 cache; returns (o [batch, 1, heads, head_dim], lse)."""
    o, lse = _token_outputs(q)
    sa_sink_attn_decode(q, k_cache, v_cache, lengths, window, sinks, o, lse, softmax_scale)
    return o, lse


def sink_attn_decode_cache4(q, cache: Cache4, lengths, window: int, sinks: int, softmax_scale: float | None = None):
    """One token per sequence over a 4-bit cache; returns (o [batch, 1, heads, head_dim], lse)."""
    o, lse = _token_outputs(q)
    sa_sink_attn_decode_cache4(q, cache, lengths, window, sinks, o, lse, softmax_scale)
    return o, lse


NAMES = [
    "sa_qk_norm_rope_fwd", "sa_qk_norm_rope_bwd", "sa_qk_norm_rope_bwd_workspace_size", "sa_sink_attn_fwd",
    "sa_sink_attn_bwd", "sa_sink_attn_bwd_workspace_size", "sa_sink_attn_decode", "sa_sink_attn_decode_cache4",
    "sa_cache4_append", "sa_cache4_read",
    "qk_norm_rope_fwd", "qk_norm_rope_bwd", "sink_attn_fwd", "sink_attn_bwd", "sink_attn_decode",
    "sink_attn_decode_cache4", "cache4_alloc", "cache4_append", "cache4_read", "Cache4",
]
__all__ = NAMES
