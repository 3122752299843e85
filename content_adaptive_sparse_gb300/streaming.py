"""Streaming attention: the calls around the sink-window graph (binding of sa_api.h's
"streaming attention" part; re-exported by the package).

Query i sees key j iff j <= i and (i - j <= window or j < sinks). ``sa_*`` functions carry the
C ABI's names and write into tensors that the caller gives; the others allocate their outputs
(and workspace) and make one call. Like the rest of the package this only marshals arguments: it
checks what the C side cannot see (types, shapes and devices of tensors) or could not name (strides)
and raises ``ValueError``, while the library's own refusals raise ``SAError``.
"""
from __future__ import annotations

import ctypes
import functools
import operator
from typing import NamedTuple

import numpy as np

_P, _I32, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
_S3 = ctypes.c_int64 * 3
_LIB = None
torch = None                  # imported by the first call (`_bind`): a tensor has come with it by then


def declare(lib) -> None:
    """Argument types of this module's entry points (called once, when the library is loaded)."""
    global _LIB
    sizes = [_I32] * 5
    rope = [_P, _P, _F32, _P, _I32, _I32, _P]          # weights, eps, frequencies, rotary, interleaved, positions
    axes = rope[:-1] + [_I32, _P, _P]                  # ..., interleaved, axes, axis of each pair, positions
    sink = [_I32] * 7 + [_F32]                         # batch, tokens, heads, kv_heads, dim, window, sinks; scale
    decode = [_I32] * 5 + [_P, _I32, _I32, _F32, _P, _P, _P]
    signatures = {
        "sa_qk_norm_rope_fwd": [_P, _P, _S3, _S3] + sizes + rope + [_P, _P, _S3, _S3, _P],
        "sa_qk_norm_rope_bwd_workspace_size": [_I32, _P],
        "sa_qk_norm_rope_bwd": [_P] * 4 + [_S3] * 4 + sizes + rope + [_P, _P, _S3, _S3, _P, _P, _P, ctypes.c_size_t, _P],
        "sa_qk_norm_rope_axes_fwd": [_P, _P, _S3, _S3] + sizes + axes + [_P, _P, _S3, _S3, _P],
        "sa_qk_norm_rope_axes_bwd": [_P] * 4 + [_S3] * 4 + sizes + axes + [_P, _P, _S3, _S3, _P, _P, _P, ctypes.c_size_t,
                                                                          _P],
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
    _LIB = lib


def _lib():
    if _LIB is None:
        from . import load_library
        load_library()
    return _LIB


def _check(name: str, code: int) -> None:
    if code != 0:
        from . import SAError
        raise SAError(name, code)


# ------------------------------------------------------------------ argument checks
#
# A decoding step is a few microseconds of GPU work, so the checks are single comparisons and the
# stride arrays are kept by their values. Each helper raises with the argument's name.

_MAX = 2**31 - 1
_TOO_LARGE = "sizes of 2^31 and more are not supported"


def _int(v: int) -> int:
    """`v` for a 32-bit argument, of which ctypes would drop the upper bits: past 32 bits the nearest number
    that fits, which the library takes or refuses as it would have taken `v` (its limits lie inside)."""
    return v if -_MAX <= v <= _MAX else _MAX if v > 0 else -_MAX


@functools.lru_cache(maxsize=1024)
def _s3(strides: tuple) -> _S3:
    return _S3(*strides[:3])


@functools.lru_cache(maxsize=1024)
def _layout(strides: tuple, shape: tuple):
    """Strides of a tensor, or what the library would refuse in it without naming the tensor."""
    if max(shape) > _MAX:
        return _TOO_LARGE
    if any(s <= 0 or s % 8 for s in strides[:3]):
        return "strides must be positive multiples of 8 elements (an expanded tensor needs .contiguous())"
    return _S3(*strides[:3])


@functools.lru_cache(maxsize=64)
def _frequencies(raw: bytes):
    """A host array of the doubles in `raw` (None for none). The caller passes the array itself, not its
    address, and so keeps it until its call is over: this cache may drop it meanwhile."""
    return (ctypes.c_double * (len(raw) // 8)).from_buffer_copy(raw) if raw else None


def _dense(shape) -> _S3:
    """Strides of a contiguous [batch, tokens, heads, head_dim] tensor."""
    _, n, h, d = shape
    return _s3((n * h * d, h * d, d))


def _bind() -> None:
    """Looks up once what every call needs: a lookup is as long as a check."""
    global torch, _BF16, _initialized, _current_device, _current_stream
    import torch as module
    _BF16 = module.bfloat16
    _initialized = module.cuda.is_initialized
    # torch.cuda.current_device() and current_stream().cuda_stream without their Python objects
    _current_device, _current_stream = module._C._cuda_getDevice, module._C._cuda_getCurrentRawStream
    torch = module                # last: another thread may be looking


def _device() -> int:
    if torch is None:
        _bind()
    return _current_device() if _initialized() else -2   # no tensor is there


def _rows(name: str, t, device: int, shape=None) -> _S3:
    """Strides of a bf16 [batch, tokens, heads, head_dim] tensor on the current device."""
    st = t.stride()
    if t.dtype is not _BF16 or len(st) != 4:
        raise ValueError(f"{name}: expected a bfloat16 [batch, tokens, heads, head_dim] tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if st[3] != 1:
        raise ValueError(f"{name}: head_dim must be contiguous")
    if t.get_device() != device:
        _elsewhere(name)
    layout = _layout(st, t.shape)
    if type(layout) is str:
        raise ValueError(f"{name}: {layout}")
    return layout


def _elsewhere(name: str):
    raise ValueError(f"{name}: expected a tensor on the current CUDA device")


def _flat(name: str, t, dtype, shape, device: int) -> int:
    """Address of a contiguous tensor of this type and shape (0 for None, which the library refuses
    where it needs the argument)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)}")
    if t.get_device() != device:
        _elsewhere(name)
    return t.data_ptr()


def _same_sequence(q, k) -> None:
    a, b = q.shape, k.shape
    if a[0] != b[0] or a[1] != b[1] or a[3] != b[3]:
        raise ValueError("q and k must agree in batch, tokens and head_dim")


def _graph(window: int, sinks: int, softmax_scale, d: int) -> tuple[int, int, float]:
    return _int(window), _int(sinks), d ** -0.5 if softmax_scale is None else float(softmax_scale)


def _stream(stream, device: int) -> int:
    if stream is not None:
        return stream.cuda_stream
    return _current_stream(device)


def _workspace(ws, device: int) -> tuple[int, int]:
    if ws.get_device() != device:
        _elsewhere("workspace")
    if not ws.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


# ------------------------------------------------------------------ norm and rotation of queries and keys

@functools.lru_cache(maxsize=64)
def _axes(pair_axes: tuple):
    """A host array of the pairs' axes (kept by the caller, as `_frequencies`)."""
    if any(not -_MAX <= a <= _MAX for a in pair_axes):
        raise ValueError("pair_axes: expected axes of the positions")
    return (ctypes.c_int32 * len(pair_axes))(*pair_axes) if pair_axes else None


def _rope_args(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, dev, pair_axes=None):
    qs, ks = _rows("q", q, dev), _rows("k", k, dev)
    _same_sequence(q, k)
    b, n, h, d = q.shape
    if type(inv_freq) is not np.ndarray or inv_freq.dtype != np.float64:
        inv_freq = np.asarray(inv_freq, dtype=np.float64)
    if inv_freq.ndim != 1:
        raise ValueError("inv_freq: expected one frequency per rotated pair")
    freq = _frequencies(inv_freq.tobytes())
    f32 = torch.float32
    if pair_axes is None:
        places = (_flat("positions", positions, torch.int32, (b, n), dev),)
    else:
        try:
            axes = tuple(map(operator.index, pair_axes))
        except TypeError:
            raise ValueError("pair_axes: expected a sequence of whole numbers") from None
        if len(axes) != inv_freq.size:
            raise ValueError("pair_axes: expected one axis per frequency")
        if positions is None or len(positions.shape) != 3:
            raise ValueError("positions: expected an int32 [batch, tokens, axes] tensor")
        a = positions.shape[2]
        places = (_int(a), _axes(axes), _flat("positions", positions, torch.int32, (b, n, a), dev))
    return (q.data_ptr(), k.data_ptr()), (qs, ks), (
        b, n, h, k.shape[2], d, _flat("q_weight", q_weight, f32, (d,), dev), _flat("k_weight", k_weight, f32, (d,), dev),
        eps, freq, _int(2 * inv_freq.size), 1 if interleaved else 0, *places)


def sa_qk_norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out, eps: float = 1e-6,
                        interleaved: bool = False, stream=None) -> None:
    """RMS norm and rotation of q and k into q_out and k_out (which may be q and k). ``inv_freq``:
    host sequence of one frequency per rotated pair, radians per position; weights (fp32 [head_dim])
    and ``positions`` (int32 [batch, tokens]) may be None."""
    dev = _device()
    ptrs, strides, args = _rope_args(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, dev)
    _check("sa_qk_norm_rope_fwd", _lib().sa_qk_norm_rope_fwd(
        *ptrs, *strides, *args, q_out.data_ptr(), k_out.data_ptr(), _rows("q_out", q_out, dev, q.shape),
        _rows("k_out", k_out, dev, k.shape), _stream(stream, dev)))


def sa_qk_norm_rope_bwd_workspace_size(head_dim: int) -> int:
    out = ctypes.c_size_t(0)
    _check("sa_qk_norm_rope_bwd_workspace_size",
           _lib().sa_qk_norm_rope_bwd_workspace_size(_int(head_dim), ctypes.byref(out)))
    return int(out.value)


def sa_qk_norm_rope_bwd(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, positions, dq, dk, dq_weight, dk_weight,
                        workspace, eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """Gradients of sa_qk_norm_rope_fwd; the weights' (fp32 [head_dim]) may be None."""
    dev = _device()
    ptrs, strides, args = _rope_args(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, dev)
    d = (q.shape[3],)
    _check("sa_qk_norm_rope_bwd", _lib().sa_qk_norm_rope_bwd(
        *ptrs, d_q_out.data_ptr(), d_k_out.data_ptr(), *strides, _rows("d_q_out", d_q_out, dev, q.shape),
        _rows("d_k_out", d_k_out, dev, k.shape), *args, dq.data_ptr(), dk.data_ptr(), _rows("dq", dq, dev, q.shape),
        _rows("dk", dk, dev, k.shape), _flat("dq_weight", dq_weight, torch.float32, d, dev),
        _flat("dk_weight", dk_weight, torch.float32, d, dev), *_workspace(workspace, dev), _stream(stream, dev)))


def qk_norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, positions=None, eps: float = 1e-6, interleaved: bool = False):
    """Returns (q_out, k_out), contiguous."""
    dev = _device()
    ptrs, strides, args = _rope_args(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, dev)
    q_out, k_out = _like(q), _like(k)
    _check("sa_qk_norm_rope_fwd", _lib().sa_qk_norm_rope_fwd(
        *ptrs, *strides, *args, q_out.data_ptr(), k_out.data_ptr(), _dense(q.shape), _dense(k.shape), _stream(None, dev)))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, positions=None, eps: float = 1e-6,
                     interleaved: bool = False):
    """Returns (dq, dk, dq_weight, dk_weight); a weight given as None has the gradient None."""
    at = _device()
    _rows("q", q, at)
    _rows("k", k, at)
    d, dev = q.shape[3], q.device
    dq, dk = _like(q), _like(k)
    dqw = None if q_weight is None else torch.empty(d, dtype=torch.float32, device=dev)
    dkw = None if k_weight is None else torch.empty(d, dtype=torch.float32, device=dev)
    ws = torch.empty(sa_qk_norm_rope_bwd_workspace_size(d), dtype=torch.uint8, device=dev)
    sa_qk_norm_rope_bwd(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, positions, dq, dk, dqw, dkw, ws, eps,
                        interleaved)
    return dq, dk, dqw, dkw


# with a position per axis (time, height, width): `pair_axes` is a host sequence of one axis per rotated
# pair, `positions` int32 [batch, tokens, axes]

def sa_qk_norm_rope_axes_fwd(q, k, q_weight, k_weight, inv_freq, pair_axes, positions, q_out, k_out, eps: float = 1e-6,
                             interleaved: bool = False, stream=None) -> None:
    """sa_qk_norm_rope_fwd with pair p turned by positions[..., pair_axes[p]] * inv_freq[p]."""
    dev = _device()
    ptrs, strides, args = _rope_args(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, dev, pair_axes)
    _check("sa_qk_norm_rope_axes_fwd", _lib().sa_qk_norm_rope_axes_fwd(
        *ptrs, *strides, *args, q_out.data_ptr(), k_out.data_ptr(), _rows("q_out", q_out, dev, q.shape),
        _rows("k_out", k_out, dev, k.shape), _stream(stream, dev)))


def sa_qk_norm_rope_axes_bwd(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, pair_axes, positions, dq, dk, dq_weight,
                             dk_weight, workspace, eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """Gradients of sa_qk_norm_rope_axes_fwd; the weights' (fp32 [head_dim]) may be None."""
    dev = _device()
    ptrs, strides, args = _rope_args(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, dev, pair_axes)
    d = (q.shape[3],)
    _check("sa_qk_norm_rope_axes_bwd", _lib().sa_qk_norm_rope_axes_bwd(
        *ptrs, d_q_out.data_ptr(), d_k_out.data_ptr(), *strides, _rows("d_q_out", d_q_out, dev, q.shape),
        _rows("d_k_out", d_k_out, dev, k.shape), *args, dq.data_ptr(), dk.data_ptr(), _rows("dq", dq, dev, q.shape),
        _rows("dk", dk, dev, k.shape), _flat("dq_weight", dq_weight, torch.float32, d, dev),
        _flat("dk_weight", dk_weight, torch.float32, d, dev), *_workspace(workspace, dev), _stream(stream, dev)))


def qk_norm_rope_axes_fwd(q, k, q_weight, k_weight, inv_freq, pair_axes, positions, eps: float = 1e-6,
                          interleaved: bool = False):
    """Returns (q_out, k_out), contiguous."""
    dev = _device()
    ptrs, strides, args = _rope_args(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, dev, pair_axes)
    q_out, k_out = _like(q), _like(k)
    _check("sa_qk_norm_rope_axes_fwd", _lib().sa_qk_norm_rope_axes_fwd(
        *ptrs, *strides, *args, q_out.data_ptr(), k_out.data_ptr(), _dense(q.shape), _dense(k.shape), _stream(None, dev)))
    return q_out, k_out


def qk_norm_rope_axes_bwd(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, pair_axes, positions, eps: float = 1e-6,
                          interleaved: bool = False):
    """Returns (dq, dk, dq_weight, dk_weight); a weight given as None has the gradient None."""
    at = _device()
    _rows("q", q, at)
    _rows("k", k, at)
    d, dev = q.shape[3], q.device
    dq, dk = _like(q), _like(k)
    dqw = None if q_weight is None else torch.empty(d, dtype=torch.float32, device=dev)
    dkw = None if k_weight is None else torch.empty(d, dtype=torch.float32, device=dev)
    ws = torch.empty(sa_qk_norm_rope_bwd_workspace_size(d), dtype=torch.uint8, device=dev)
    sa_qk_norm_rope_axes_bwd(q, k, d_q_out, d_k_out, q_weight, k_weight, inv_freq, pair_axes, positions, dq, dk, dqw, dkw,
                             ws, eps, interleaved)
    return dq, dk, dqw, dkw


# ------------------------------------------------------------------ sink-window attention

def _sink_inputs(q, k, v, dev):
    strides = _rows("q", q, dev), _rows("k", k, dev), _rows("v", v, dev, k.shape)
    _same_sequence(q, k)
    return (q.data_ptr(), k.data_ptr(), v.data_ptr()), strides


def sa_sink_attn_fwd(q, k, v, window: int, sinks: int, o, lse, softmax_scale: float | None = None, stream=None) -> None:
    dev = _device()
    ptrs, strides = _sink_inputs(q, k, v, dev)
    b, n, h, d = q.shape
    _check("sa_sink_attn_fwd", _lib().sa_sink_attn_fwd(
        *ptrs, *strides, _rows("o", o, dev, q.shape), b, n, h, k.shape[2], d, *_graph(window, sinks, softmax_scale, d),
        o.data_ptr(), _flat("lse", lse, torch.float32, (b, h, n), dev), _stream(stream, dev)))


def sa_sink_attn_bwd_workspace_size(batch: int, n_tokens: int, heads: int, kv_heads: int, head_dim: int, window: int,
                                    sinks: int) -> int:
    out = ctypes.c_size_t(0)
    sizes = map(_int, (batch, n_tokens, heads, kv_heads, head_dim, window, sinks))
    _check("sa_sink_attn_bwd_workspace_size", _lib().sa_sink_attn_bwd_workspace_size(*sizes, ctypes.byref(out)))
    return int(out.value)


_sink_bwd_bytes = functools.lru_cache(maxsize=64)(sa_sink_attn_bwd_workspace_size)


def sa_sink_attn_bwd(q, k, v, o, d_o, lse, window: int, sinks: int, dq, dk, dv, workspace,
                     softmax_scale: float | None = None, stream=None) -> None:
    dev = _device()
    ptrs, strides = _sink_inputs(q, k, v, dev)
    b, n, h, d = q.shape
    _check("sa_sink_attn_bwd", _lib().sa_sink_attn_bwd(
        *ptrs, o.data_ptr(), d_o.data_ptr(), _flat("lse", lse, torch.float32, (b, h, n), dev), *strides,
        _rows("o", o, dev, q.shape), _rows("d_o", d_o, dev, q.shape), b, n, h, k.shape[2], d,
        *_graph(window, sinks, softmax_scale, d), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _rows("dq", dq, dev, q.shape),
        _rows("dk", dk, dev, k.shape), _rows("dv", dv, dev, k.shape), *_workspace(workspace, dev), _stream(stream, dev)))


def sink_attn_fwd(q, k, v, window: int, sinks: int, softmax_scale: float | None = None):
    """Returns (o, lse): causal attention over the `window` keys before each query, itself and the
    first `sinks` tokens."""
    dev = _device()
    ptrs, strides = _sink_inputs(q, k, v, dev)
    b, n, h, d = q.shape
    o = _like(q)
    lse = torch.empty((b, h, n), dtype=torch.float32, device=q.device)
    _check("sa_sink_attn_fwd", _lib().sa_sink_attn_fwd(
        *ptrs, *strides, _dense(q.shape), b, n, h, k.shape[2], d, *_graph(window, sinks, softmax_scale, d),
        o.data_ptr(), lse.data_ptr(), _stream(None, dev)))
    return o, lse


def sink_attn_bwd(q, k, v, o, lse, d_o, window: int, sinks: int, softmax_scale: float | None = None):
    """Returns (dq, dk, dv) from sink_attn_fwd's inputs and outputs."""
    dev = _device()
    ptrs, strides = _sink_inputs(q, k, v, dev)
    b, n, h, d = q.shape
    hk = k.shape[2]
    os, gs = _rows("o", o, dev, q.shape), _rows("d_o", d_o, dev, q.shape)
    lse_at = _flat("lse", lse, torch.float32, (b, h, n), dev)
    dq, dk, dv = _like(q), _like(k), _like(v)
    size = _sink_bwd_bytes(b, n, h, hk, d, window, sinks)
    ws = torch.empty(size, dtype=torch.uint8, device=q.device)
    kv = _dense(k.shape)
    _check("sa_sink_attn_bwd", _lib().sa_sink_attn_bwd(
        *ptrs, o.data_ptr(), d_o.data_ptr(), lse_at, *strides, os, gs, b, n, h, hk, d,
        *_graph(window, sinks, softmax_scale, d), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _dense(q.shape), kv, kv,
        ws.data_ptr(), size, _stream(None, dev)))
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


def _cache4(cache, dev):
    """Addresses of a cache's four tensors, and (batch, kv_heads, capacity, head_dim)."""
    kc, ks, vc, vs = cache
    codes = kc.shape
    if len(codes) != 4:
        raise ValueError("cache: expected codes of shape [batch, kv_heads, capacity, head_dim / 2]")
    if max(codes) > _MAX:
        raise ValueError(f"cache: {_TOO_LARGE}")
    b, hk, cap, half = codes
    scales = (b, hk, cap, half // 16)
    u8 = torch.uint8
    return (_flat("k_codes", kc, u8, codes, dev), _flat("k_scales", ks, _BF16, scales, dev),
            _flat("v_codes", vc, u8, codes, dev), _flat("v_scales", vs, _BF16, scales, dev)), (b, hk, cap, 2 * half)


def sa_cache4_append(cache: Cache4, k, v, start=None, stream=None) -> None:
    """Writes rows start[s] .. start[s] + n - 1 of every sequence (``start``: int32 [batch] on the
    device, None for 0; a negative one leaves its sequence out)."""
    dev = _device()
    at, (b, hk, cap, d) = _cache4(cache, dev)
    ks = _rows("k", k, dev)
    n = k.shape[1]
    if k.shape != (b, n, hk, d):
        raise ValueError(f"k: expected rows of the cache's shape {(b, n, hk, d)}, got {tuple(k.shape)}")
    _check("sa_cache4_append", _lib().sa_cache4_append(
        k.data_ptr(), v.data_ptr(), ks, _rows("v", v, dev, k.shape), b, n, hk, d, cap,
        _flat("start", start, torch.int32, (b,), dev), *at, _stream(stream, dev)))


def sa_cache4_read(cache: Cache4, start, k, v, stream=None) -> None:
    """Reads rows start[s] .. start[s] + n - 1 of every sequence into k and v."""
    dev = _device()
    at, (b, hk, cap, d) = _cache4(cache, dev)
    ks = _rows("k", k, dev)
    n = k.shape[1]
    if k.shape != (b, n, hk, d):
        raise ValueError(f"k: expected rows of the cache's shape {(b, n, hk, d)}, got {tuple(k.shape)}")
    _check("sa_cache4_read", _lib().sa_cache4_read(
        *at, b, n, hk, d, cap, _flat("start", start, torch.int32, (b,), dev), k.data_ptr(), v.data_ptr(), ks,
        _rows("v", v, dev, k.shape), _stream(stream, dev)))


def cache4_append(cache: Cache4, k, v, start=None) -> None:
    sa_cache4_append(cache, k, v, start)


def cache4_read(cache: Cache4, start, n_tokens: int):
    """Returns (k, v), bfloat16 [batch, n_tokens, kv_heads, head_dim]."""
    dev = _device()
    at, (b, hk, cap, d) = _cache4(cache, dev)
    if n_tokens > _MAX:
        raise ValueError(f"n_tokens: {_TOO_LARGE}")
    k = torch.empty((b, n_tokens, hk, d), dtype=torch.bfloat16, device=cache[0].device)
    v = torch.empty_like(k)
    st = _dense(k.shape)
    _check("sa_cache4_read", _lib().sa_cache4_read(
        *at, b, n_tokens, hk, d, cap, _flat("start", start, torch.int32, (b,), dev), k.data_ptr(), v.data_ptr(), st, st,
        _stream(None, dev)))
    return k, v


def _token(q, b: int, d: int, dev: int) -> _S3:
    st = _rows("q", q, dev)
    shape = q.shape
    if shape[0] != b or shape[1] != 1 or shape[3] != d:
        raise ValueError("q: expected one token per sequence, [batch, 1, heads, head_dim]")
    return st


def _token_outputs(q):
    return _like(q), torch.empty((q.shape[0], q.shape[2], 1), dtype=torch.float32, device=q.device)


def sa_sink_attn_decode(q, k_cache, v_cache, lengths, window: int, sinks: int, o, lse,
                        softmax_scale: float | None = None, stream=None) -> None:
    """``lengths``: int32 [batch] on the device, tokens in each cache with the query's own key."""
    dev = _device()
    if len(k_cache.shape) != 4:
        raise ValueError("k_cache: expected a bfloat16 [batch, capacity, kv_heads, head_dim] tensor")
    b, cap, hk, d = k_cache.shape
    qs, h = _token(q, b, d, dev), q.shape[2]
    _check("sa_sink_attn_decode", _lib().sa_sink_attn_decode(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), qs, _rows("k_cache", k_cache, dev),
        _rows("v_cache", v_cache, dev, k_cache.shape), _rows("o", o, dev, q.shape), b, cap, h, hk, d,
        _flat("lengths", lengths, torch.int32, (b,), dev), *_graph(window, sinks, softmax_scale, d), o.data_ptr(),
        _flat("lse", lse, torch.float32, (b, h, 1), dev), _stream(stream, dev)))


def sa_sink_attn_decode_cache4(q, cache: Cache4, lengths, window: int, sinks: int, o, lse,
                               softmax_scale: float | None = None, stream=None) -> None:
    dev = _device()
    at, (b, hk, cap, d) = _cache4(cache, dev)
    qs, h = _token(q, b, d, dev), q.shape[2]
    _check("sa_sink_attn_decode_cache4", _lib().sa_sink_attn_decode_cache4(
        q.data_ptr(), *at, qs, _rows("o", o, dev, q.shape), b, cap, h, hk, d,
        _flat("lengths", lengths, torch.int32, (b,), dev), *_graph(window, sinks, softmax_scale, d), o.data_ptr(),
        _flat("lse", lse, torch.float32, (b, h, 1), dev), _stream(stream, dev)))


def sink_attn_decode(q, k_cache, v_cache, lengths, window: int, sinks: int, softmax_scale: float | None = None):
    """One token per sequence over a bf16 cache; returns (o [batch, 1, heads, head_dim], lse)."""
    dev = _device()
    if len(k_cache.shape) != 4:
        raise ValueError("k_cache: expected a bfloat16 [batch, capacity, kv_heads, head_dim] tensor")
    b, cap, hk, d = k_cache.shape
    qs = _token(q, b, d, dev)
    o, lse = _token_outputs(q)
    _check("sa_sink_attn_decode", _lib().sa_sink_attn_decode(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), qs, _rows("k_cache", k_cache, dev),
        _rows("v_cache", v_cache, dev, k_cache.shape), _dense(q.shape), b, cap, q.shape[2], hk, d,
        _flat("lengths", lengths, torch.int32, (b,), dev), *_graph(window, sinks, softmax_scale, d), o.data_ptr(),
        lse.data_ptr(), _stream(None, dev)))
    return o, lse


def sink_attn_decode_cache4(q, cache: Cache4, lengths, window: int, sinks: int, softmax_scale: float | None = None):
    """One token per sequence over a 4-bit cache; returns (o [batch, 1, heads, head_dim], lse)."""
    dev = _device()
    at, (b, hk, cap, d) = _cache4(cache, dev)
    qs = _token(q, b, d, dev)
    o, lse = _token_outputs(q)
    _check("sa_sink_attn_decode_cache4", _lib().sa_sink_attn_decode_cache4(
        q.data_ptr(), *at, qs, _dense(q.shape), b, cap, q.shape[2], hk, d,
        _flat("lengths", lengths, torch.int32, (b,), dev), *_graph(window, sinks, softmax_scale, d), o.data_ptr(),
        lse.data_ptr(), _stream(None, dev)))
    return o, lse


NAMES = [
    "sa_qk_norm_rope_fwd", "sa_qk_norm_rope_bwd", "sa_qk_norm_rope_bwd_workspace_size", "sa_sink_attn_fwd",
    "sa_qk_norm_rope_axes_fwd", "sa_qk_norm_rope_axes_bwd", "qk_norm_rope_axes_fwd", "qk_norm_rope_axes_bwd",
    "sa_sink_attn_bwd", "sa_sink_attn_bwd_workspace_size", "sa_sink_attn_decode", "sa_sink_attn_decode_cache4",
    "sa_cache4_append", "sa_cache4_read",
    "qk_norm_rope_fwd", "qk_norm_rope_bwd", "sink_attn_fwd", "sink_attn_bwd", "sink_attn_decode",
    "sink_attn_decode_cache4", "cache4_alloc", "cache4_append", "cache4_read", "Cache4",
]
__all__ = NAMES
