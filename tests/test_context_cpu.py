"""Shared contexts and bounded caches without a GPU: refusals of the C entry points and of the binding,
and pins of the float64 oracles."""
import ctypes
import os
import shutil
import subprocess
import types

import numpy as np
import pytest

import content_adaptive_sparse_gb300 as sa
from oracle import context as oc
from oracle import streaming as ref
from test_streaming_cpu import A, CAPACITY, INVALID, P, S3, UNSUPPORTED, Call, lib, st  # noqa: F401


# ------------------------------------------------------------------ norm and rotation with several axes

@pytest.mark.parametrize("backward", [False, True])
def test_axes_refusals(lib, backward):  # noqa: F811
    freq = (ctypes.c_double * 32)(*[0.5] * 32)
    axes = (ctypes.c_int32 * 32)(*[p % 3 for p in range(32)])
    a = dict(q=A, k=A)
    if backward:
        a.update(dq_out=A, dk_out=A)
    a.update(qs=st(4, 64, 8), ks=st(2, 64, 8))
    if backward:
        a.update(gqs=st(4, 64, 8), gks=st(2, 64, 8))
    a.update(batch=2, n=8, heads=4, kv_heads=2, d=64, wq=A, wk=A, eps=1e-6, freq=ctypes.cast(freq, P), rotary=64, inter=0,
             axes=3, pair=ctypes.cast(axes, P), pos=A, qo=A, ko=A, qos=st(4, 64, 8), kos=st(2, 64, 8))
    if backward:
        a.update(dwq=A, dwk=A, ws=A, ws_bytes=0)         # too small: never valid
    a.update(stream=0)
    c = Call(lib, "sa_qk_norm_rope_axes_bwd" if backward else "sa_qk_norm_rope_axes_fwd", **a)
    for bad in (dict(q=0), dict(qo=0), dict(n=0), dict(eps=0.0), dict(inter=2), dict(rotary=80), dict(freq=None),
                dict(axes=0), dict(axes=-1), dict(axes=2), dict(pair=None), dict(pos=0)):
        assert c.with_(**bad) == INVALID, bad
    for x in (-1, 3, 1 << 30):
        axes[31] = x
        assert c.with_() == INVALID, x
    axes[31] = 0
    for bad in (dict(d=96), dict(rotary=24), dict(q=A + 8), dict(axes=9), dict(kos=S3(1024, 0, 64))):
        assert c.with_(**bad) == UNSUPPORTED, bad
    if backward:
        assert c.with_() == CAPACITY and c.with_(rotary=0, pair=None, freq=None) == CAPACITY
        assert c.with_(ws=0) == INVALID and c.with_(ws=A + 64) == UNSUPPORTED and c.with_(dk_out=A + 4) == UNSUPPORTED


def test_axes_binding_refuses(monkeypatch):
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(1, 4, 3, dtype=torch.int32)
    monkeypatch.setattr(sa.streaming, "_device", lambda: (sa.streaming._bind() if sa.streaming.torch is None else None, -1)[1])
    freq = [0.5] * 16
    for pair, p, what in (([0] * 15, pos, "pair_axes"), ([0] * 16, pos[..., 0], "positions"), ([0] * 16, None, "positions"),
                          ([0] * 16, pos.long(), "positions"), ([0] * 16, pos[:, :3], "positions"), ([1 << 40] * 16, pos, "pair_axes")):
        with pytest.raises(ValueError, match=what):
            sa.qk_norm_rope_axes_fwd(q, q, None, None, freq, pair, p)
        with pytest.raises(ValueError, match=what):
            sa.qk_norm_rope_axes_bwd(q, q, q, q, None, None, freq, pair, p)


@pytest.mark.parametrize("pair", [[0.5] * 16, [1.0] * 16, [None] * 16, ["0"] * 16])
def test_axes_binding_takes_whole_numbers(monkeypatch, pair):
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(1, 4, 3, dtype=torch.int32)
    monkeypatch.setattr(sa.streaming, "_device", lambda: (sa.streaming._bind() if sa.streaming.torch is None else None, -1)[1])
    with pytest.raises(sa.SAError):                       # the library's own answer, without a device
        sa.sa_qk_norm_rope_axes_fwd(q, q, None, None, [0.5] * 16, np.ones(16, np.int64), pos, q, q,
                                    stream=types.SimpleNamespace(cuda_stream=0))
    with pytest.raises(ValueError, match="pair_axes"):
        sa.qk_norm_rope_axes_fwd(q, q, None, None, [0.5] * 16, pair, pos)


@pytest.mark.parametrize("inter", [False, True])
def test_axes_oracle(inter):
    """Pairs with positions of their own, one pair at a time; gradients against differences."""
    rng = np.random.default_rng(0)
    d, axes = 32, 3
    x, w = rng.standard_normal((1, 2, 1, d)), rng.standard_normal(d)
    freq = 0.9 ** np.arange(d // 2)
    pair = rng.integers(0, axes, d // 2)
    pos = rng.integers(-9, 9, (1, 2, axes))
    y, _ = ref.norm_rope(x, w, pos[:, :, pair], freq, 1e-5, inter)
    for p in range(d // 2):
        a, b = (2 * p, 2 * p + 1) if inter else (p, p + d // 2)
        z = x[0, 1, 0] / np.sqrt((x[0, 1, 0] ** 2).mean() + 1e-5) * w
        turn = (z[a] + 1j * z[b]) * np.exp(1j * pos[0, 1, pair[p]] * freq[p])
        assert np.allclose([y[0, 1, 0, a], y[0, 1, 0, b]], [turn.real, turn.imag])
    dy = rng.standard_normal(x.shape)
    (dx, dw), _ = ref.norm_rope_backward(x, w, dy, pos[:, :, pair], freq, 1e-5, inter)
    f = lambda x, w: (dy * ref.norm_rope(x, w, pos[:, :, pair], freq, 1e-5, inter)[0]).sum()  # noqa: E731
    for e in (0, 5, 31):
        h = np.zeros_like(x)
        h[0, 1, 0, e] = 1e-6
        assert abs((f(x + h, w) - f(x - h, w)) / 2e-6 - dx[0, 1, 0, e]) < 1e-7
        h = np.zeros_like(w)
        h[e] = 1e-6
        assert abs((f(x, w + h) - f(x, w - h)) / 2e-6 - dw[e]) < 1e-7


# ------------------------------------------------------------------ refusals of the other calls

def prefix_call(lib, decode):  # noqa: F811
    tokens = 64 if decode else 8
    a = dict(q=A, kp=A, vp=A, k=A, v=A, qs=st(4, 64, 1 if decode else 8), kps=st(2, 64, 100), vps=st(2, 64, 100),
             ks=st(2, 64, tokens), vs=st(2, 64, tokens), os=st(4, 64, 1 if decode else 8), batch=2)
    a.update(dict(prefix=100, capacity=64) if decode else dict(n=8, prefix=100))
    a.update(heads=4, kv_heads=2, d=64)
    if decode:
        a.update(lengths=A)
    a.update(window=5, scale=0.125, o=A, lse=A, ws=A, ws_bytes=0, stream=0)      # no room: never valid
    return Call(lib, "sa_prefix_attn_decode" if decode else "sa_prefix_attn_fwd", **a)


@pytest.mark.parametrize("decode", [False, True])
def test_prefix_refusals(lib, decode):  # noqa: F811
    c = prefix_call(lib, decode)
    n = "capacity" if decode else "n"
    assert c.with_() == CAPACITY and c.with_(prefix=0, kp=None, vp=None, kps=S3(0, 0, 0), vps=S3(0, 0, 0)) == CAPACITY
    assert c.with_(kps=S3(0, 128, 64), vps=S3(-3, 128, 64)) == CAPACITY          # the batch stride is not used
    for bad in (dict(q=0), dict(kp=0), dict(vp=0), dict(k=0), dict(v=0), dict(o=0), dict(lse=0), dict(ws=0), dict(batch=0),
                {n: 0}, dict(prefix=-1), dict(heads=0), dict(heads=3), dict(window=-1),
                dict(scale=0.0), dict(scale=float("nan")), dict(scale=2.4e38)):
        assert c.with_(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(q=A + 8), dict(kp=A + 8), dict(vp=A + 2), dict(k=A + 8), dict(o=A + 4), dict(ws=A + 128),
                dict(kps=S3(1, 0, 64)), dict(vps=S3(12800, 128, 60)), dict(ks=S3(1, 128, 64)), dict(vs=S3(4096, -128, 64)),
                dict(prefix=(1 << 30) + 1), {n: (1 << 30) + 1}):
        assert c.with_(**bad) == UNSUPPORTED, bad
    if decode:
        assert c.with_(lengths=None) == INVALID and c.with_(batch=70000) == UNSUPPORTED
    else:
        assert c.with_(batch=1 << 23) == UNSUPPORTED and c.with_(n=(1 << 24) + 1) == UNSUPPORTED


def test_prefix_workspace_sizes(lib):  # noqa: F811
    """Nothing but a small block where the items write the result; else D + 2 floats for every row and part."""
    assert sa.sa_prefix_attn_fwd_workspace_size(4, 8192, 0, 16, 4, 128, 4095) == 256
    assert sa.sa_prefix_attn_fwd_workspace_size(1, 8192, 57344, 16, 4, 128, 4095) == 256
    assert sa.sa_prefix_attn_decode_workspace_size(64, 32768, 16, 4, 128) == 152 * 128 * (128 + 2) * 4
    assert sa.sa_prefix_attn_decode_workspace_size(64, 0, 16, 4, 128) == 256
    joint = sa.sa_prefix_attn_fwd_workspace_size(32, 37, 16384, 16, 4, 128, 36)
    assert joint == 4 * 37 * 2 * 128 * (128 + 2) * 4
    for bad in ((0, 8, 8, 4, 2, 64, 3), (1, 0, 8, 4, 2, 64, 3), (1, 8, -1, 4, 2, 64, 3), (1, 8, 8, 3, 2, 64, 3), (1, 8, 8, 4, 2, 80, 3),
                (1, 8, 8, 4, 2, 64, -1)):
        with pytest.raises(sa.SAError):
            sa.sa_prefix_attn_fwd_workspace_size(*bad)
    with pytest.raises(sa.SAError):
        sa.sa_prefix_attn_decode_workspace_size(1, 8, 4, 3, 64)


def test_scored_append_refusals(lib):  # noqa: F811
    a = dict(k=A, v=A, ks=st(2, 64, 4), vs=st(2, 64, 4), batch=2, n=4, kv_heads=2, d=64, capacity=64, start=0, tokens=0, kc=A, vc=A,
             kcs=st(2, 64, 64), vcs=st(2, 64, 64), w=A, pos=A, stream=0)
    c = Call(lib, "sa_scored_append", **a)
    for bad in (dict(k=0), dict(v=0), dict(kc=0), dict(vc=0), dict(w=0), dict(pos=0), dict(batch=0),
                dict(n=0), dict(kv_heads=0), dict(capacity=0)):
        assert c.with_(**bad) == INVALID, bad
    for bad in (dict(d=48), dict(k=A + 8), dict(vc=A + 4), dict(vs=S3(512, 128, 60)), dict(kcs=S3(8192, 0, 64)), dict(batch=32768),
                dict(capacity=(1 << 20) + 1), dict(n=1 << 26, kv_heads=4)):
        assert c.with_(**bad) == UNSUPPORTED, bad


def test_scored_decode_refusals(lib):  # noqa: F811
    a = dict(q=A, k=A, v=A, qs=st(4, 64, 1), ks=st(2, 64, 64), vs=st(2, 64, 64), os=st(4, 64, 1), batch=2, capacity=64, heads=4,
             kv_heads=2, d=64, lengths=A, scale=0.125, decay=1.0, w=A, wo=A, o=A, lse=A, ws=A, ws_bytes=0, stream=0)
    c = Call(lib, "sa_scored_attn_decode", **a)
    assert c.with_() == CAPACITY and c.with_(decay=0.0) == CAPACITY
    for bad in (dict(q=0), dict(k=0), dict(lengths=None), dict(w=0), dict(wo=0), dict(o=0), dict(lse=0), dict(ws=0), dict(batch=0),
                dict(capacity=0), dict(heads=5), dict(scale=-1.0), dict(decay=-0.1), dict(decay=1.01), dict(decay=float("nan"))):
        assert c.with_(**bad) == INVALID, bad
    for bad in (dict(d=80), dict(q=A + 8), dict(ws=A + 64), dict(ks=S3(8192, 128, 63)), dict(capacity=(1 << 20) + 1),
                dict(heads=258, kv_heads=2), dict(batch=32768)):
        assert c.with_(**bad) == UNSUPPORTED, bad
    # scores of the query heads, a power of two of floats a row, 16 of them at a time
    for heads, kv_heads, floats in ((4, 2, 2), (3, 1, 4), (12, 1, 16), (16, 1, 16), (40, 2, 32), (256, 2, 128)):
        assert sa.sa_scored_attn_decode_workspace_size(3, 100, heads, kv_heads) == 3 * kv_heads * 100 * floats * 4
    for bad in ((0, 8, 4, 2), (1, 0, 4, 2), (1, 8, 5, 2), (1, 8, 258, 2), (1, (1 << 20) + 1, 4, 2)):
        with pytest.raises(sa.SAError):
            sa.sa_scored_attn_decode_workspace_size(*bad)


def test_scored_evict_refusals(lib):  # noqa: F811
    a = dict(k=A, v=A, ks=st(2, 64, 64), vs=st(2, 64, 64), batch=2, kv_heads=2, d=64, capacity=64, keep=32, sinks=4, recent=8, w=A,
             pos=A, n=A, wo=A, po=A, no=0, stream=0)                              # no lengths out: never valid
    c = Call(lib, "sa_scored_evict", **a)
    more = dict(no=A)
    for bad in (dict(k=0), dict(v=0), dict(w=0), dict(pos=0), dict(n=0), dict(wo=0), dict(po=0), dict(no=0), dict(keep=0),
                dict(keep=-3), dict(sinks=-1), dict(recent=-1), dict(sinks=20, recent=13), dict(sinks=2**31 - 1, recent=2**31 - 1),
                dict(batch=0), dict(capacity=0)):
        assert c.with_(**{**more, **bad}) == INVALID, bad
    for bad in (dict(d=96), dict(k=A + 8), dict(vs=S3(8192, 128, 4)), dict(capacity=(1 << 20) + 1), dict(batch=32768),
                dict(kv_heads=65536)):
        assert c.with_(**{**more, **bad}) == UNSUPPORTED, bad


def test_sink_weights_refusals(lib):  # noqa: F811
    a = dict(q=A, k=A, lse=A, qs=st(4, 64, 100), ks=st(2, 64, 100), batch=2, n=100, heads=4, kv_heads=2, d=64, window=10, sinks=4,
             first=0, scale=0.125, w=A, ws=A, ws_bytes=0, stream=0)
    c = Call(lib, "sa_sink_attn_weights", **a)
    assert c.with_() == CAPACITY and c.with_(first=99) == CAPACITY
    for bad in (dict(q=0), dict(k=0), dict(lse=0), dict(w=0), dict(ws=0), dict(batch=0), dict(n=0), dict(heads=3), dict(window=-1),
                dict(sinks=-1), dict(first=-1), dict(first=100), dict(scale=0.0), dict(scale=2.4e38)):
        assert c.with_(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(sinks=129), dict(n=(1 << 24) + 1), dict(q=A + 8), dict(ks=S3(1, 128, 64)), dict(ws=A + 64),
                dict(scale=1e-31)):
        assert c.with_(**bad) == UNSUPPORTED, bad
    assert sa.sa_sink_attn_weights_workspace_size() > 0


# ------------------------------------------------------------------ the binding

@pytest.fixture
def binding(monkeypatch):
    """Host tensors count as the current device's, so that the checks of shapes, strides and types are reached."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(sa.streaming, "_device", lambda: -1)
    monkeypatch.setattr(sa.context, "_device", lambda: -1)
    if sa.streaming.torch is None:
        sa.streaming._bind()
    return torch


def test_decoding_calls_refuse_wrong_tensors(binding):
    torch = binding
    bf = torch.bfloat16
    q, k, kp = torch.zeros(2, 1, 4, 64, dtype=bf), torch.zeros(2, 8, 2, 64, dtype=bf), torch.zeros(1, 9, 2, 64, dtype=bf)
    n = torch.zeros(2, dtype=torch.int32)
    for args, what in (((q.float(), kp, kp, k, k, n), "q: expected a bfloat16"), ((q, kp, kp.half(), k, k, n), "v_prefix: expected a bf"),
                       ((q[:1], kp, kp, k, k, n), "q: expected one token"), ((q, kp, kp, k, k[:, :7], n), "v_cache: expected shape"),
                       ((q, kp, kp, k[0], k, n), "k_cache: expected a bf"), ((q, k, k, k, k, n), "k_prefix: expected a .1, prefix"),
                       ((q, kp, kp[:, :5], k, k, n), "v_prefix: expected shape"), ((q, kp[:, :, :1], kp, k, k, n), "k_prefix"),
                       ((q, kp, kp, k, k, n.long()), "lengths"), ((q, kp, kp, k, k, n[:1]), "lengths"),
                       ((q, kp, kp, k.transpose(2, 3).contiguous().transpose(2, 3), k, n), "k_cache: head_dim"),
                       ((q, kp, kp, k[:, :1].expand(2, 8, 2, 64), k, n), "k_cache: strides"),
                       ((q, kp[:, :1].expand(1, 9, 2, 64), kp, k, k, n), "k_prefix: strides")):
        with pytest.raises(ValueError, match=what):
            sa.prefix_attn_decode(*args, 7)
    cache = sa.scored_alloc(2, 8, 2, 64, device="cpu")
    for c, args, what in ((cache._replace(k=k.float()), (q, n), "k: expected a bf"), (cache._replace(v=k[:, :7]), (q, n), "v: expected shape"),
                          (cache._replace(weights=cache.weights[:, :, :7]), (q, n), "weights"), (cache, (q[:, :, :, :32], n), "q: expected one"),
                          (cache, (q, n[:1]), "lengths"), (cache._replace(weights=cache.weights.double()), (q, n), "weights")):
        with pytest.raises(ValueError, match=what):
            sa.scored_attn_decode(args[0], c, args[1])
    with pytest.raises(ValueError, match="weights_out"):
        sa.scored_attn_decode(q, cache, n, 1.0, cache.weights[:1])


def test_cache_calls_refuse_wrong_tensors(binding):
    torch = binding
    cache = sa.scored_alloc(2, 8, 2, 64, device="cpu")
    k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    for args, what in (((k.float(), k), "k: expected a bf"), ((k, k[:, :2]), "v: expected shape"), ((k[:1], k[:1]), "k: expected rows"),
                       ((k[:, :, :1], k[:, :, :1]), "k: expected rows"), ((k, k, n.long()), "start"), ((k, k, n, n[:1]), "tokens")):
        with pytest.raises(ValueError, match=what):
            sa.scored_append(cache, *args)
    for c, args, what in ((cache._replace(positions=cache.positions.long()), (n,), "positions"), (cache, (n[:1],), "lengths"),
                          (cache._replace(weights=cache.weights.transpose(1, 2).contiguous().transpose(1, 2)), (n,), "weights")):
        with pytest.raises(ValueError, match=what):
            sa.scored_evict(c, *args, 4, 0, 0)
    for out, what in ((dict(weights_out=cache.weights[:1]), "weights_out"), (dict(positions_out=cache.weights), "positions_out"),
                      (dict(lengths_out=n.long()), "lengths_out")):
        with pytest.raises(ValueError, match=what):
            sa.scored_evict(cache, n, 4, 0, 0, **out)


def test_prompt_calls_refuse_wrong_tensors(binding):
    torch = binding
    q, k = torch.zeros(2, 5, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)
    kp = torch.zeros(1, 9, 2, 64, dtype=torch.bfloat16)
    for args, what in (((q, kp, kp, k[:, :4], k[:, :4]), "agree"), ((q, kp, kp, k, k[:, :4]), "v: expected shape"),
                       ((q, k, k, k, k), "k_prefix"), ((q, kp, kp[:, :1], k, k), "v_prefix: expected shape"), ((q.float(), kp, kp, k, k), "q")):
        with pytest.raises(ValueError, match=what):
            sa.prefix_attn_fwd(*args, 4)
    lse = torch.zeros(2, 4, 5)
    for args, what in (((q, k[:, :4], lse), "agree"), ((q, k, lse[:, :, :4]), "lse"), ((q, k, lse.double()), "lse"), ((q, k.float(), lse), "k")):
        with pytest.raises(ValueError, match=what):
            sa.sink_attn_weights(*args, 4, 0)


def test_tensors_elsewhere_are_refused():
    torch = pytest.importorskip("torch")
    q, k, kp = (torch.zeros(1, x, 2, 64, dtype=torch.bfloat16) for x in (1, 8, 9))
    n = torch.zeros(1, dtype=torch.int32)
    cache = sa.scored_alloc(1, 8, 2, 64, device="cpu")
    for call in (lambda: sa.prefix_attn_decode(q, kp, kp, k, k, n, 7), lambda: sa.prefix_attn_fwd(k, kp, kp, k, k, 7),
                 lambda: sa.scored_attn_decode(q, cache, n), lambda: sa.scored_append(cache, k, k), lambda: sa.scored_evict(cache, n, 4, 0, 0),
                 lambda: sa.sink_attn_weights(k, k, torch.zeros(1, 2, 8), 4, 0)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


# ------------------------------------------------------------------ pins of the oracle

def rows(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_prefix_oracle_is_attention_over_the_whole_sequence():
    """A prefix and own tokens of one sequence are that sequence; decoding is its last row."""
    p, n, h, hk, d, w = 7, 9, 4, 2, 32, 100
    q, k, v = rows(1, p + n, h, d), rows(1, p + n, hk, d, seed=1), rows(1, p + n, hk, d, seed=2)
    whole, lse, _ = ref.sink_attention(q, k, v, w, 0)
    o, l, _ = oc.prefix_attention(q[:, p:], k[:, :p], v[:, :p], k[:, p:], v[:, p:], w)
    assert np.allclose(o, whole[:, p:]) and np.allclose(l, lse[:, :, p:])
    o, l, _ = oc.prefix_decode(q[:, -1:], k[:, :p], v[:, :p], k[:, p:], v[:, p:], [n], w)
    assert np.allclose(o, whole[:, -1:]) and np.allclose(l, lse[:, :, -1:])
    # a window over the own tokens alone: the prefix takes the place of the sinks
    whole, lse, _ = ref.sink_attention(q, k, v, 2, p)
    o, l, _ = oc.prefix_attention(q[:, p:], k[:, :p], v[:, :p], k[:, p:], v[:, p:], 2)
    assert np.allclose(o, whole[:, p:]) and np.allclose(l, lse[:, :, p:])


def test_scored_oracle_and_prompt_weights_agree():
    """Tokens decoded one by one over a growing cache give the weights of the prompt at once."""
    n, h, hk, d = 11, 4, 2, 32
    q, k, v = rows(1, n, h, d), rows(1, n, hk, d, seed=1), rows(1, n, hk, d, seed=2)
    whole, lse, _ = ref.sink_attention(q, k, v, n, 0)
    w = np.zeros((1, hk, n))
    for i in range(n):
        o, l, _, w, _ = oc.scored_decode(q[:, i:i + 1], k, v, [i + 1], w, 1.0)
        assert np.allclose(o[:, 0], whole[:, i]) and np.allclose(l[:, :, 0], lse[:, :, i])
    got, _ = oc.sink_weights(q, k, lse, n, 0, 0)
    assert np.allclose(got, w) and np.isclose(w.sum(), n * h)
    late, _ = oc.sink_weights(q, k, lse, n, 0, 8)
    assert np.isclose(late.sum(), 3 * h)


def test_eviction_oracle():
    k = np.arange(6.0).reshape(1, 6, 1, 1)
    w = np.array([[[5.0, 1.0, 3.0, 3.0, 2.0, 0.5]]])
    pos = np.array([[[0, 10, 11, 12, 13, 14]]])
    # token 14 is recent; of the rest weights 5, 3, 3 stay: the equal ones are slots 2 and 3
    k2, v2, w2, p2, n2 = oc.evict(k, -k, w, pos, [6], 4, 0, 1)
    assert k2[0, :, 0, 0].tolist() == [0, 5, 2, 3, 4, 5] and (v2 == -k2).all() and n2 == [4]
    assert w2[0, 0].tolist() == [5, 0.5, 3, 3, 2, 0.5] and p2[0, 0].tolist() == [0, 14, 11, 12, 13, 14]
    # ties at the border go to the lower slot
    assert oc.evict(k, k, w, pos, [6], 2, 0, 0)[3][0, 0, :2].tolist() == [0, 11]
    # a list that is short enough stays
    assert oc.evict(k, k, w, pos, [3], 4, 0, 1)[4] == [3]


# ------------------------------------------------------------------ the selection of an eviction

def test_the_border_of_an_eviction_is_found(tmp_path):
    """key_range.h, as the kernel uses it, over random keys, many of them the largest (NaN), against sorted keys."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    here = os.path.dirname(os.path.abspath(__file__))
    exe = tmp_path / "key_range"
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", os.path.join(os.path.dirname(here), "content_adaptive_sparse_gb300", "csrc"),
                    os.path.join(here, "c", "key_range.cpp"), "-o", str(exe)], check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout
