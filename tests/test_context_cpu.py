"""Shared contexts and bounded caches without a GPU: refusals of the C entry points and of the binding,
and pins of the float64 oracles."""
import ctypes

import numpy as np
import pytest

import content_adaptive_sparse_gb300 as sa
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
