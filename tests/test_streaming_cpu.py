"""Streaming attention without a GPU: refusals of the C entry points and of the binding, and pins of
the float64 oracle."""
import ctypes
import functools

import numpy as np
import pytest

import content_adaptive_sparse_gb300 as sa
from oracle import streaming as ref

INVALID, UNSUPPORTED, CAPACITY = -1, -2, -3
P = ctypes.c_void_p
S3 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def lib():
    sa.build_library()
    return sa.load_library()


# Stand-in addresses: every call below is refused before anything reads them.
A = 1 << 20


class Call:
    """A call with named arguments in their C order; `with_` gives the status with some replaced."""

    def __init__(self, lib, name, **args):
        self.fn, self.args = getattr(lib, name), args

    def with_(self, **changes):
        assert set(changes) <= set(self.args)
        return self.fn(*{**self.args, **changes}.values())


def st(heads, d, tokens):
    return S3(tokens * heads * d, heads * d, d)


def rope(lib, backward):
    freq = (ctypes.c_double * 32)(*[0.5] * 32)
    a = dict(q=A, k=A)
    if backward:
        a.update(dq_out=A, dk_out=A)
    a.update(qs=st(4, 64, 8), ks=st(2, 64, 8))
    if backward:
        a.update(gqs=st(4, 64, 8), gks=st(2, 64, 8))
    a.update(batch=2, n=8, heads=4, kv_heads=2, d=64, wq=A, wk=A, eps=1e-6, freq=ctypes.cast(freq, P), rotary=64, inter=0,
             pos=0, qo=A, ko=A, qos=st(4, 64, 8), kos=st(2, 64, 8))
    if backward:
        a.update(dwq=A, dwk=A, ws=A, ws_bytes=0)         # too small: never valid
    a.update(stream=0)
    c = Call(lib, "sa_qk_norm_rope_bwd" if backward else "sa_qk_norm_rope_fwd", **a)
    c.keep = freq
    return c


@pytest.mark.parametrize("backward", [False, True])
def test_norm_rope_refusals(lib, backward):
    c = rope(lib, backward)
    for bad in (dict(q=0), dict(k=0), dict(qo=0), dict(batch=0), dict(n=-1), dict(heads=0),
                dict(kv_heads=0), dict(eps=0.0), dict(eps=float("nan")), dict(inter=2), dict(rotary=-16), dict(rotary=80),
                dict(freq=None)):
        assert c.with_(**bad) == INVALID, bad
    for f in (-0.1, 6.3, float("nan"), float("inf")):
        c.keep[31] = f
        assert c.with_() == INVALID, f
    c.keep[31] = 0.5
    for bad in (dict(d=48, rotary=32), dict(d=256), dict(rotary=24), dict(q=A + 8), dict(ko=A + 2), dict(qs=S3(2048, 256, 60)),
                dict(kos=S3(1024, 0, 64)), dict(batch=1 << 15, n=1 << 15), dict(heads=65536)):
        assert c.with_(**bad) == UNSUPPORTED, bad
    if backward:
        assert c.with_() == CAPACITY
        assert c.with_(ws=0) == INVALID and c.with_(dq_out=0) == INVALID
        assert c.with_(ws=A + 64) == UNSUPPORTED and c.with_(dk_out=A + 4) == UNSUPPORTED
    assert sa.sa_qk_norm_rope_bwd_workspace_size(128) >= 2 * 128 * 4
    with pytest.raises(sa.SAError):
        sa.sa_qk_norm_rope_bwd_workspace_size(96)


def sink(lib, backward):
    a = dict(q=A, k=A, v=A)
    if backward:
        a.update(o=A, d_o=A, lse=A)
    a.update(qs=st(4, 64, 100), ks=st(2, 64, 100), vs=st(2, 64, 100), os=st(4, 64, 100))
    if backward:
        a.update(dos=st(4, 64, 100))
    a.update(batch=2, n=100, heads=4, kv_heads=2, d=64, window=10, sinks=4, scale=0.125)
    if backward:
        a.update(dq=A, dk=A, dv=A, dqs=st(4, 64, 100), dks=st(2, 64, 100), dvs=st(2, 64, 100), ws=A, ws_bytes=0, stream=0)
    else:
        a.update(o=A, lse=0, stream=0)                   # no LSE: never valid
    return Call(lib, "sa_sink_attn_bwd" if backward else "sa_sink_attn_fwd", **a)


@pytest.mark.parametrize("backward", [False, True])
def test_sink_attention_refusals(lib, backward):
    c = sink(lib, backward)
    more = {} if backward else {"lse": A}
    for bad in (dict(q=0), dict(k=0), dict(v=0), dict(o=0), dict(batch=0), dict(n=0), dict(heads=0),
                dict(heads=3), dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(scale=float("nan")),
                dict(scale=float("inf"))):
        assert c.with_(**{**more, **bad}) == INVALID, bad
    for bad in (dict(d=96), dict(sinks=129), dict(n=(1 << 24) + 1), dict(q=A + 8), dict(v=A + 2), dict(o=A + 4),
                dict(ks=S3(1, 128, 64)), dict(vs=S3(12800, -128, 64)), dict(os=S3(25600, 256, 4)), dict(batch=1 << 23, heads=4),
                dict(batch=1 << 10, heads=64, kv_heads=2, n=1 << 20)):
        assert c.with_(**{**more, **bad}) == UNSUPPORTED, bad
    if backward:
        for bad in (dict(d_o=0), dict(dq=0), dict(dk=0), dict(dv=0),                     dict(ws=0), dict(lse=0)):
            assert c.with_(**bad) == INVALID, bad
        for bad in (dict(d_o=A + 8), dict(dq=A + 8), dict(dk=A + 8), dict(dv=A + 8), dict(ws=A + 128), dict(dvs=S3(1, 1, 1)),
                    dict(batch=1, heads=2048, n=(1 << 20) - 127)):
            assert c.with_(**bad) == UNSUPPORTED, bad


def test_sink_workspace_size(lib):
    """D and LSE padded to whole tiles, and the sinks' partial sums where queries lie past the window."""
    rows = 2 * 4 * 128 * 4
    assert sa.sa_sink_attn_bwd_workspace_size(1, 1, 4, 2, 64, 0, 4) == rows
    assert sa.sa_sink_attn_bwd_workspace_size(1, 128, 4, 2, 64, 5, 0) == rows
    assert sa.sa_sink_attn_bwd_workspace_size(1, 129, 4, 2, 64, 5, 4) == 2 * rows
    big = sa.sa_sink_attn_bwd_workspace_size(1, 4096, 4, 2, 64, 127, 4)
    # tiles 2 .. 31 of the first key tile's queries in 4 chunks of 8, besides its ordinary item
    assert big == 32 * rows + 2 * 5 * 2 * 4 * 64 * 4
    for bad in ((0, 1, 4, 2, 64, 5, 4), (1, 1, 3, 2, 64, 5, 4), (1, 1, 4, 2, 64, -1, 4), (1, 1, 4, 2, 64, 5, 129)):
        with pytest.raises(sa.SAError):
            sa.sa_sink_attn_bwd_workspace_size(*bad)


def test_scales_that_overflow_in_log2_units(lib):
    """2.4e38 log2(e) is no fp32 number; 2.3e38 log2(e) is, and the next check refuses the call."""
    for backward in (False, True):
        c = sink(lib, backward)
        more = {"d": 96} if backward else {"d": 96, "lse": A}
        assert c.with_(scale=2.4e38, **more) == INVALID and c.with_(scale=2.3e38, **more) == UNSUPPORTED
    a = dict(q=A, k=A, v=A, qs=st(4, 64, 1), kst=st(2, 64, 64), vst=st(2, 64, 64), os=st(4, 64, 1), batch=2, capacity=64, heads=4,
             kv_heads=2, d=80, lengths=A, window=10, sinks=4, scale=0.125, o=A, lse=A, stream=0)
    c = Call(lib, "sa_sink_attn_decode", **a)
    assert c.with_(scale=2.4e38) == INVALID and c.with_(scale=2.3e38) == UNSUPPORTED


def test_sink_workspace_size_refuses_what_the_backward_refuses(lib):
    c = sink(lib, True)
    for batch, n, heads, kv_heads, d, s in ((1, (1 << 20) - 127, 2048, 2, 64, 4), (1, 1 << 24, 128, 128, 32, 0),
                                            (1, (1 << 24) + 1, 4, 2, 64, 4), (1, 8, 4, 2, 96, 4), (1, 8, 4, 2, 64, 129)):
        assert c.with_(batch=batch, n=n, heads=heads, kv_heads=kv_heads, d=d, sinks=s) == UNSUPPORTED
        with pytest.raises(sa.SAError) as e:
            sa.sa_sink_attn_bwd_workspace_size(batch, n, heads, kv_heads, d, 10, s)
        assert e.value.code == UNSUPPORTED
    # one tile less is taken (and then misses a device, or its workspace)
    assert c.with_(batch=1, n=(1 << 24) - 128, heads=128, kv_heads=128, d=32) in (CAPACITY, -4)
    assert sa.sa_sink_attn_bwd_workspace_size(1, (1 << 24) - 128, 128, 128, 32, 10, 0) == 2 * 4 * 128 * ((1 << 24) - 128)


@pytest.mark.parametrize("cache4", [False, True])
def test_decode_refusals(lib, cache4):
    a = dict(q=A, k=A, ks=A, v=A, vs=A) if cache4 else dict(q=A, k=A, v=A)
    a.update(qs=st(4, 64, 1))
    if not cache4:
        a.update(kst=st(2, 64, 64), vst=st(2, 64, 64))
    a.update(os=st(4, 64, 1), batch=2, capacity=64, heads=4, kv_heads=2, d=64, lengths=A, window=10, sinks=4, scale=0.125,
             o=A, lse=0, stream=0)                       # no LSE: never valid
    c = Call(lib, "sa_sink_attn_decode_cache4" if cache4 else "sa_sink_attn_decode", **a)
    for bad in (dict(q=0), dict(k=0), dict(v=0), dict(lengths=None), dict(o=0), dict(batch=0),
                dict(capacity=0), dict(heads=5), dict(window=-1), dict(sinks=-2), dict(scale=-1.0), dict()):
        assert c.with_(**{"lse": A if bad else 0, **bad}) == INVALID, bad
    for bad in (dict(d=80), dict(sinks=200), dict(q=A + 8), dict(k=A + 8), dict(o=A + 8), dict(qs=S3(4, 64, 64)),
                dict(os=S3(256, 256, 4)), dict(batch=70000), dict(capacity=(1 << 30) + 8), dict(heads=80000, kv_heads=80000)):
        assert c.with_(**{"lse": A, **bad}) == UNSUPPORTED, bad
    if cache4:
        for bad in (dict(ks=0), dict(vs=0)):
            assert c.with_(lse=A, **bad) == INVALID
        for bad in (dict(ks=A + 8), dict(capacity=60)):
            assert c.with_(lse=A, **bad) == UNSUPPORTED
    else:
        assert c.with_(lse=A, vst=S3(8192, 128, 63)) == UNSUPPORTED


@pytest.mark.parametrize("read", [False, True])
def test_cache4_refusals(lib, read):
    rows = dict(k=A, v=A, kst=st(2, 64, 4), vst=st(2, 64, 4))
    cache = dict(kc=A, ks=A, vc=A, vs=A)
    sizes = dict(batch=2, n=4, kv_heads=2, d=64, capacity=64, start=0)
    a = {**cache, **sizes, **rows} if read else {**rows, **sizes, **cache}
    c = Call(lib, "sa_cache4_read" if read else "sa_cache4_append", **a, stream=0)
    for bad in (dict(k=0), dict(v=0), dict(kc=0), dict(ks=0), dict(vc=0), dict(vs=0), dict(batch=0),
                dict(n=0), dict(kv_heads=0), dict(capacity=0)):
        assert c.with_(**bad) == INVALID, bad
    for bad in (dict(d=16), dict(capacity=60), dict(capacity=(1 << 30) + 8), dict(k=A + 8), dict(vc=A + 4), dict(vs=A + 2),
                dict(vst=S3(512, 128, 60)), dict(n=1 << 25, kv_heads=16), dict(batch=40000)):
        assert c.with_(**bad) == UNSUPPORTED, bad


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        sa.sink_attn_fwd(q, q, q, 1, 1)
    with pytest.raises(ValueError, match="bfloat16"):
        sa.sink_attn_fwd(q.float(), q, q, 1, 1)
    with pytest.raises(ValueError, match="contiguous"):
        sa.qk_norm_rope_fwd(q.transpose(2, 3), q, None, None, [1.0] * 32)
    with pytest.raises(ValueError, match="bfloat16"):
        sa.sink_attn_decode(q[0], q, q, None, 1, 1)
    with pytest.raises(ValueError, match="multiple"):
        sa.cache4_alloc(1, 12, 1, 64, device="cpu")
    cache = sa.cache4_alloc(1, 16, 1, 64, device="cpu")
    assert cache.k_codes.shape == (1, 1, 16, 32) and cache.v_scales.shape == (1, 1, 16, 2)
    with pytest.raises(ValueError):
        sa.cache4_append(cache, q, q)


def test_expanded_and_misaligned_tensors_are_named():
    """An expanded gradient, as a sum's backward gives it, and an odd stride."""
    torch = pytest.importorskip("torch")
    from content_adaptive_sparse_gb300 import streaming
    streaming._device()
    g = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    assert list(streaming._rows("d_o", g, -1)) == [512, 128, 64]
    for bad in (g.expand(3, 4, 2, 64), g[:, :1].expand(1, 9, 2, 64), g[:, :, :1].expand(1, 4, 5, 64),
                torch.zeros(1, 4, 2, 68, dtype=torch.bfloat16)[..., :64]):
        with pytest.raises(ValueError, match="d_o: strides .*contiguous"):
            streaming._rows("d_o", bad, -1)


class Recorder:
    """In the library's place: keeps each call's arguments and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def recorder(monkeypatch):
    """The binding over CPU tensors and a library that only records."""
    pytest.importorskip("torch")
    from content_adaptive_sparse_gb300 import streaming
    streaming._device()
    rec = Recorder()
    monkeypatch.setattr(streaming, "_LIB", rec)
    monkeypatch.setattr(streaming, "_device", lambda: -1)
    monkeypatch.setattr(streaming, "_stream", lambda stream, device: 0)
    streaming._sink_bwd_bytes.cache_clear()
    yield rec
    streaming._sink_bwd_bytes.cache_clear()


BIG = 2**31 - 1


@pytest.mark.parametrize("window,sinks,want", [(5, 4, (5, 4)), (1 << 32, 0, (BIG, 0)), (2**32 + 5, 2**32 + 4, (BIG, BIG)),
                                               (2**31, 2**40, (BIG, BIG)), (-2**32 + 5, 2**31, (-BIG, BIG)),
                                               (3, -2**32 + 1, (3, -BIG))])
def test_windows_and_sinks_past_32_bits(recorder, window, sinks, want):
    """What does not fit a 32-bit argument is not cut to its low bits: a huge window is the whole sequence,
    a huge or negative number of sinks a refusal."""
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 2, 64, dtype=torch.bfloat16)
    n = torch.ones(2, dtype=torch.int32)
    o, lse = sa.sink_attn_fwd(q, k, k, window, sinks)
    sa.sa_sink_attn_fwd(q, k, k, window, sinks, o, lse)
    sa.sink_attn_bwd(q, k, k, o, lse, o, window, sinks)
    sa.sa_sink_attn_bwd(q, k, k, o, o, lse, window, sinks, o, k, k, torch.zeros(8))
    sa.sa_sink_attn_bwd_workspace_size(2, 8, 4, 2, 64, window, sinks)
    o, lse = sa.sink_attn_decode(q[:, :1], k, k, n, window, sinks)
    sa.sa_sink_attn_decode(q[:, :1], k, k, n, window, sinks, o, lse)
    cache = sa.cache4_alloc(2, 8, 2, 64, device="cpu")
    sa.sink_attn_decode_cache4(q[:, :1], cache, n, window, sinks)
    sa.sa_sink_attn_decode_cache4(q[:, :1], cache, n, window, sinks, o, lse)
    assert len(recorder.calls) == 10
    for name, args in recorder.calls:
        after = args.index(64) + 1                       # head_dim; the decoding calls have the lengths' address next
        if "decode" in name:
            after += 1
        assert args[after:after + 2] == want, name


def test_sizes_past_32_bits(recorder, lib):
    torch = pytest.importorskip("torch")
    from content_adaptive_sparse_gb300 import streaming
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    for shape in ((2**32 + 1, 1, 1, 64), (1, 2**32 + 5, 1, 64), (1, 1, 2**31, 64)):
        with pytest.raises(ValueError, match="x: sizes"):
            streaming._rows("x", x.expand(shape), -1)
    assert "sizes" in streaming._layout((64, 64, 64, 1), (1, BIG + 1, 1, 64))
    assert streaming._layout((64, 64, 64, 1), (1, BIG, 1, 64))[1] == 64
    cache = sa.cache4_alloc(1, 8, 1, 64, device="cpu")
    with pytest.raises(ValueError, match="cache: sizes"):
        streaming._cache4([t[:, :, :1].expand(1, 1, 2**32 + 8, -1) for t in cache], -1)
    with pytest.raises(ValueError, match="n_tokens: sizes"):
        sa.cache4_read(cache, None, 2**32 + 1)
    streaming._LIB = lib
    for bad in ((2**32 + 1, 8, 4, 2, 64, 1, 1), (1, 2**32 + 8, 4, 2, 64, 1, 1), (1, 8, 4, 2, 2**32 + 64, 1, 1)):
        with pytest.raises(sa.SAError):
            sa.sa_sink_attn_bwd_workspace_size(*bad)
    with pytest.raises(sa.SAError):
        sa.sa_qk_norm_rope_bwd_workspace_size(2**32 + 64)
    whole = sa.sa_sink_attn_bwd_workspace_size(1, 4096, 4, 2, 64, 4095, 4)
    assert sa.sa_sink_attn_bwd_workspace_size(1, 4096, 4, 2, 64, 2**32 + 5, 4) == whole


@pytest.mark.parametrize("backward", [False, True])
def test_frequencies_live_until_the_call_is_over(recorder, monkeypatch, backward):
    """Other threads rotate with tables of their own meanwhile: the call's table stays where it is."""
    import gc
    import weakref
    torch = pytest.importorskip("torch")
    from content_adaptive_sparse_gb300 import streaming
    made, seen = {}, []
    array = ctypes.c_double * 32
    freq = np.linspace(0.1, 1.0, 32)
    plain = streaming._frequencies.__wrapped__

    @functools.lru_cache(maxsize=64)
    def frequencies(raw):
        out = plain(raw)
        made[raw], = (weakref.ref(x) for x in (out if type(out) is tuple else (out,)) if isinstance(x, array))
        return out

    def call(*args):
        for i in range(100):
            frequencies(np.full(32, 2.0 + i).tobytes())
        gc.collect()
        seen.append(made[freq.tobytes()]() is not None)
        return 0
    monkeypatch.setattr(streaming, "_frequencies", frequencies)
    monkeypatch.setattr(recorder, "sa_qk_norm_rope_bwd" if backward else "sa_qk_norm_rope_fwd", call, raising=False)
    q = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    if backward:
        sa.qk_norm_rope_bwd(q, q, q, q, None, None, freq)
    else:
        sa.qk_norm_rope_fwd(q, q, None, None, freq)
        sa.sa_qk_norm_rope_fwd(q, q, None, None, freq, None, q, q)
    assert seen and all(seen)


# ------------------------------------------------------------------ the oracle

def test_sink_mask_is_the_definition():
    for n, w, s in ((9, 2, 3), (7, 0, 0), (8, 100, 1), (6, 1, 128)):
        m = ref.sink_mask(n, w, s)
        for i in range(n):
            keys = {j for j in range(i + 1) if i - j <= w} | {j for j in range(min(s, i + 1))}
            assert set(np.flatnonzero(m[i])) == keys


def test_sink_oracle_gradients_against_differences():
    rng = np.random.default_rng(0)
    q, k, v, g = (rng.standard_normal((1, 12, h, 4)) for h in (4, 2, 2, 4))
    grads, _ = ref.sink_attention_backward(q, k, v, g, 3, 2)

    def loss(*x):
        return (ref.sink_attention(*x, 3, 2)[0] * g).sum()
    for i, grad in enumerate(grads):
        for _ in range(12):
            at = tuple(rng.integers(0, m) for m in grad.shape)
            up, down = [x.copy() for x in (q, k, v)], [x.copy() for x in (q, k, v)]
            up[i][at] += 1e-5
            down[i][at] -= 1e-5
            assert abs((loss(*up) - loss(*down)) / 2e-5 - grad[at]) < 1e-6


def test_sink_oracle_window_of_everything_is_causal_attention():
    from oracle import dense_masked_attention
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((1, 20, 2, 8)) for _ in range(3))
    o, lse, _ = ref.sink_attention(q, k, v, 19, 0)
    o2, lse2 = dense_masked_attention(q, k, v, np.tril(np.ones((20, 20), bool)))
    assert np.allclose(o, o2, atol=1e-12) and np.allclose(lse, lse2, atol=1e-12)


def test_decode_oracle_is_the_last_row_of_the_prompt_oracle():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((2, 15, h, 8)) for h in (4, 2, 2))
    o, lse, _ = ref.sink_attention(q, k, v, 5, 2)
    o1, lse1, _ = ref.sink_decode(q[:, -1:], k, v, [15, 15], 5, 2)
    assert np.allclose(o1, o[:, -1:], atol=1e-12) and np.allclose(lse1[..., 0], lse[..., -1], atol=1e-12)


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_oracle(inter):
    """A pair turns by its angle (norm kept), scores depend on the distance only, gradients against
    differences."""
    rng = np.random.default_rng(3)
    x, w, g = rng.standard_normal((1, 5, 2, 32)), 1 + 0.1 * rng.standard_normal(32), rng.standard_normal((1, 5, 2, 32))
    pos, freq = np.array([[0, 1, 7, 100, 5]]), 100.0 ** (-np.arange(8) / 8.0)
    y, _ = ref.norm_rope(x, np.ones(32), pos, freq, 1e-9, inter)
    assert np.allclose((y * y).mean(-1), 1.0, atol=1e-6)
    far, _ = ref.norm_rope(x, w, pos + 1000, freq, 1e-6, inter)
    near, _ = ref.norm_rope(x, w, pos, freq, 1e-6, inter)
    assert np.allclose(np.einsum("bihd,bjhd->hij", far, far), np.einsum("bihd,bjhd->hij", near, near), atol=1e-9)
    (dx, dw), _ = ref.norm_rope_backward(x, w, g, pos, freq, 1e-6, inter)

    def loss(x, w):
        return (ref.norm_rope(x, w, pos, freq, 1e-6, inter)[0] * g).sum()
    for _ in range(20):
        at = tuple(rng.integers(0, m) for m in x.shape)
        e = np.zeros(x.shape)
        e[at] = 1e-5
        assert abs((loss(x + e, w) - loss(x - e, w)) / 2e-5 - dx[at]) < 1e-6
        f = np.zeros(32)
        f[at[-1]] = 1e-5
        assert abs((loss(x, w + f) - loss(x, w - f)) / 2e-5 - dw[at[-1]]) < 1e-6


def test_bf16_rounding_of_the_oracle():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(4)
    x = np.float32(rng.standard_normal(20000) * 10.0 ** rng.integers(-41, 38, 20000)).astype(np.float64)
    assert np.array_equal(ref.bf16_round(x), torch.from_numpy(x).float().to(torch.bfloat16).double().numpy())


def test_rows_in_4_bits():
    """Every error is at most half a step; pack is a bijection onto the documented places."""
    rng = np.random.default_rng(5)
    x = ref.bf16_round(rng.standard_normal((50, 128)) * 10.0 ** rng.integers(-3, 4, (50, 1)))
    codes, scales = ref.quantise(x)
    assert codes.min() >= -7 and codes.max() <= 7
    step = np.repeat(scales, 32, axis=-1)
    # the scale is rounded to bf16: the largest element may lie up to 7 x 2^-8 of a step past code 7
    assert np.all(np.abs(ref.values(codes, scales) - x) <= step * (0.5 + 7 * 2.0 ** -8) + 1e-300)
    for d in (32, 64, 128):
        seen = set()
        for e in range(d):
            one = np.full(d, -8)
            one[e] = 7
            row = ref.pack(one)
            (byte,) = np.flatnonzero(row)
            assert row[byte] in (0x0f, 0xf0)
            seen.add((byte, int(row[byte])))
        assert len(seen) == d
