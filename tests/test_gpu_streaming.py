"""Streaming attention on the GPU against float64 (oracle/streaming.py): norm and rotation, the
sink-window graph forward and backward, single tokens over bf16 and 4-bit caches, and a run of
them together. Tolerances are the oracle's elementwise bounds."""
import numpy as np
import pytest

import content_adaptive_sparse_gb300 as sa
from gpu_helpers import bf16_to_f64, torch_cuda
from oracle import streaming as ref

pytestmark = pytest.mark.gpu

# LSE in fp32: scores of |s| <= about 20 carry a few 2^-24 of sum |q k|, the exponentials and the
# logarithm 2^-22 each; 1e-4 is an order of magnitude above their sum
LSE_TOL = 1e-4


def rand(seed, *shape, scale=1.0):
    """bf16 CUDA tensor and its float64 values."""
    torch = torch_cuda()
    x = (torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * scale)).to(torch.bfloat16).cuda()
    return x, bf16_to_f64(x)


def close(got, want, bound, what):
    got = got.detach().double().cpu().numpy() if not isinstance(got, np.ndarray) else got
    assert got.shape == want.shape, what
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.abs(got - want) - bound
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{what}: {got[at]} against {want[at]}, bound {np.broadcast_to(bound, want.shape)[at]} at {at}"


def status_ok():
    torch_cuda().cuda.synchronize()
    assert sa.sa_device_status() == 0


# ------------------------------------------------------------------ sink-window attention

SINK_CASES = [
    # batch, tokens, heads, kv_heads, dim, window, sinks
    (1, 1, 1, 1, 32, 0, 0), (1, 1, 2, 1, 64, 5, 4), (1, 2, 2, 2, 128, 0, 1),
    (2, 31, 2, 1, 64, 7, 3), (1, 33, 4, 2, 128, 0, 0), (1, 127, 2, 2, 32, 31, 32), (2, 128, 2, 1, 64, 32, 33),
    (1, 129, 2, 2, 128, 33, 1), (1, 300, 4, 1, 64, 64, 4), (1, 300, 2, 2, 128, 100, 17), (2, 257, 6, 3, 32, 128, 5),
    (1, 640, 2, 1, 64, 0, 128), (1, 640, 2, 1, 128, 1, 127), (1, 641, 3, 3, 32, 255, 0), (1, 500, 2, 1, 64, 499, 4),
    (1, 500, 2, 1, 128, 100000, 4), (1, 1500, 2, 1, 64, 127, 4), (1, 1411, 4, 2, 128, 200, 9), (3, 200, 5, 5, 64, 96, 64),
    (1, 2900, 1, 1, 32, 3, 100),
]


@pytest.mark.parametrize("b,n,h,hk,d,w,s", SINK_CASES)
def test_sink_attention_forward_and_backward(b, n, h, hk, d, w, s):
    (q, qf), (k, kf), (v, vf), (g, gf) = (rand(i, b, n, x, d) for i, x in enumerate((h, hk, hk, h)))
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    status_ok()
    of, lf, ob = ref.sink_attention(qf, kf, vf, w, s)
    close(o, of, ob, "o")
    close(lse, lf, LSE_TOL, "lse")
    grads = sa.sink_attn_bwd(q, k, v, o, lse, g, w, s)
    status_ok()
    want, bounds = ref.sink_attention_backward(qf, kf, vf, gf, w, s)
    for name, x, y, e in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(x, y, e, name)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_sink_attention_large_scores(d):
    """Scores of hundreds that grow along the sequence: the running maximum is rescaled often."""
    n, w, s = 400, 90, 6
    (q, qf), (k, kf), (v, vf) = rand(0, 1, n, 2, d, scale=6.0), rand(1, 1, n, 1, d, scale=6.0), rand(2, 1, n, 1, d)
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    status_ok()
    of, lf, ob = ref.sink_attention(qf, kf, vf, w, s)
    # |s| up to 400: fp32 scores are off by up to about 400 x 2^-20, and so is ln P
    close(o, of, ob + 8e-4 * np.abs(vf).max(), "o")
    close(lse, lf, 4e-4, "lse")


def test_sink_attention_strided_scaled_and_repeated():
    """Packed Q/K/V views, outputs and gradients with strides of their own, an explicit scale; the
    backward gives the same bits twice."""
    torch = torch_cuda()
    b, n, h, hk, d, w, s = 2, 333, 4, 2, 64, 75, 5
    packed, pf = rand(3, b, n, h + 2 * hk, d)
    q, k, v = packed[:, :, :h], packed[:, :, h:h + hk], packed[:, :, h + hk:]
    qf, kf, vf = pf[:, :, :h], pf[:, :, h:h + hk], pf[:, :, h + hk:]
    wide_g, wgf = rand(4, b, n, 2 * h, d)
    g, gf = wide_g[:, :, h:], wgf[:, :, h:]
    o = torch.empty(b, n, 2, h, d, dtype=torch.bfloat16, device="cuda")[:, :, 1]
    lse = torch.empty(b, h, n, dtype=torch.float32, device="cuda")
    sa.sa_sink_attn_fwd(q, k, v, w, s, o, lse, softmax_scale=0.2)
    of, lf, ob = ref.sink_attention(qf, kf, vf, w, s, scale=0.2)
    status_ok()
    close(o, of, ob, "o")
    close(lse, lf, LSE_TOL, "lse")
    dpacked = torch.full_like(packed, 7.0)
    dq, dk, dv = dpacked[:, :, :h], dpacked[:, :, h:h + hk], dpacked[:, :, h + hk:]
    ws = torch.empty(sa.sa_sink_attn_bwd_workspace_size(b, n, h, hk, d, w, s), dtype=torch.uint8, device="cuda")
    sa.sa_sink_attn_bwd(q, k, v, o, g, lse, w, s, dq, dk, dv, ws, softmax_scale=0.2)
    status_ok()
    want, bounds = ref.sink_attention_backward(qf, kf, vf, gf, w, s, scale=0.2)
    for name, x, y, e in zip(("dq", "dk", "dv"), (dq, dk, dv), want, bounds):
        close(x, y, e, name)
    first = dpacked.clone()
    ws.fill_(0xff)
    sa.sa_sink_attn_bwd(q, k, v, o, g, lse, w, s, dq, dk, dv, ws, softmax_scale=0.2)
    status_ok()
    assert torch.equal(first.view(torch.int16), dpacked.view(torch.int16))


def test_windows_past_32_bits_are_the_whole_sequence():
    torch = torch_cuda()
    b, n, h, hk, d = 1, 200, 4, 2, 64
    q, k, v, g = (rand(i, b, n, x, d)[0] for i, x in enumerate((h, hk, hk, h)))
    length = torch.tensor([n], dtype=torch.int32, device="cuda")
    cache = sa.cache4_alloc(b, n, hk, d)
    sa.cache4_append(cache, k, v)

    def calls(w):
        o, lse = sa.sink_attn_fwd(q, k, v, w, 0)
        return (o, lse) + sa.sink_attn_bwd(q, k, v, o, lse, g, w, 0) + sa.sink_attn_decode(q[:, -1:], k, v, length, w, 0) + \
            sa.sink_attn_decode_cache4(q[:, -1:], cache, length, w, 0)

    want = calls(n - 1)
    for w in (1 << 32, 2**32 + 5, 1 << 63):
        assert all(torch.equal(x, y) for x, y in zip(calls(w), want))
    status_ok()


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("n,w,s", [(1, 0, 0), (1, 9, 4), (131, 0, 0)])
def test_sink_attention_backward_of_one_visible_key(n, w, s, d):
    """P is 1 whatever the scores are: the gradients of queries and keys are zero, not the rounding of
    two equal sums."""
    torch = torch_cuda()
    q, k, v, g = (rand(i, 2, n, 2 if i in (1, 2) else 6, d)[0] for i in range(4))
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    dq, dk, dv = sa.sink_attn_bwd(q, k, v, o, lse, g, w, s)
    status_ok()
    assert not dq.any() and not dk.any()
    want = g.double().unflatten(2, (2, 3)).sum(3)
    # three bf16 numbers summed in 32 bits, and one rounding
    assert ((dv.double() - want).abs() <= 2.0**-8 * want.abs() + 2.0**-20 * g.double().abs().max()).all()


@pytest.mark.parametrize("n,h,hk,d,w,s", [(2, 4, 1, 64, 9, 0), (8, 4, 4, 32, 50, 3), (300, 6, 2, 128, 1, 0), (150, 4, 2, 64, 4, 3),
                                          (131, 2, 1, 32, 2, 5), (32, 3, 3, 64, 31, 0), (23, 4, 2, 128, 6, 9)])
def test_sink_attention_backward_of_few_visible_keys(n, h, hk, d, w, s):
    """Up to eight keys a query, or 32 tokens: the rounding of O leaves the gradients alone."""
    q, qf = rand(0, 2, n, h, d)
    k, kf = rand(1, 2, n, hk, d)
    v, vf = rand(2, 2, n, hk, d)
    g, gf = rand(3, 2, n, h, d)
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    got = sa.sink_attn_bwd(q, k, v, o, lse, g, w, s)
    status_ok()
    want, bounds = ref.sink_attention_backward(qf, kf, vf, gf, w, s, rounded_o=False)
    for name, x, y, e in zip(("dq", "dk", "dv"), got, want, bounds):
        close(x, y, e, name)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("n", [33, 200, 257, 1500])
def test_first_tokens_gradients_in_sequences_of_any_length(n, d):
    """The first 32 tokens see few keys however long the sequence is: the rounding of O leaves their dQ alone."""
    (q, qf), (k, kf), (v, vf), (g, gf) = (rand(i, 2, n, x, d) for i, x in enumerate((4, 2, 2, 4)))
    o, lse = sa.sink_attn_fwd(q, k, v, 600, 4)
    dq, _, _ = sa.sink_attn_bwd(q, k, v, o, lse, g, 600, 4)
    status_ok()
    want, bounds = ref.sink_attention_backward(qf, kf, vf, gf, 600, 4, rounded_o=False)
    close(dq[:, :32], want[0][:, :32], bounds[0][:, :32], "dq")


# ------------------------------------------------------------------ single tokens over a cache

DECODE_CASES = [
    # heads, kv_heads, dim, capacity, window, sinks, lengths
    (1, 1, 32, 8, 0, 0, [1]), (2, 1, 64, 16, 3, 2, [0, 1, 16]), (4, 4, 128, 64, 100, 4, [64, 63, 1]),
    (8, 2, 64, 72, 16, 16, [72, 40, 17, 16]), (16, 1, 128, 200, 50, 33, [200, 84, 51, 3]), (20, 1, 64, 136, 65, 1, [136, 5]),
    (40, 2, 32, 264, 500, 0, [264, 130]), (6, 3, 128, 1000, 700, 128, [1000, 900, 701, 128]),
    (4, 1, 64, 4096, 4095, 4, [4096, 4001, 2]), (2, 2, 32, 6000, 3000, 70, [5999, 3071, 3001, 10]),
    (5, 5, 128, 2048, 1, 65, [2000]), (12, 12, 64, 520, 511, 4, [7, 520, 519]),
]


@pytest.mark.parametrize("h,hk,d,cap,w,s,lengths", DECODE_CASES)
def test_decode_over_a_bf16_cache(h, hk, d, cap, w, s, lengths):
    """Rows that the query does not see hold NaN and infinities."""
    torch = torch_cuda()
    b = len(lengths)
    q, qf = rand(0, b, 1, h, d)
    k, kf = rand(1, b, cap, hk, d)
    v, vf = rand(2, b, cap, hk, d)
    for i, n in enumerate(lengths):
        j = torch.arange(cap, device="cuda")
        unseen = (j >= n) | ((n - 1 - j > w) & (j >= s))
        k[i, unseen] = float("nan")
        v[i, unseen] = float("inf")
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, lse = sa.sink_attn_decode(q, k, v, n, w, s)
    status_ok()
    of, lf, ob = ref.sink_decode(qf, kf, vf, lengths, w, s)
    close(o, of, ob, "o")
    lse = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(lse), np.isneginf(lf))
    some = ~np.isneginf(lf)
    close(lse[some], lf[some], LSE_TOL, "lse")


@pytest.mark.parametrize("h,hk,d,cap,w,s,lengths", DECODE_CASES)
def test_decode_over_a_4_bit_cache(h, hk, d, cap, w, s, lengths):
    """The rows are written by the append; rows that are not seen hold random codes and NaN scales."""
    torch = torch_cuda()
    b = len(lengths)
    q, qf = rand(0, b, 1, h, d)
    k, kf = rand(1, b, cap, hk, d)
    v, vf = rand(2, b, cap, hk, d, scale=3.0)
    cache = sa.cache4_alloc(b, cap, hk, d)
    sa.cache4_append(cache, k, v)
    j = torch.arange(cap, device="cuda")
    for i, n in enumerate(lengths):
        unseen = (j >= n) | ((n - 1 - j > w) & (j >= s))
        cache.k_codes[i][:, unseen] = 255
        cache.v_codes[i][:, unseen] = 0
        cache.k_scales[i][:, unseen] = float("nan")
        cache.v_scales[i][:, unseen] = float("nan")
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, lse = sa.sink_attn_decode_cache4(q, cache, n, w, s)
    status_ok()
    kq, vq = (ref.values(*ref.quantise(x)) for x in (kf, vf))
    of, lf, ob = ref.sink_decode(qf, kq, vq, lengths, w, s)
    close(o, of, ob, "o")
    lse = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(lse), np.isneginf(lf))
    some = ~np.isneginf(lf)
    close(lse[some], lf[some], LSE_TOL, "lse")


def test_decode_lengths_outside_the_cache_are_cut():
    torch = torch_cuda()
    q, qf = rand(0, 3, 1, 4, 64)
    k, kf = rand(1, 3, 40, 2, 64)
    v, vf = rand(2, 3, 40, 2, 64)
    n = torch.tensor([-5, 1000, 40], dtype=torch.int32, device="cuda")
    o, lse = sa.sink_attn_decode(q, k, v, n, 20, 3)
    status_ok()
    of, lf, ob = ref.sink_decode(qf, kf, vf, [0, 40, 40], 20, 3)
    close(o, of, ob, "o")
    close(lse[1:], lf[1:], LSE_TOL, "lse")
    assert torch.isneginf(lse[0]).all() and not o[0].any()


def test_decode_strided_cache_and_large_scores():
    """Keys and values interleaved in one buffer, queries from a packed projection."""
    torch = torch_cuda()
    b, h, hk, d, cap = 2, 8, 2, 128, 300
    kv, kvf = rand(1, b, cap, 2 * hk, d, scale=4.0)
    packed, pf = rand(0, b, 1, h + 2 * hk, d, scale=4.0)
    q, qf = packed[:, :, :h], pf[:, :, :h]
    n = torch.tensor([300, 211], dtype=torch.int32, device="cuda")
    o, lse = sa.sink_attn_decode(q, kv[:, :, :hk], kv[:, :, hk:], n, 150, 4)
    status_ok()
    of, lf, ob = ref.sink_decode(qf, kvf[:, :, :hk], kvf[:, :, hk:], [300, 211], 150, 4)
    close(o, of, ob + 4e-4 * np.abs(kvf).max(), "o")
    close(lse, lf, 4e-4, "lse")


# ------------------------------------------------------------------ numbers that are not numbers

@pytest.mark.parametrize("scale", [1e-44, 1e-20, None])
@pytest.mark.parametrize("h,hk,d", [(4, 2, 32), (24, 2, 64), (4, 2, 128)])
def test_decode_of_zero_queries(h, hk, d, scale):
    """A query of zeros sees every key alike, however small the scale: the mean of the values."""
    torch = torch_cuda()
    b, cap, w, s, lengths = 3, 72, 40, 3, [1, 13, 71]
    q, qf = rand(0, b, 1, h, d)
    q[:, :, 1] = 0.0
    qf[:, :, 1] = 0.0
    k, kf = rand(1, b, cap, hk, d)
    v, vf = rand(2, b, cap, hk, d)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    cache = sa.cache4_alloc(b, cap, hk, d)
    sa.cache4_append(cache, k, v)
    got = sa.sink_attn_decode(q, k, v, n, w, s, scale), sa.sink_attn_decode_cache4(q, cache, n, w, s, scale)
    status_ok()
    quant = [ref.values(*ref.quantise(x)) for x in (kf, vf)]
    for (o, lse), (kx, vx) in zip(got, ((kf, vf), quant)):
        of, lf, ob = ref.sink_decode(qf, kx, vx, lengths, w, s, scale)
        close(o, of, ob, "o")
        close(lse, lf, LSE_TOL, "lse")


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("h", [4, 24])
def test_decode_keeps_nan_of_what_is_seen(h, d):
    """A NaN in a query, in the only key and in one key of many: o and lse are NaN for the heads that see it,
    not the zeros of an empty sequence, and the others are as without it."""
    torch = torch_cuda()
    b, hk, cap, w, s = 4, 2, 512, 511, 0
    lengths = [1, 400, 400, 0]
    q, k, v = (rand(i, b, x, y, d)[0] for i, (x, y) in enumerate(((1, h), (cap, hk), (cap, hk))))
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")

    def both():
        cache = sa.cache4_alloc(b, cap, hk, d)
        sa.cache4_append(cache, k, v)
        out = sa.sink_attn_decode(q, k, v, n, w, s), sa.sink_attn_decode_cache4(q, cache, n, w, s)
        status_ok()
        return out

    clean = both()
    group = h // hk
    hit = torch.zeros(b, h, dtype=torch.bool, device="cuda")
    hit[0, :group] = hit[1, group:] = hit[2, 1] = True
    k[0, 0, 0, 5] = float("nan")                          # the only key of key head 0
    k[1, 371, 1, d - 1] = float("nan")                    # one of 400 of key head 1
    q[2, 0, 1, 3] = float("nan")
    for (o, lse), (o1, lse1) in zip(both(), clean):
        assert torch.isnan(o[:, 0][hit]).all() and torch.isnan(lse[..., 0][hit]).all()
        assert torch.equal(o[:, 0][~hit], o1[:, 0][~hit]) and torch.equal(lse[..., 0][~hit], lse1[..., 0][~hit])
        assert torch.isneginf(lse[3]).all() and not o[3].any()


@pytest.mark.parametrize("d", [32, 64, 128])
def test_sink_attention_keeps_nan_queries(d):
    torch = torch_cuda()
    b, n, h, w, s = 1, 300, 2, 40, 3
    q, k, v = (rand(i, b, n, h, d)[0] for i in range(3))
    q[0, 7, 1, 2] = q[0, 290, 0, 0] = float("nan")
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    status_ok()
    for i, e in ((7, 1), (290, 0)):
        assert torch.isnan(o[0, i, e]).all() and torch.isnan(lse[0, e, i])
    assert int(torch.isnan(lse).sum()) == 2 and not torch.isneginf(lse).any()


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("j", [2, 150])
def test_sink_attention_keeps_nan_keys(j, d):
    """A sink, or a key of the middle, with a NaN: NaN for the queries that see it and for no other."""
    torch = torch_cuda()
    b, n, h, w, s = 1, 300, 2, 40, 3
    q, k, v = (rand(i, b, n, h, d)[0] for i in range(3))
    o1, lse1 = sa.sink_attn_fwd(q, k, v, w, s)
    k[0, j, 0, d // 2] = float("nan")
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    status_ok()
    hit = torch.zeros(n, h, dtype=torch.bool, device="cuda")
    hit[:, 0] = torch.from_numpy(ref.sink_mask(n, w, s)[:, j]).cuda()
    assert torch.isnan(o[0][hit]).all() and torch.isnan(lse[0].T[hit]).all()
    assert torch.equal(o[0][~hit], o1[0][~hit]) and torch.equal(lse[0].T[~hit], lse1[0].T[~hit])


# ------------------------------------------------------------------ 4-bit cache

@pytest.mark.parametrize("b,n,hk,d,cap,start", [(1, 1, 1, 32, 8, [7]), (2, 5, 3, 64, 16, [0, 11]), (3, 70, 2, 128, 96, [3, 26, 9]),
                                                (1, 333, 4, 32, 1000, [600]), (2, 129, 1, 64, 136, None)])
def test_cache4_rows(b, n, hk, d, cap, start):
    """Codes, scales, what they read back as, and the other rows untouched; a run of zeros, one of a
    single subnormal, one of the largest magnitudes."""
    torch = torch_cuda()
    k, _ = rand(1, b, n, hk, d)
    v, _ = rand(2, b, n, hk, d, scale=100.0)
    k[0, 0, 0, :32] = 0.0
    v[0, 0, 0, :32] = torch.tensor([1e-39] + [0.0] * 31)
    v[0, n - 1, hk - 1, -32:] = 3.0e38 * torch.linspace(-1, 1, 32)
    kf, vf = bf16_to_f64(k), bf16_to_f64(v)
    cache = sa.cache4_alloc(b, cap, hk, d)
    for x in cache:
        x.view(torch.uint8).fill_(0x5a)
    at = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
    sa.cache4_append(cache, k, v, at)
    k2, v2 = sa.cache4_read(cache, at, n)
    status_ok()
    for x, codes, scales, back in ((kf, cache.k_codes, cache.k_scales, k2), (vf, cache.v_codes, cache.v_scales, v2)):
        c, s = ref.quantise(x)
        assert np.array_equal(bf16_to_f64(back), ref.bf16_round(ref.values(c, s)))
        codes, scales = codes.cpu().numpy(), bf16_to_f64(scales)
        packed = ref.pack(c)
        for i in range(b):
            lo = 0 if start is None else start[i]
            assert np.array_equal(codes[i, :, lo:lo + n], packed[i].transpose(1, 0, 2))
            assert np.array_equal(scales[i, :, lo:lo + n], s[i].transpose(1, 0, 2))
            other = np.delete(codes[i], np.arange(lo, lo + n), axis=1)
            assert np.all(other == 0x5a)


@pytest.mark.parametrize("hk,d", [(4, 128), (3, 128), (16, 64), (5, 32)])
def test_cache4_long_and_short_calls_agree(hk, d):
    """A long prompt in one call and in pieces: the same codes and scales, read back alike."""
    torch = torch_cuda()
    b, n = 2, 6007 * 512 // (hk * d)
    n += 1 - n % 2
    cap = -(-n // 8) * 8 + 16
    start = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(b, n, hk, d, device="cuda").bfloat16() for _ in range(2))
    whole, parts = sa.cache4_alloc(b, cap, hk, d), sa.cache4_alloc(b, cap, hk, d)
    for x in whole + parts:
        x.zero_()
    sa.cache4_append(whole, k, v, start)
    step = n // 16 + 1
    for i in range(0, n, step):
        sa.cache4_append(parts, k[:, i:i + step], v[:, i:i + step], start + i)
    rk, rv = sa.cache4_read(whole, start, n)
    pieces = [sa.cache4_read(whole, start + i, min(step, n - i)) for i in range(0, n, step)]
    status_ok()
    assert all(torch.equal(x, y) for x, y in zip(whole, parts))
    assert torch.equal(rk, torch.cat([x for x, _ in pieces], 1)) and torch.equal(rv, torch.cat([x for _, x in pieces], 1))


def test_cache4_left_out_and_overfull_sequences():
    torch = torch_cuda()
    b, n, hk, d, cap = 3, 6, 2, 64, 16
    (k, kf), (v, vf) = rand(1, b, n, hk, d), rand(2, b, n, hk, d)
    k[1, 2, 0, 3] = float("inf")
    k[1, 3, 1, 40] = float("nan")
    cache = sa.cache4_alloc(b, cap, hk, d)
    for x in cache:
        x.zero_()
    start = torch.tensor([-1, 4, 12], dtype=torch.int32, device="cuda")
    sa.cache4_append(cache, k, v, start)
    torch.cuda.synchronize()
    assert sa.sa_device_status() == -6                    # two rows of the third sequence did not fit
    assert not cache.k_codes[0].any() and not cache.v_scales[0].any()
    k2, v2 = sa.cache4_read(cache, start, n)
    torch.cuda.synchronize()
    assert sa.sa_device_status() == -6
    assert not k2[0].any() and not v2[0].any() and not k2[2, 4:].any()
    assert np.array_equal(bf16_to_f64(k2[2, :4]), ref.bf16_round(ref.values(*ref.quantise(kf[2, :4]))))
    nan = torch.isnan(k2[1])
    assert nan[2, 0, :32].all() and nan[3, 1, 32:].all() and int(nan.sum()) == 64
    assert np.array_equal(bf16_to_f64(v2[1]), ref.bf16_round(ref.values(*ref.quantise(vf[1]))))


# ------------------------------------------------------------------ norm and rotation

ROPE_CASES = [
    # batch, tokens, heads, kv_heads, dim, rotary, interleaved, weights, positions
    (1, 1, 1, 1, 32, 32, False, True, None), (2, 3, 5, 2, 64, 64, False, True, "far"), (1, 7, 4, 4, 128, 128, True, True, "far"),
    (1, 40, 3, 1, 128, 64, False, False, None), (2, 33, 12, 12, 64, 32, True, True, "far"), (1, 129, 2, 1, 32, 16, False, True, "negative"),
    (1, 5, 9, 1, 64, 0, False, True, None), (3, 1, 16, 4, 128, 128, False, True, "far"), (2, 700, 6, 2, 32, 32, True, False, "far"),
]


@pytest.mark.parametrize("b,n,h,hk,d,rotary,inter,weights,where", ROPE_CASES)
def test_norm_rope_forward_and_backward(b, n, h, hk, d, rotary, inter, weights, where):
    torch = torch_cuda()
    rng = np.random.default_rng(5)
    packed, pf = rand(0, b, n, h + 2 * hk, d)
    packed[0, 0, 0] = 0.0                                  # a row of zeros
    pf[0, 0, 0] = 0.0
    q, k, qf, kf = packed[:, :, :h], packed[:, :, h:h + hk], pf[:, :, :h], pf[:, :, h:h + hk]
    (gq, gqf), (gk, gkf) = rand(1, b, n, h, d), rand(2, b, n, hk, d)
    w = [np.float32(1 + 0.2 * rng.standard_normal(d)) if weights else np.ones(d, np.float32) for _ in range(2)]
    wt = [torch.from_numpy(x).cuda() if weights else None for x in w]
    freq = 10000.0 ** (-2.0 * np.arange(rotary // 2) / max(rotary, 1))
    pos = np.broadcast_to(np.arange(n), (b, n))
    if where:
        pos = rng.integers(0, 1 << 30, (b, n)) if where == "far" else -rng.integers(0, 100000, (b, n))
    pt = torch.from_numpy(pos.astype(np.int32)).cuda() if where else None
    eps = 1e-5
    outs = sa.qk_norm_rope_fwd(q, k, *wt, freq, pt, eps, inter)
    status_ok()
    for name, x, xf, wf in zip("qk", outs, (qf, kf), w):
        y, bound = ref.norm_rope(xf, wf.astype(np.float64), pos, freq, eps, inter)
        close(x, y, bound, name + "_out")
    dq, dk, dqw, dkw = sa.qk_norm_rope_bwd(q, k, gq, gk, *wt, freq, pt, eps, inter)
    status_ok()
    for name, x, dw, xf, gf, wf in zip("qk", (dq, dk), (dqw, dkw), (qf, kf), (gqf, gkf), w):
        (dxf, dwf), (bx, bw) = ref.norm_rope_backward(xf, wf.astype(np.float64), gf, pos, freq, eps, inter)
        close(x, dxf, bx, "d" + name)
        if weights:
            close(dw, dwf, bw, "dw_" + name)
        else:
            assert dw is None
    # in place, and the same bits twice
    qc, kc = q.clone(memory_format=torch.contiguous_format), k.clone(memory_format=torch.contiguous_format)
    sa.sa_qk_norm_rope_fwd(qc, kc, *wt, freq, pt, qc, kc, eps, inter)
    status_ok()
    assert torch.equal(qc, outs[0]) and torch.equal(kc, outs[1])
    again = sa.qk_norm_rope_bwd(q, k, gq, gk, *wt, freq, pt, eps, inter)
    for x, y in zip((dq, dk, dqw, dkw), again):
        assert (x is None and y is None) or torch.equal(x, y)


# ------------------------------------------------------------------ together

def _model(seed, b, n, h, hk, d):
    packed, pf = rand(seed, b, n, h + 2 * hk, d)
    rng = np.random.default_rng(9)
    w = [np.float32(1 + 0.1 * rng.standard_normal(d)) for _ in range(2)]
    freq = 10000.0 ** (-2.0 * np.arange(d // 2) / d)
    return packed, pf, w, freq


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_then_tokens_agree_with_one_pass(d):
    """A prompt through norm, rotation and the window, its rows into both caches, then one token at a
    time on another stream: every token's output is the row that one pass over all tokens gives."""
    torch = torch_cuda()
    b, n, prompt, h, hk, w, s = 2, 90, 83, 4, 2, 40, 3
    packed, _, wts, freq = _model(0, b, n, h, hk, d)
    wt = [torch.from_numpy(x).cuda() for x in wts]
    q, k, v = packed[:, :, :h], packed[:, :, h:h + hk], packed[:, :, h + hk:]
    qr, kr = sa.qk_norm_rope_fwd(q, k, *wt, freq)
    o, lse = sa.sink_attn_fwd(qr, kr, v, w, s)
    status_ok()
    qf, kf, vf = (bf16_to_f64(x) for x in (qr, kr, v))
    of, lf, ob = ref.sink_attention(qf, kf, vf, w, s)
    close(o, of, ob, "one pass")
    k4, v4 = (ref.values(*ref.quantise(x)) for x in (kf, vf))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cap = 96
        kcache = torch.full((b, cap, hk, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        vcache = torch.full_like(kcache, float("nan"))
        kcache[:, :prompt], vcache[:, :prompt] = kr[:, :prompt], v[:, :prompt]
        cache = sa.cache4_alloc(b, cap, hk, d)
        sa.cache4_append(cache, kr[:, :prompt], v[:, :prompt])
        outs, outs4 = [], []
        for i in range(prompt, n):
            at = torch.full((b,), i, dtype=torch.int32, device="cuda")
            qi, ki = sa.qk_norm_rope_fwd(q[:, i:i + 1], k[:, i:i + 1], *wt, freq, at[:, None])
            kcache[:, i], vcache[:, i] = ki[:, 0], v[:, i]
            sa.cache4_append(cache, ki, v[:, i:i + 1], at)
            outs.append(sa.sink_attn_decode(qi, kcache, vcache, at + 1, w, s))
            outs4.append(sa.sink_attn_decode_cache4(qi, cache, at + 1, w, s))
    side.synchronize()
    assert sa.sa_device_status(side) == 0
    o4, l4, ob4 = ref.sink_attention(qf, k4, v4, w, s)
    for got, want, bound, lw in ((outs, of, ob, lf), (outs4, o4, ob4, l4)):
        close(torch.cat([x[0] for x in got], 1), want[:, prompt:], bound[:, prompt:], "tokens")
        close(torch.cat([x[1] for x in got], 2), lw[:, :, prompt:], LSE_TOL, "tokens' lse")


def test_training_chain_against_differences():
    """Norm, rotation and attention with their gradients chained, against the float64 chain's
    differences along random directions."""
    torch = torch_cuda()
    b, n, h, hk, d, w, s = 1, 150, 4, 2, 64, 30, 3
    packed, pf, wts, freq = _model(1, b, n, h, hk, d)
    wt = [torch.from_numpy(x).cuda() for x in wts]
    g, gf = rand(7, b, n, h, d)
    q, k, v = packed[:, :, :h], packed[:, :, h:h + hk], packed[:, :, h + hk:]
    qr, kr = sa.qk_norm_rope_fwd(q, k, *wt, freq)
    o, lse = sa.sink_attn_fwd(qr, kr, v, w, s)
    dqr, dkr, dv = sa.sink_attn_bwd(qr, kr, v, o, lse, g, w, s)
    dq, dk, dqw, dkw = sa.qk_norm_rope_bwd(q, k, dqr, dkr, *wt, freq)
    status_ok()
    pos = np.arange(n)[None]

    def loss(x, wq, wk):
        a, _ = ref.norm_rope(x[:, :, :h], wq, pos, freq, 1e-6, False)
        c, _ = ref.norm_rope(x[:, :, h:h + hk], wk, pos, freq, 1e-6, False)
        return (ref.sink_attention(a, c, x[:, :, h + hk:], w, s)[0] * gf).sum()

    grad = np.concatenate([bf16_to_f64(x) for x in (dq, dk, dv)], axis=2)
    gw = [x.double().cpu().numpy() for x in (dqw, dkw)]
    rng = np.random.default_rng(11)
    for trial in range(4):
        dx, dwq, dwk = rng.standard_normal(pf.shape), rng.standard_normal(d), rng.standard_normal(d)
        e = 1e-5
        w64 = [x.astype(np.float64) for x in wts]
        num = (loss(pf + e * dx, w64[0] + e * dwq, w64[1] + e * dwk) - loss(pf - e * dx, w64[0] - e * dwq, w64[1] - e * dwk)) / (2 * e)
        got = (grad * dx).sum() + gw[0] @ dwq + gw[1] @ dwk
        # each gradient element is off by a few independent bf16 roundings (2^-8 at most, about 2^-9
        # on average) of its size, and the roundings of q_out, k_out, P and O before it add about as
        # much again: along a random direction their sum is far below 4 x 2^-8 of the gradient's norm
        size = np.sqrt((grad ** 2).sum() + (gw[0] ** 2).sum() + (gw[1] ** 2).sum())
        assert abs(num - got) <= 4 * ref.U * size, (trial, num, got, size)


def _ends(x, head, tail):
    """The first `head` and last `tail` tokens of a tensor, as one short sequence."""
    torch = torch_cuda()
    return torch.cat((x[:, :head], x[:, -tail:]), 1).contiguous()


def test_attention_over_more_than_2_31_elements():
    """The last queries and keys of a sequence whose tensors pass 32-bit offsets see what those of a
    short one with the same ends see."""
    torch = torch_cuda()
    n, h, d, w, s, tail = (1 << 20) + 77, 17, 128, 100, 4, 500
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, g = (torch.randn(1, n, h, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    freq = 1000.0 ** -np.arange(d // 2)
    positions = torch.arange(n, device="cuda", dtype=torch.int32)[None]
    qr, kr = sa.qk_norm_rope_fwd(q, k, None, None, freq, positions)
    small = [_ends(x, s, tail) for x in (q, k, v, g)]
    want_q, want_k = sa.qk_norm_rope_fwd(small[0], small[1], None, None, freq, _ends(positions, s, tail))
    assert torch.equal(_ends(qr, s, tail), want_q) and torch.equal(_ends(kr, s, tail), want_k)
    o, lse = sa.sink_attn_fwd(qr, kr, v, w, s)
    grads = sa.sink_attn_bwd(qr, kr, v, o, lse, g, w, s)
    status_ok()
    qf, kf, vf, gf = (bf16_to_f64(x) for x in (want_q, want_k, small[2], small[3]))
    of, lf, ob = ref.sink_attention(qf, kf, vf, w, s)
    rows = slice(-tail + 2 * w, None)                 # past the seam and its queries' windows
    close(o[:, -tail + 2 * w:], of[:, rows], ob[:, rows], "o")
    close(lse[:, :, -tail + 2 * w:], lf[:, :, rows], LSE_TOL, "lse")
    want, bounds = ref.sink_attention_backward(qf, kf, vf, gf, w, s)
    for name, x, y, e in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(x[:, -tail + 2 * w:], y[:, rows], e[:, rows], name)


def test_first_tokens_of_more_than_2_31_elements():
    """The first tokens' outputs and dQ (a persistent CTA's last items) are those of a short sequence, and the
    sinks' dK and dV are the sums over all of a million queries."""
    torch = torch_cuda()
    n, h, d, w, s, head = (1 << 20) + 77, 17, 128, 100, 4, 300
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v, g = (torch.randn(1, n, h, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    assert q.numel() > 1 << 31
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    dq, dk, dv = sa.sink_attn_bwd(q, k, v, o, lse, g, w, s)
    status_ok()
    first = [bf16_to_f64(x[:, :head]) for x in (q, k, v, g)]
    of, lf, ob = ref.sink_attention(*first[:3], w, s)
    close(o[:, :head], of, ob, "o")
    close(lse[:, :, :head], lf, LSE_TOL, "lse")
    want, bounds = ref.sink_attention_backward(*first, w, s)
    close(dq[:, :head], want[0], bounds[0], "dq")
    for e in (0, 9, h - 1):
        kd, vd = k[0, :s, e].double(), v[0, :s, e].double()
        sums = [torch.zeros(s, d, dtype=torch.float64, device="cuda") for _ in range(4)]
        for i0 in range(0, n, 1 << 17):
            rows = slice(i0, min(n, i0 + (1 << 17)))
            qd, gd, od = (x[0, rows, e].double() for x in (q, g, o))
            seen = torch.arange(s, device="cuda") <= torch.arange(rows.start, rows.stop, device="cuda")[:, None]
            p = torch.where(seen, torch.exp(qd @ kd.T * d ** -0.5 - lse[0, e, rows].double()[:, None]), 0.0)
            ds = p * (gd @ vd.T - (gd * od).sum(-1, keepdim=True)) * d ** -0.5
            for x, y in zip(sums, (ds.T @ qd, p.T @ gd, ds.abs().T @ qd.abs(), p.T @ gd.abs())):
                x += y
        # as over many chunks: P and dS once rounded, and the result; P off by 2 LSE_TOL; fp32 sums of 1024
        # rows in the tensor core and 1025 parts lose less than 2^-12 of the magnitudes
        for name, got, total, size in (("dk", dk, sums[0], sums[2]), ("dv", dv, sums[1], sums[3])):
            bound = 1.02 * ref.U * (total.abs() + size) + (2 * LSE_TOL + 2.0 ** -12) * size + 1e-6
            close(got[0, :s, e], total.cpu().numpy(), bound.cpu().numpy(), name)


def test_caches_of_more_than_2_31_elements():
    torch = torch_cuda()
    b, hk, h, d, w, s, tail = 3, 4, 8, 128, 40, 4, 64
    cap = 1 << 22
    ends = [rand(i, b, s + tail, hk, d)[0] for i in (1, 2)]
    q, qf = rand(3, b, 1, h, d)
    lengths = torch.full((b,), cap, dtype=torch.int32, device="cuda")
    first = torch.zeros(b, dtype=torch.int32, device="cuda")
    kf, vf = (bf16_to_f64(x) for x in ends)
    cache = sa.cache4_alloc(b, cap, hk, d)
    assert cache.k_codes.numel() > 1 << 31
    sa.cache4_append(cache, *(x[:, :s] for x in ends), first)
    sa.cache4_append(cache, *(x[:, s:] for x in ends), first + (cap - tail))
    back = sa.cache4_read(cache, first + (cap - tail), tail)
    o, lse = sa.sink_attn_decode_cache4(q, cache, lengths, w, s)
    status_ok()
    k4, v4 = (ref.values(*ref.quantise(x)) for x in (kf, vf))
    for x, y in zip(back, (k4, v4)):
        assert np.array_equal(bf16_to_f64(x), ref.bf16_round(y[:, s:]))
    of, lf, ob = ref.sink_decode(qf, k4, v4, [s + tail] * b, w, s)
    close(o, of, ob, "o")
    close(lse, lf, LSE_TOL, "lse")
    del cache, back
    k, v = (torch.empty(b, cap, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 1 << 32
    for x, e in ((k, ends[0]), (v, ends[1])):
        x[:, :s] = e[:, :s]
        x[:, -tail:] = e[:, s:]
    o, lse = sa.sink_attn_decode(q, k, v, lengths, w, s)
    status_ok()
    of, lf, ob = ref.sink_decode(qf, kf, vf, [s + tail] * b, w, s)
    close(o, of, ob, "o")
    close(lse, lf, LSE_TOL, "lse")


class Guard:
    """bf16, fp32 or byte tensors inside poisoned buffers; `check` finds any byte changed around them."""

    def __init__(self):
        self.kept = []

    def __call__(self, *shape, dtype=None, every_other_head=False):
        torch = torch_cuda()
        dtype = dtype or torch.bfloat16
        full = list(shape)
        if every_other_head:
            full[2] *= 2
        size = int(np.prod(full)) * torch.empty(0, dtype=dtype).element_size()
        raw = torch.full((size + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        t = raw[4096:4096 + size].view(dtype).view(full)
        self.kept += [raw[:4096], raw[-4096:]] + ([t[:, :, 1::2]] if every_other_head else [])
        return t[:, :, ::2] if every_other_head else t

    def check(self):
        torch = torch_cuda()
        assert all(bool((x.contiguous().view(torch.uint8) == 0x5A).all()) for x in self.kept)


@pytest.mark.parametrize("n,d", [(1, 128), (333, 64), (130, 32)])
def test_nothing_is_written_around_the_outputs(n, d):
    torch = torch_cuda()
    b, h, hk, w, s = 2, 4, 2, 70, 9
    f32 = torch.float32
    x = {i: rand(i, b, n, h if i in (0, 3) else hk, d)[0] for i in range(5)}
    q, k, v, g = x[0], x[1], x[2], x[3]
    weight = torch.ones(d, dtype=f32, device="cuda")
    freq = 100.0 ** -np.arange(d // 2)
    guard = Guard()
    qo, ko = guard(b, n, h, d, every_other_head=True), guard(b, n, hk, d, every_other_head=True)
    sa.sa_qk_norm_rope_fwd(q, k, weight, weight, freq, None, qo, ko)
    dqw, dkw = guard(d, dtype=f32), guard(d, dtype=f32)
    dq, dk = guard(b, n, h, d, every_other_head=True), guard(b, n, hk, d, every_other_head=True)
    ws = guard(sa.sa_qk_norm_rope_bwd_workspace_size(d), dtype=torch.uint8)
    sa.sa_qk_norm_rope_bwd(q, k, g, x[4], weight, weight, freq, None, dq, dk, dqw, dkw, ws)
    o, lse = guard(b, n, h, d, every_other_head=True), guard(b, h, n, dtype=f32)
    sa.sa_sink_attn_fwd(q, k, v, w, s, o, lse)
    dq, dk, dv = (guard(b, n, e, d, every_other_head=True) for e in (h, hk, hk))
    ws = guard(sa.sa_sink_attn_bwd_workspace_size(b, n, h, hk, d, w, s), dtype=torch.uint8)
    sa.sa_sink_attn_bwd(q, k, v, o, g, lse, w, s, dq, dk, dv, ws)
    lengths = torch.tensor([n, max(0, n - 3)], dtype=torch.int32, device="cuda")
    o, lse = guard(b, 1, h, d, every_other_head=True), guard(b, h, 1, dtype=f32)
    sa.sa_sink_attn_decode(q[:, :1], k, v, lengths, w, s, o, lse)
    cap = -(-n // 8) * 8
    u8, bf16 = torch.uint8, torch.bfloat16
    cache = sa.Cache4(guard(b, hk, cap, d // 2, dtype=u8), guard(b, hk, cap, d // 32, dtype=bf16),
                      guard(b, hk, cap, d // 2, dtype=u8), guard(b, hk, cap, d // 32, dtype=bf16))
    sa.sa_cache4_append(cache, k, v)
    ko, vo = (guard(b, n, hk, d, every_other_head=True) for _ in range(2))
    sa.sa_cache4_read(cache, None, ko, vo)
    o, lse = guard(b, 1, h, d, every_other_head=True), guard(b, h, 1, dtype=f32)
    sa.sa_sink_attn_decode_cache4(q[:, :1], cache, lengths, w, s, o, lse)
    status_ok()
    guard.check()


def test_captured_and_replayed_on_new_inputs():
    """One CUDA graph of the whole chain, replayed after its inputs changed."""
    torch = torch_cuda()
    b, n, h, hk, d, w, s, cap = 2, 260, 4, 2, 64, 60, 4, 264
    packed, _, wts, freq = _model(2, b, n, h, hk, d)
    wt = [torch.from_numpy(x).cuda() for x in wts]
    g, _ = rand(8, b, n, h, d)
    cache = sa.cache4_alloc(b, cap, hk, d)
    lengths = torch.tensor([n, 131], dtype=torch.int32, device="cuda")

    def chain():
        q, k, v = packed[:, :, :h], packed[:, :, h:h + hk], packed[:, :, h + hk:]
        qr, kr = sa.qk_norm_rope_fwd(q, k, *wt, freq)
        o, lse = sa.sink_attn_fwd(qr, kr, v, w, s)
        grads = sa.sink_attn_bwd(qr, kr, v, o, lse, g, w, s)
        back = sa.qk_norm_rope_bwd(q, k, grads[0], grads[1], *wt, freq)
        sa.cache4_append(cache, kr, v)
        last = qr[:, -1:].contiguous()
        return (o, lse) + grads + back + sa.sink_attn_decode(last, kr, v, lengths, w, s) + \
            sa.sink_attn_decode_cache4(last, cache, lengths, w, s) + sa.cache4_read(cache, None, n)

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain()
    for seed in (21, 22):
        packed.copy_(rand(seed, *packed.shape)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        for x, y in zip(got, chain()):
            assert torch.equal(x, y)
    status_ok()


def test_two_streams_at_once():
    """The same calls on two streams with separate outputs and workspaces do not meet."""
    torch = torch_cuda()
    b, n, h, hk, d, w, s = 1, 2000, 8, 2, 128, 300, 4
    sets = []
    for i in range(2):
        t = [rand(10 * i + j, b, n, x, d)[0] for j, x in enumerate((h, hk, hk, h))]
        sets.append(t)

    def both(q, k, v, g):
        o, lse = sa.sink_attn_fwd(q, k, v, w, s)
        return (o, lse) + sa.sink_attn_bwd(q, k, v, o, lse, g, w, s)

    want = [both(*t) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for rep in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = both(*sets[i])
    torch.cuda.synchronize()
    status_ok()
    for a, c in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, c))


# ------------------------------------------------------------------ several rounds of every loop

def several_per_sm(items):
    count = torch_cuda().cuda.get_device_properties(0).multi_processor_count
    assert items >= 3 * count, (items, count)


@pytest.mark.parametrize("b,n,h,hk,d,w,s", [(14, 517, 14, 7, 32, 150, 5), (14, 520, 14, 7, 64, 100, 70),
                                            (14, 515, 14, 7, 128, 60, 9), (14, 530, 14, 7, 64, 600, 0)])
def test_sink_attention_with_several_items_a_cta(b, n, h, hk, d, w, s):
    """Persistent CTAs that take three work items and more, forward, dQ and dK / dV, every row checked."""
    several_per_sm(b * hk * -(-n // 128))
    (q, qf), (k, kf), (v, vf), (g, gf) = (rand(i, b, n, x, d) for i, x in enumerate((h, hk, hk, h)))
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    grads = sa.sink_attn_bwd(q, k, v, o, lse, g, w, s)
    status_ok()
    of, lf, ob = ref.sink_attention(qf, kf, vf, w, s)
    close(o, of, ob, "o")
    close(lse, lf, LSE_TOL, "lse")
    want, bounds = ref.sink_attention_backward(qf, kf, vf, gf, w, s)
    for name, x, y, e in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(x, y, e, name)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_sinks_gradients_over_many_chunks(d):
    """The sinks' keys and values gather from every query of a long sequence, in some 50 partial sums; P and
    D in float64 from the forward's outputs."""
    torch = torch_cuda()
    n, h, hk, w, s = 50021, 4, 2, 60, 6
    q, k, v, g = (rand(i, 1, n, x, d)[0] for i, x in enumerate((h, hk, hk, h)))
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    _, dk, dv = sa.sink_attn_bwd(q, k, v, o, lse, g, w, s)
    status_ok()
    i, j = torch.arange(n, device="cuda")[:, None], torch.arange(s, device="cuda")[None]
    for hd in range(hk):
        want_k, want_v, size_k, size_v = (torch.zeros(s, d, dtype=torch.float64, device="cuda") for _ in range(4))
        for e in range(hd * h // hk, (hd + 1) * h // hk):
            qd, gd, od = (x[0, :, e].double() for x in (q, g, o))
            kd, vd = (x[0, :s, hd].double() for x in (k, v))
            p = torch.where(j <= i, torch.exp(qd @ kd.T * d ** -0.5 - lse[0, e].double()[:, None]), 0.0)
            ds = p * (gd @ vd.T - (gd * od).sum(-1, keepdim=True)) * d ** -0.5
            want_k += ds.T @ qd
            want_v += p.T @ gd
            size_k += ds.abs().T @ qd.abs()
            size_v += p.T @ gd.abs()
        # P and dS once rounded, and the result; P itself is off by 2 LSE_TOL; fp32 sums of some 130 rows a step,
        # 400 steps and 50 parts lose less than 2^-12 of the magnitudes
        for name, got, want, size in (("dk", dk, want_k, size_k), ("dv", dv, want_v, size_v)):
            bound = 1.02 * ref.U * (want.abs() + size) + (2 * LSE_TOL + 2.0 ** -12) * size + 1e-6
            close(got[0, :s, hd], want.cpu().numpy(), bound.cpu().numpy(), name)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_sink_attention_backward_of_large_scores(d):
    n, w, s = 400, 90, 6
    (q, qf), (k, kf) = rand(0, 1, n, 2, d, scale=6.0), rand(1, 1, n, 1, d, scale=6.0)
    (v, vf), (g, gf) = rand(2, 1, n, 1, d), rand(3, 1, n, 2, d)
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    grads = sa.sink_attn_bwd(q, k, v, o, lse, g, w, s)
    status_ok()
    want, bounds = ref.sink_attention_backward(qf, kf, vf, gf, w, s)
    # |s| up to 400: scores and LSE are each off by up to 400 x 2^-20, so P by 8e-4 of itself and O by
    # twice that of P |v|. dS then gains 8e-4 |dS| + 16e-4 P |dO| P |v| and P 8e-4 P, at most 16e-4 / U = 0.41 of what
    # the bounds hold for the roundings of P, dS and O
    for name, x, y, e in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(x, y, 1.41 * e, name)


@pytest.mark.parametrize("b,n,h,hk,d,rotary,inter", [(3, 3001, 29, 5, 32, 32, False), (3, 3001, 13, 5, 64, 64, True),
                                                     (3, 3001, 13, 5, 128, 128, False), (3, 3001, 13, 5, 128, 64, True),
                                                     (2, 501, 40, 5, 128, 128, False), (7, 700, 31, 2, 64, 32, False)])
def test_norm_rope_with_several_tokens_a_warp(b, n, h, hk, d, rotary, inter):
    """Warps that take several tokens (or ranges of a token's heads) in several batches; the backward also
    over its own inputs."""
    torch = torch_cuda()
    several_per_sm(b * n / 8 if h < 40 else b * n * 9 / 8 / 2)
    rng = np.random.default_rng(6)
    (q, qf), (k, kf), (gq, gqf), (gk, gkf) = (rand(i, b, n, x, d) for i, x in enumerate((h, hk, h, hk)))
    w = [np.float32(1 + 0.2 * rng.standard_normal(d)) for _ in range(2)]
    wt = [torch.from_numpy(x).cuda() for x in w]
    freq = 10000.0 ** (-2.0 * np.arange(rotary // 2) / rotary)
    pos = rng.integers(0, 1 << 20, (b, n))
    pt = torch.from_numpy(pos.astype(np.int32)).cuda()
    outs = sa.qk_norm_rope_fwd(q, k, *wt, freq, pt, 1e-5, inter)
    grads = sa.qk_norm_rope_bwd(q, k, gq, gk, *wt, freq, pt, 1e-5, inter)
    status_ok()
    for name, y, dx, dw, xf, gf, wf in zip("qk", outs, grads[:2], grads[2:], (qf, kf), (gqf, gkf), w):
        want, bound = ref.norm_rope(xf, wf.astype(np.float64), pos, freq, 1e-5, inter)
        close(y, want, bound, name + "_out")
        (dxf, dwf), (bx, bw) = ref.norm_rope_backward(xf, wf.astype(np.float64), gf, pos, freq, 1e-5, inter)
        close(dx, dxf, bx, "d" + name)
        close(dw, dwf, bw, "dw_" + name)
    dqw, dkw = torch.empty_like(wt[0]), torch.empty_like(wt[1])
    ws = torch.empty(sa.sa_qk_norm_rope_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    sa.sa_qk_norm_rope_bwd(q, k, gq, gk, *wt, freq, pt, gq, gk, dqw, dkw, ws, 1e-5, inter)
    sa.sa_qk_norm_rope_fwd(q, k, *wt, freq, pt, q, k, 1e-5, inter)
    status_ok()
    assert all(torch.equal(x, y) for x, y in zip((q, k, gq, gk, dqw, dkw), outs + grads))


@pytest.mark.parametrize("cache4", [False, True])
@pytest.mark.parametrize("h,hk,d", [(4, 2, 32), (24, 2, 32), (4, 2, 64), (24, 2, 64), (4, 2, 128), (24, 2, 128)])
def test_decode_with_several_rounds_of_the_ring(h, hk, d, cache4):
    """Long sequences: every CTA fills its ring three times and more; the scores grow along the sequence, so
    that the running maximum is followed again and again."""
    torch = torch_cuda()
    cap, w, s, lengths = 16384, 16100, 70, [16384, 16201, 13007]
    b = len(lengths)
    q, qf = rand(0, b, 1, h, d)
    v, vf = rand(2, b, cap, hk, d)
    k = torch.randn(b, cap, hk, d, generator=torch.Generator().manual_seed(1))
    k = (k * torch.linspace(0.1, 4.0, cap)[:, None, None]).to(torch.bfloat16).cuda()
    kf = bf16_to_f64(k)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if cache4:
        cache = sa.cache4_alloc(b, cap, hk, d)
        sa.cache4_append(cache, k, v)
        o, lse = sa.sink_attn_decode_cache4(q, cache, n, w, s)
        kf, vf = (ref.values(*ref.quantise(x)) for x in (kf, vf))
    else:
        o, lse = sa.sink_attn_decode(q, k, v, n, w, s)
    status_ok()
    of, lf, ob = ref.sink_decode(qf, kf, vf, lengths, w, s)
    close(o, of, ob, "o")
    close(lse, lf, LSE_TOL, "lse")


FRESH = '''
import threading
import numpy as np, torch
import content_adaptive_sparse_gb300 as sa

b, n, h, hk, d, w, s, threads, calls = 1, 200, 4, 2, 64, 30, 3, 8, 24
gen = torch.Generator(device="cuda").manual_seed(1)
q, k, v, g = (torch.randn(b, n, x, d, generator=gen, device="cuda").bfloat16() for x in (h, hk, hk, h))
length = torch.tensor([n], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()

def chain(i):
    freq = (100.0 + i) ** (-np.arange(d // 2) / 32.0)
    qr, kr = sa.qk_norm_rope_fwd(q, k, None, None, freq)
    o, lse = sa.sink_attn_fwd(qr, kr, v, w, s)
    cache = sa.cache4_alloc(b, n, hk, d)
    sa.cache4_append(cache, kr, v)
    return (qr, kr, o, lse) + sa.sink_attn_bwd(qr, kr, v, o, lse, g, w, s) + sa.sink_attn_decode_cache4(qr[:, -1:], cache, length, w, s)

start = threading.Barrier(threads)
got, errors = {}, []

def work(t):
    try:
        start.wait()
        with torch.cuda.stream(torch.cuda.Stream()):
            for c in range(calls):
                got[t, c] = chain(t * calls + c)
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        errors.append(repr(e))

pool = [threading.Thread(target=work, args=(t,)) for t in range(threads)]
for t in pool: t.start()
for t in pool: t.join()
assert not errors, errors
for (t, c), x in got.items():
    assert all(torch.equal(a, e) for a, e in zip(x, chain(t * calls + c))), (t, c)
torch.cuda.synchronize()
assert sa.sa_device_status() == 0
'''


def in_a_fresh_process(script):
    import os
    import subprocess
    import sys
    torch_cuda()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-3000:]


def test_first_calls_from_several_host_threads():
    """A process whose first calls come from eight threads at once, each on a stream and with frequency
    tables of its own (192 in all)."""
    in_a_fresh_process(FRESH)


CAPTURED = '''
import numpy as np, torch
import content_adaptive_sparse_gb300 as sa
b, n, h, hk, d, w, s = 2, 300, 4, 2, 64, 30, 3
torch.manual_seed(0)
q, k, v, g = (torch.randn(b, n, x, d, device="cuda").bfloat16() for x in (h, hk, hk, h))
length = torch.tensor([n, 100], dtype=torch.int32, device="cuda")
freq = 100.0 ** (-np.arange(d // 2) / 32.0)
cache = sa.cache4_alloc(b, 304, hk, d)
wt = torch.ones(d, device="cuda")
def chain():
    qr, kr = sa.qk_norm_rope_fwd(q, k, wt, wt, freq)
    o, lse = sa.sink_attn_fwd(qr, kr, v, w, s)
    gr = sa.sink_attn_bwd(qr, kr, v, o, lse, g, w, s)
    back = sa.qk_norm_rope_bwd(q, k, gr[0], gr[1], wt, wt, freq)
    sa.cache4_append(cache, kr, v)
    return (o, lse) + gr + back + sa.sink_attn_decode(qr[:, -1:], kr, v, length, w, s) + sa.sink_attn_decode_cache4(qr[:, -1:], cache, length, w, s) + sa.cache4_read(cache, None, n)
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    outs = chain()
gr.replay(); torch.cuda.synchronize()
got = [x.clone() for x in outs]
assert all(torch.equal(x, y) for x, y in zip(got, chain()))
torch.cuda.synchronize(); assert sa.sa_device_status() == 0
'''


def test_first_calls_inside_a_capture():
    """A process that captures every call into a graph before it has made it once."""
    in_a_fresh_process(CAPTURED)
