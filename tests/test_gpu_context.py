"""Shared contexts and bounded caches on the GPU against float64 (oracle/streaming.py, oracle/context.py):
norm and rotation with several axes, attention behind a shared prefix, the cache of slots with
accumulated weights, and runs of them together. Tolerances are the oracles' elementwise bounds."""
import numpy as np
import pytest

import content_adaptive_sparse_gb300 as sa
from gpu_helpers import torch_cuda
from oracle import context as oc
from oracle import streaming as ref
from test_gpu_streaming import LSE_TOL, close, rand, status_ok

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norm and rotation with several axes

AXES_CASES = [
    # batch, tokens, heads, kv_heads, dim, rotary, axes, axis of each pair, interleaved, weights
    (1, 1, 1, 1, 32, 32, 1, "runs", False, True), (2, 3, 5, 2, 64, 64, 3, "runs", False, True), (1, 7, 4, 4, 128, 128, 3, "turns", True, True),
    (1, 40, 3, 1, 128, 64, 2, "runs", False, False), (2, 33, 12, 12, 64, 32, 4, "turns", True, True),
    (1, 129, 2, 1, 32, 16, 8, "turns", False, True), (1, 5, 9, 1, 64, 0, 2, "runs", False, True),
    (3, 1, 16, 4, 128, 128, 3, "runs", False, True), (2, 700, 6, 2, 32, 32, 3, "random", True, False),
    (3, 3001, 13, 5, 128, 128, 3, "random", False, True), (3, 3001, 13, 5, 64, 64, 2, "random", True, True),
]


@pytest.mark.parametrize("b,n,h,hk,d,rotary,axes,which,inter,weights", AXES_CASES)
def test_norm_rope_of_several_axes(b, n, h, hk, d, rotary, axes, which, inter, weights):
    torch = torch_cuda()
    rng = np.random.default_rng(5)
    packed, pf = rand(0, b, n, h + 2 * hk, d)
    packed[0, 0, 0] = 0.0                                  # a row of zeros
    pf[0, 0, 0] = 0.0
    q, k, qf, kf = packed[:, :, :h], packed[:, :, h:h + hk], pf[:, :, :h], pf[:, :, h:h + hk]
    (gq, gqf), (gk, gkf) = rand(1, b, n, h, d), rand(2, b, n, hk, d)
    w = [np.float32(1 + 0.2 * rng.standard_normal(d)) if weights else np.ones(d, np.float32) for _ in range(2)]
    wt = [torch.from_numpy(x).cuda() if weights else None for x in w]
    half = rotary // 2
    freq = 10000.0 ** (-2.0 * np.arange(half) / max(rotary, 1))
    pair = {"runs": [p * axes // max(half, 1) for p in range(half)], "turns": [p % axes for p in range(half)],
            "random": rng.integers(0, axes, half).tolist()}[which]
    pos = rng.integers(-(1 << 30), 1 << 30, (b, n, axes))
    pt = torch.from_numpy(pos.astype(np.int32)).cuda()
    each = pos[:, :, pair]
    args = (*wt, freq, pair, pt, 1e-5, inter)
    outs = sa.qk_norm_rope_axes_fwd(q, k, *args)
    status_ok()
    for name, x, xf, wf in zip("qk", outs, (qf, kf), w):
        y, bound = ref.norm_rope(xf, wf.astype(np.float64), each, freq, 1e-5, inter)
        close(x, y, bound, name + "_out")
    grads = sa.qk_norm_rope_axes_bwd(q, k, gq, gk, *args)
    status_ok()
    for name, x, dw, xf, gf, wf in zip("qk", grads[:2], grads[2:], (qf, kf), (gqf, gkf), w):
        (dxf, dwf), (bx, bw) = ref.norm_rope_backward(xf, wf.astype(np.float64), gf, each, freq, 1e-5, inter)
        close(x, dxf, bx, "d" + name)
        if weights:
            close(dw, dwf, bw, "dw_" + name)
        else:
            assert dw is None
    # over their own inputs, and the same bits
    dws = [torch.empty_like(x) if x is not None else None for x in wt]
    ws = torch.empty(sa.sa_qk_norm_rope_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    sa.sa_qk_norm_rope_axes_bwd(q, k, gq, gk, *wt, freq, pair, pt, gq, gk, *dws, ws, 1e-5, inter)
    sa.sa_qk_norm_rope_axes_fwd(q, k, *wt, freq, pair, pt, q, k, 1e-5, inter)
    status_ok()
    for x, y in zip((q, k, gq, gk, *dws), outs + grads):
        assert (x is None and y is None) or torch.equal(x, y)


@pytest.mark.parametrize("inter", [False, True])
def test_equal_axes_are_one_axis(inter):
    """Every axis at the token's position: the bits of the one-axis calls."""
    torch = torch_cuda()
    b, n, h, hk, d = 2, 70, 6, 2, 128
    q, k, gq, gk = (rand(i, b, n, x, d)[0] for i, x in enumerate((h, hk, h, hk)))
    w = 1 + 0.1 * torch.randn(d, device="cuda")
    freq = 10000.0 ** (-2.0 * np.arange(d // 2) / d)
    pos = torch.randint(0, 1 << 30, (b, n), dtype=torch.int32, device="cuda")
    pair = [p % 3 for p in range(d // 2)]
    wide = pos[:, :, None].expand(b, n, 3).contiguous()
    got = sa.qk_norm_rope_axes_fwd(q, k, w, w, freq, pair, wide, 1e-6, inter) + \
        sa.qk_norm_rope_axes_bwd(q, k, gq, gk, w, w, freq, pair, wide, 1e-6, inter)
    want = sa.qk_norm_rope_fwd(q, k, w, w, freq, pos, 1e-6, inter) + sa.qk_norm_rope_bwd(q, k, gq, gk, w, w, freq, pos, 1e-6, inter)
    status_ok()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


# ------------------------------------------------------------------ attention behind a shared prefix

PREFIX_CASES = [
    # batch, tokens, prefix, heads, kv_heads, dim, window
    (1, 1, 1, 1, 1, 32, 0), (1, 1, 0, 2, 1, 64, 0), (2, 3, 0, 4, 2, 128, 1), (1, 2, 127, 2, 2, 64, 9), (3, 5, 128, 6, 2, 128, 4),
    (2, 7, 129, 5, 1, 32, 2), (1, 33, 300, 12, 12, 64, 32), (4, 37, 1000, 8, 2, 128, 36), (9, 19, 513, 12, 1, 64, 5),
    (1, 128, 128, 2, 1, 64, 127), (2, 129, 64, 3, 1, 128, 40), (1, 300, 5, 4, 4, 32, 299), (2, 260, 700, 6, 3, 64, 17),
    (1, 500, 2000, 2, 1, 128, 130), (5, 100, 1, 7, 7, 64, 99), (40, 3, 260, 4, 2, 64, 2), (1, 700, 0, 4, 1, 64, 100),
    (2, 200, 333, 20, 1, 32, 1 << 40),
]


def assert_close_attention(o, lse, want, what=""):
    of, lf, ob = want
    close(o, of, ob, what + "o")
    lse = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(lse), np.isneginf(lf))
    some = ~np.isneginf(lf)
    close(lse[some], lf[some], LSE_TOL, what + "lse")


@pytest.mark.parametrize("b,n,p,h,hk,d,w", PREFIX_CASES)
def test_prefix_attention(b, n, p, h, hk, d, w):
    (q, qf), (k, kf), (v, vf) = (rand(i, b, n, x, d) for i, x in enumerate((h, hk, hk)))
    (kp, kpf), (vp, vpf) = (rand(i, 1, p, hk, d) for i in (3, 4))
    o, lse = sa.prefix_attn_fwd(q, kp, vp, k, v, w)
    status_ok()
    assert_close_attention(o, lse, oc.prefix_attention(qf, kpf, vpf, kf, vf, w))


PREFIX_DECODE_CASES = [
    # heads, kv_heads, dim, prefix, capacity, window, lengths
    (1, 1, 32, 1, 1, 0, [1]), (2, 1, 64, 0, 16, 3, [0, 1, 16]), (2, 1, 64, 5, 16, 3, [0, 1, 16]), (4, 4, 128, 128, 64, 100, [64, 63, 1, 0]),
    (8, 2, 64, 1000, 70, 16, [70, 40, 17, 16, 9]), (16, 1, 128, 129, 200, 50, [200, 84]), (20, 1, 64, 777, 136, 65, [136, 5, 0]),
    (40, 2, 32, 3000, 260, 500, [260, 130]), (6, 3, 128, 5000, 1000, 700, [1000, 900, 701, 128]), (12, 12, 64, 300, 520, 511, [7, 520, 519] * 9),
    (4, 1, 64, 20000, 3, 2, [3]), (3, 1, 128, 400, 40, 1 << 33, [40] * 50),
]


@pytest.mark.parametrize("h,hk,d,p,cap,w,lengths", PREFIX_DECODE_CASES)
def test_prefix_decode(h, hk, d, p, cap, w, lengths):
    """Own rows that the query does not see hold NaN and infinities."""
    torch = torch_cuda()
    b = len(lengths)
    q, qf = rand(0, b, 1, h, d)
    (k, kf), (v, vf) = (rand(i, b, cap, hk, d) for i in (1, 2))
    (kp, kpf), (vp, vpf) = (rand(i, 1, p, hk, d) for i in (3, 4))
    j = torch.arange(cap, device="cuda")
    for i, n in enumerate(lengths):
        unseen = (j >= n) | (n - 1 - j > w)
        k[i, unseen] = float("nan")
        v[i, unseen] = float("inf")
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, lse = sa.prefix_attn_decode(q, kp, vp, k, v, n, w)
    status_ok()
    assert_close_attention(o, lse, oc.prefix_decode(qf, kpf, vpf, kf, vf, lengths, w))


# ------------------------------------------------------------------ a cache of slots with accumulated weights

SCORED_CASES = [
    # heads, kv_heads, dim, capacity, decay, lengths
    (1, 1, 32, 1, 1.0, [1]), (2, 1, 64, 16, 1.0, [0, 1, 16]), (4, 4, 128, 64, 0.5, [64, 63, 1]), (8, 2, 64, 71, 0.0, [71, 40, 17, 16]),
    (16, 1, 128, 200, 0.9, [200, 84, 51, 3]), (20, 1, 64, 136, 1.0, [136, 5]), (40, 2, 32, 264, 0.99, [264, 130, 0]),
    (128, 1, 64, 333, 1.0, [333, 64]), (6, 3, 128, 1000, 1.0, [1000, 900, 701, 128]), (3, 1, 64, 4096, 0.75, [4096, 4001, 2]),
    (24, 2, 32, 6000, 1.0, [5999, 3071, 3001, 10]), (5, 5, 128, 2048, 1.0, [2000]), (12, 12, 64, 520, 1.0, [7, 520, 519]),
]


@pytest.mark.parametrize("h,hk,d,cap,decay,lengths", SCORED_CASES)
def test_scored_decode(h, hk, d, cap, decay, lengths):
    """Slots past the lengths hold NaN and infinities, and their weights stay as they were."""
    torch = torch_cuda()
    b = len(lengths)
    q, qf = rand(0, b, 1, h, d)
    (k, kf), (v, vf) = (rand(i, b, cap, hk, d) for i in (1, 2))
    wf = np.float32(np.random.default_rng(3).exponential(size=(b, hk, cap)))
    for i, n in enumerate(lengths):
        k[i, n:] = float("nan")
        v[i, n:] = float("inf")
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    w = torch.from_numpy(wf).cuda()
    cache = sa.ScoredCache(k, v, w.clone(), torch.zeros(b, hk, cap, dtype=torch.int32, device="cuda"))
    out = torch.full_like(w, -7.0)
    o, lse = sa.scored_attn_decode(q, cache, n, decay, out)
    status_ok()
    of, lf, ob, want, bound = oc.scored_decode(qf, kf, vf, lengths, wf.astype(np.float64), decay)
    assert_close_attention(o, lse, (of, lf, ob))
    assert torch.equal(cache.weights, w)
    unseen = torch.arange(cap, device="cuda") >= n[:, None, None]
    assert (out[unseen.expand_as(out)] == -7.0).all()
    close(torch.where(unseen, w, out), want, bound, "weights")
    o2, lse2 = sa.scored_attn_decode(q, cache, n, decay)
    status_ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(cache.weights, torch.where(unseen, w, out))


def test_scored_append():
    torch = torch_cuda()
    b, cap, hk, d, n = 3, 20, 2, 64, 5
    (k, _), (v, _) = (rand(i, b, n, 2 * hk, d) for i in (1, 2))
    k, v = k[:, :, ::2], v[:, :, hk:]
    cache = sa.scored_alloc(b, cap, hk, d)
    for x in cache:
        x.fill_(9)
    start = torch.tensor([-1, 4, 17], dtype=torch.int32, device="cuda")
    tokens = torch.tensor([5, 1000, 2**31 - 3], dtype=torch.int32, device="cuda")
    want = [x.clone() for x in cache]
    sa.scored_append(cache, k, v, start, tokens)
    torch.cuda.synchronize()
    assert sa.sa_device_status() == -6                    # two rows of the third sequence did not fit
    for s, (at, m, tok) in ((1, (4, 5, 1000)), (2, (17, 3, 2**31 - 3))):
        want[0][s, at:at + m] = k[s, :m]
        want[1][s, at:at + m] = v[s, :m]
        want[2][s, :, at:at + m] = 0
        want[3][s, :, at:at + m] = (tok + torch.arange(m, device="cuda")).to(torch.int32)
    assert all(torch.equal(x, y) for x, y in zip(cache, want))
    sa.scored_append(cache, k, v)
    status_ok()
    assert torch.equal(cache.k[:, :n], k) and torch.equal(cache.v[:, :n], v) and not cache.weights[:, :, :n].any()
    assert torch.equal(cache.positions[:, :, :n], torch.arange(n, dtype=torch.int32, device="cuda").expand(b, hk, n))


EVICT_CASES = [
    # batch, capacity, kv_heads, dim, lengths, keep, sinks, recent
    (1, 1, 1, 32, [1], 1, 0, 0), (2, 8, 2, 64, [8, 3], 3, 1, 1), (3, 40, 1, 128, [0, 40, 11], 10, 0, 10), (2, 33, 3, 32, [33, 32], 32, 4, 8),
    (4, 700, 2, 64, [700, 699, 513, 20], 512, 4, 100), (2, 700, 2, 128, [700, 400], 30, 4, 0), (1, 5000, 3, 32, [5000], 4999, 0, 0),
    (2, 4104, 4, 128, [4097, 4104], 4096, 4, 512), (1, 9000, 2, 64, [9000], 1, 0, 1), (3, 3000, 2, 32, [3000, 2999, 1501], 1500, 16, 700),
    (1, 20000, 2, 32, [20000], 9000, 4, 1000), (2, 17001, 1, 64, [17001, 16999], 16998, 1, 1), (2, 50, 2, 64, [50, 49], 60, 0, 0),
    (1, 33000, 2, 32, [33000], 20000, 4, 1000), (2, 8192, 1, 32, [8192, 8191], 4096, 0, 4096), (2, 8193, 1, 64, [8193, 100], 4000, 100, 0),
]


def evict_inputs(b, cap, hk, d, ties=False):
    torch = torch_cuda()
    rng = np.random.default_rng(7)
    k, v = rand(1, b, cap, hk, d)[0], rand(2, b, cap, hk, d)[0]
    w = np.float32(np.exp(2 * rng.standard_normal((b, hk, cap))))
    if ties:
        w = np.float32(rng.integers(0, 3, (b, hk, cap)))
    pos = np.stack([np.stack([rng.permutation(2 * cap)[:cap] for _ in range(hk)]) for _ in range(b)]).astype(np.int32)
    return k, v, torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()


def bits(t):
    torch = torch_cuda()
    return t.contiguous().view({2: torch.int16, 4: torch.int32}[t.element_size()])


def check_evict(k, v, w, pos, lengths, keep, sinks, recent):
    """Out of place and over its inputs, against the oracle, bit by bit."""
    torch = torch_cuda()
    kb, vb = bits(k).cpu().numpy(), bits(v).cpu().numpy()
    want = oc.evict(kb, vb, w.cpu().numpy(), pos.cpu().numpy(), lengths, keep, sinks, recent)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    used = torch.arange(w.shape[2], device="cuda") < torch.tensor(want[4], device="cuda")[:, None, None]
    for over in (False, True):
        cache = sa.ScoredCache(k.clone(), v.clone(), w.clone(), pos.clone())
        m = n.clone()
        outs = () if over else (torch.full_like(w, -1.0), torch.full_like(pos, -1), torch.full_like(n, -1))
        got = sa.scored_evict(cache, m, keep, sinks, recent, *outs)
        status_ok()
        assert np.array_equal(bits(cache.k).cpu().numpy(), want[0]) and np.array_equal(bits(cache.v).cpu().numpy(), want[1])
        for x, y, before in ((got[0], want[2], w), (got[1], want[3], pos)):
            y = torch.from_numpy(y).cuda()
            rest = before if over else torch.full_like(before, -1)
            assert torch.equal(bits(x), bits(torch.where(used, y, rest)))
        assert got[2].tolist() == want[4] and (over or m.tolist() == lengths)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("b,cap,hk,d,lengths,keep,sinks,recent", EVICT_CASES)
def test_evict(b, cap, hk, d, lengths, keep, sinks, recent, ties):
    check_evict(*evict_inputs(b, cap, hk, d, ties), lengths, keep, sinks, recent)


def test_evict_of_weights_that_are_not_numbers():
    """NaN counts as the largest weight, -0 as 0; infinities and negative weights are in order."""
    torch = torch_cuda()
    b, cap, hk, d = 2, 300, 2, 64
    k, v, w, pos = evict_inputs(b, cap, hk, d)
    for i, x in enumerate((float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -3.0, 1e-42, -1e-42)):
        w[:, :, i::17] = x
    w[0, 0, 5] = torch.tensor(-1, dtype=torch.int32).view(torch.float32)      # a NaN with its sign set
    for keep in (1, 20, 40, 150, 280):
        check_evict(k, v, w, pos, [300, 299], keep, 0, 0)


# ------------------------------------------------------------------ the weights of a prompt

WEIGHTS_CASES = [
    # batch, tokens, heads, kv_heads, dim, window, sinks, first
    (1, 1, 1, 1, 32, 0, 0, 0), (2, 2, 2, 1, 64, 1, 0, 1), (1, 127, 2, 2, 128, 126, 0, 0), (2, 128, 2, 1, 64, 32, 33, 5), (1, 129, 3, 1, 32, 500, 0, 128),
    (1, 300, 4, 1, 64, 299, 0, 0), (2, 257, 6, 3, 128, 128, 5, 100), (1, 640, 2, 1, 64, 0, 128, 0), (1, 641, 3, 3, 32, 255, 0, 640),
    (1, 1500, 2, 1, 64, 127, 4, 0), (1, 1500, 2, 1, 128, 127, 4, 1400), (1, 1411, 4, 2, 128, 1410, 0, 700), (3, 200, 5, 5, 64, 96, 64, 0),
    (1, 2900, 1, 1, 32, 3, 100, 0), (1, 2900, 1, 1, 32, 3, 0, 2800), (2, 1024, 4, 2, 64, 1023, 0, 960), (1, 513, 24, 1, 32, 512, 0, 0),
]


@pytest.mark.parametrize("b,n,h,hk,d,w,s,first", WEIGHTS_CASES)
def test_sink_weights(b, n, h, hk, d, w, s, first):
    """LSE of the queries before the first one is NaN: it is not used."""
    torch = torch_cuda()
    (q, qf), (k, kf) = (rand(i, b, n, x, d) for i, x in enumerate((h, hk)))
    _, lse = sa.sink_attn_fwd(q, k, k, w, s)
    lse[:, :, :first] = float("nan")
    got = sa.sink_attn_weights(q, k, lse, w, s, first)
    again = sa.sink_attn_weights(q, k, lse, w, s, first)
    status_ok()
    want, bound = oc.sink_weights(qf, kf, lse.double().cpu().numpy(), w, s, first)
    close(got, want, bound, "weights")
    assert torch.equal(got, again)
