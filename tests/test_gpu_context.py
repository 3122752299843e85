"""Shared contexts and bounded caches on the GPU against float64 (oracle/streaming.py, oracle/context.py):
norm and rotation with several axes, attention behind a shared prefix, the cache of slots with
accumulated weights, and runs of them together. Tolerances are the oracles' elementwise bounds."""
import numpy as np
import pytest

import content_adaptive_sparse_gb300 as sa
from gpu_helpers import torch_cuda
from oracle import context as oc
from oracle import streaming as ref
from test_gpu_streaming import LSE_TOL, Guard, close, in_a_fresh_process, rand, several_per_sm, status_ok

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


@pytest.mark.parametrize("group", [33, 48, 66, 80, 96, 97, 112])
@pytest.mark.parametrize("hk,d,cap,lengths", [(1, 64, 700, [700, 129, 3]), (2, 128, 65, [65]), (3, 32, 260, [0, 1, 260, 64, 63])])
def test_scored_decode_of_many_head_groups(group, hk, d, cap, lengths):
    """3, 5, 6 and 7 groups of 16 query heads of a key head, whose CTAs make clusters of sizes that are no powers of two."""
    torch = torch_cuda()
    b, h = len(lengths), group * hk
    (q, qf), (k, kf), (v, vf) = rand(0, b, 1, h, d), rand(1, b, cap, hk, d), rand(2, b, cap, hk, d)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    cache = sa.ScoredCache(k, v, torch.ones(b, hk, cap, device="cuda"), torch.zeros(b, hk, cap, dtype=torch.int32, device="cuda"))
    o, lse = sa.scored_attn_decode(q, cache, n, 0.75)
    status_ok()
    of, lf, ob, w, wb = oc.scored_decode(qf, kf, vf, lengths, np.ones((b, hk, cap)), 0.75)
    assert_close_attention(o, lse, (of, lf, ob))
    close(cache.weights, w, wb + 1e-30, "weights")


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


@pytest.mark.parametrize("cap,keep", [(40, 10), (300, 200), (1000, 480), (8192, 4096), (8193, 4000), (33000, 20000)])
@pytest.mark.parametrize("low", [0.1234, 0.7, 3e-39])
def test_evict_of_more_nan_than_there_is_room_for(cap, keep, low):
    """NaN beside ordinary positive weights: the lowest slots among the NaN stay. Lists of every form."""
    torch = torch_cuda()
    k, v, w, pos = evict_inputs(2, cap, 1, 32)
    w.clamp_(min=low)
    assert (w > 0).all()
    w[0, :, torch.randperm(cap, generator=torch.Generator().manual_seed(1))[:(cap + keep) // 2].cuda()] = float("nan")
    w[1, :, cap // 8:] = float("nan")
    check_evict(k, v, w, pos, [cap, cap - 1], keep, 0, 0)
    check_evict(k, v, w, pos, [cap, cap - 1], keep, 2, keep // 4)


def test_rows_after_a_nan_query_are_evicted_in_order():
    """A NaN query makes every weight NaN; rows appended behind them gather numbers, and the eviction counts those as less."""
    torch = torch_cuda()
    b, cap, hk, h, d, n, more, keep = 2, 200, 2, 4, 64, 150, 40, 100
    rows = [rand(i, b, n + more, hk, d)[0] for i in (1, 2)]
    cache = sa.scored_alloc(b, cap, hk, d)
    sa.scored_append(cache, *(x[:, :n] for x in rows))
    q = rand(0, b, 1, h, d)[0]
    lengths = torch.full((b,), n, dtype=torch.int32, device="cuda")
    bad = q.clone()
    bad[0, 0, :, 3] = float("nan")
    sa.scored_attn_decode(bad, cache, lengths)
    sa.scored_append(cache, *(x[:, n:] for x in rows), lengths, lengths)
    lengths += more
    sa.scored_attn_decode(q, cache, lengths)
    status_ok()
    assert torch.isnan(cache.weights[0, :, :n]).all() and (cache.weights[0, :, n:n + more] > 0).all() and (cache.weights[1, :, :n + more] > 0).all()
    check_evict(*cache, lengths.tolist(), keep, 4, 16)


@pytest.mark.parametrize("cap,keep", [(300, 299), (300, 100), (1500, 700), (9000, 8999), (9000, 4000)])
@pytest.mark.parametrize("over", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1)])
def test_evict_with_some_outputs_over_the_inputs(cap, keep, over):
    """Weights, positions and lengths each in place or elsewhere."""
    torch = torch_cuda()
    lengths = [cap, keep - 1, keep + 1]
    k, v, w, pos = evict_inputs(3, cap, 1, 32)
    want = oc.evict(bits(k).cpu().numpy(), bits(v).cpu().numpy(), w.cpu().numpy(), pos.cpu().numpy(), lengths, keep, 1, keep // 3)
    cache = sa.ScoredCache(k, v, w.clone(), pos.clone())
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    m = n.clone()
    outs = [x if o else torch.full_like(x, -1) for x, o in zip((cache.weights, cache.positions, m), over)]
    got = sa.scored_evict(cache, m, keep, 1, keep // 3, *outs)
    status_ok()
    assert np.array_equal(bits(k).cpu().numpy(), want[0]) and np.array_equal(bits(v).cpu().numpy(), want[1])
    used = torch.arange(cap, device="cuda") < torch.tensor(want[4], device="cuda")[:, None, None]
    for x, y, before, kept, o in ((got[0], want[2], w, cache.weights, over[0]), (got[1], want[3], pos, cache.positions, over[1])):
        assert torch.equal(bits(x), bits(torch.where(used, torch.from_numpy(y).cuda(), before if o else torch.full_like(before, -1))))
        assert o or torch.equal(kept, before)
    assert got[2].tolist() == want[4] and (over[2] or m.tolist() == lengths)


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


# ------------------------------------------------------------------ large scores, strides, NaN, many items

# |s| up to 400: fp32 scores and LSE are each off by up to about 400 x 2^-20, and P by 8e-4 of itself
LARGE_P = 8e-4


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("b,n,p,h,hk", [(2, 300, 200, 2, 1), (3, 9, 900, 4, 2)])
def test_prefix_attention_of_large_scores(b, n, p, h, hk, d):
    (q, qf), (k, kf), (kp, kpf) = (rand(i, *x, d, scale=6.0) for i, x in enumerate(((b, n, h), (b, n, hk), (1, p, hk))))
    (v, vf), (vp, vpf) = rand(3, b, n, hk, d), rand(4, 1, p, hk, d)
    o, lse = sa.prefix_attn_fwd(q, kp, vp, k, v, 60)
    status_ok()
    of, lf, ob = oc.prefix_attention(qf, kpf, vpf, kf, vf, 60)
    close(o, of, ob + LARGE_P * np.abs(np.concatenate((vf.ravel(), vpf.ravel()))).max(), "o")
    close(lse, lf, 4e-4, "lse")


@pytest.mark.parametrize("h,hk,d", [(4, 2, 32), (24, 2, 64), (4, 2, 128), (24, 2, 128)])
def test_decode_of_large_growing_scores(h, hk, d):
    """Scores that grow along the prefix and the caches, in several rounds of every ring; both decoding forms."""
    torch = torch_cuda()
    cap, p, lengths = 9000, 6000, [9000, 8191, 7001]
    b = len(lengths)
    q, qf = rand(0, b, 1, h, d)
    (v, vf), (vp, vpf) = rand(2, b, cap, hk, d), rand(4, 1, p, hk, d)
    gen = torch.Generator().manual_seed(1)
    k, kp = (torch.randn(x, y, hk, d, generator=gen) * torch.linspace(0.1, 4.0, y)[:, None, None] for x, y in ((b, cap), (1, p)))
    k, kp = k.to(torch.bfloat16).cuda(), kp.to(torch.bfloat16).cuda()
    kf, kpf = k.double().cpu().numpy(), kp.double().cpu().numpy()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, lse = sa.prefix_attn_decode(q, kp, vp, k, v, n, cap)
    status_ok()
    assert_close_attention(o, lse, oc.prefix_decode(qf, kpf, vpf, kf, vf, lengths, cap))
    cache = sa.ScoredCache(k, v, torch.zeros(b, hk, cap, device="cuda"), torch.zeros(b, hk, cap, dtype=torch.int32, device="cuda"))
    o, lse = sa.scored_attn_decode(q, cache, n)
    status_ok()
    of, lf, ob, w, wb = oc.scored_decode(qf, kf, vf, lengths, np.zeros((b, hk, cap)), 1.0)
    assert_close_attention(o, lse, (of, lf, ob))
    close(cache.weights, w, wb + 1e-30, "weights")


@pytest.mark.parametrize("d", [32, 64, 128])
def test_sink_weights_of_large_scores(d):
    n, w, s = 400, 90, 6
    (q, qf), (k, kf) = rand(0, 1, n, 2, d, scale=6.0), rand(1, 1, n, 1, d, scale=6.0)
    _, lse = sa.sink_attn_fwd(q, k, k, w, s)
    got = sa.sink_attn_weights(q, k, lse, w, s)
    status_ok()
    want, _ = oc.sink_weights(qf, kf, lse.double().cpu().numpy(), w, s, 0)
    close(got, want, LARGE_P * want + 1e-30, "weights")


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("value", [-200.0, -float("inf"), float("inf")])
def test_sink_weights_past_the_fp32_range(d, value):
    """LSE of some queries that is not the forward's: the keys that they see gather infinity (or nothing from them), however many
    queries follow, and the others what they do without."""
    torch = torch_cuda()
    n, h, w, s = 2600, 16, 2000, 3                         # several steps a CTA
    (q, qf), (k, kf) = rand(0, 1, n, h, d), rand(1, 1, n, 2, d)
    _, lse = sa.sink_attn_fwd(q, k, k, w, s)
    for e, i in ((0, 300), (1, 640), (1, 0), (11, 899), (15, 2599)):
        lse[0, e, i] = value
    got = sa.sink_attn_weights(q, k, lse, w, s).double().cpu().numpy()
    status_ok()
    want, bound = oc.sink_weights(qf, kf, lse.double().cpu().numpy(), w, s, 0)
    over = want > np.finfo(np.float32).max
    assert np.array_equal(np.isposinf(got), over) and over.any() == (value < 0) and not over.all()
    close(got[~over], want[~over], bound[~over], "weights")


@pytest.mark.parametrize("d", [32, 64, 128])
def test_sink_weights_of_scores_that_are_minus_infinity(d):
    """Queries without a finite score, whose LSE from the forward is -inf, add nothing."""
    n, w, s = 700, 300, 4
    (q, qf), (k, kf) = rand(0, 1, n, 2, d), rand(1, 1, n, 1, d)
    for t in (q, qf):
        t[..., 0] = 0.0
        t[:, :, 1] = 0.0
    q[:, 100:, 1, 0] = 3e38
    for t in (k, kf):
        t[..., 0] = -4.0
    _, lse = sa.sink_attn_fwd(q, k, k, w, s)
    got = sa.sink_attn_weights(q, k, lse, w, s)
    status_ok()
    finite = np.isfinite(lse.double().cpu().numpy())
    assert finite[0, 0].all() and finite[0, 1].sum() == 100
    want, bound = oc.sink_weights(qf, kf, np.where(finite, lse.double().cpu().numpy(), np.inf), w, s, 0)
    close(got, want, bound, "weights")


@pytest.mark.parametrize("value", [3.4e38, -3.4e38])
def test_sink_weights_of_the_largest_lse(value):
    """LSE next to the largest number, which rounds to infinity in bf16: its query gives nothing, or infinity."""
    torch = torch_cuda()
    n, w = 300, 299
    (q, qf), (k, kf) = rand(0, 1, n, 2, 64, scale=0.3), rand(1, 1, n, 1, 64, scale=0.3)
    _, lse = sa.sink_attn_fwd(q, k, k, w, 0, 1.0)
    lse[0, 1, 170] = value
    got = sa.sink_attn_weights(q, k, lse, w, 0, 0, 1.0).double().cpu().numpy()
    status_ok()
    with np.errstate(over="ignore"):
        want, bound = oc.sink_weights(qf, kf, lse.double().cpu().numpy(), w, 0, 0, 1.0)
    over = want > np.finfo(np.float32).max
    assert np.array_equal(np.isposinf(got), over) and over.sum() == (171 if value < 0 else 0)
    close(got[~over], want[~over], bound[~over], "weights")


def test_prefix_attention_strided_scaled_and_repeated():
    """Views of packed projections, one buffer of prefix keys and values, outputs with strides of their own."""
    torch = torch_cuda()
    b, n, p, h, hk, d, w = 3, 50, 700, 6, 2, 64, 20
    packed, pf = rand(0, b, n, h + 2 * hk, d)
    q, k, v = packed[:, :, :h], packed[:, :, h:h + hk], packed[:, :, h + hk:]
    both, bf = rand(1, 1, p, 2 * hk, d)
    kp, vp = both[:, :, :hk], both[:, :, hk:]
    o = torch.empty(b, n, 2, h, d, dtype=torch.bfloat16, device="cuda")[:, :, 1]
    lse = torch.empty(b, h, n, dtype=torch.float32, device="cuda")
    ws = torch.empty(sa.sa_prefix_attn_fwd_workspace_size(b, n, p, h, hk, d, w), dtype=torch.uint8, device="cuda")
    want = oc.prefix_attention(pf[:, :, :h], bf[:, :, :hk], bf[:, :, hk:], pf[:, :, h:h + hk], pf[:, :, h + hk:], w, scale=0.2)
    first = None
    for fill in (0, 0xff):
        ws.fill_(fill)
        sa.sa_prefix_attn_fwd(q, kp, vp, k, v, w, o, lse, ws, softmax_scale=0.2)
        status_ok()
        assert_close_attention(o, lse, want)
        first = (o.clone(), lse.clone()) if first is None else first
    assert torch.equal(first[0], o) and torch.equal(first[1], lse)
    # its last token, decoded over the same rows (the window is the same; a cache with a row to spare)
    ws = torch.empty(sa.sa_prefix_attn_decode_workspace_size(b, p, h, hk, d), dtype=torch.uint8, device="cuda")
    wide = torch.cat((packed, packed[:, :1]), 1)
    lengths = torch.full((b,), n, dtype=torch.int32, device="cuda")
    o1, lse1 = torch.empty(b, 1, h, d, dtype=torch.bfloat16, device="cuda"), torch.empty(b, h, 1, device="cuda")
    for fill in (0, 0xff):
        ws.fill_(fill)
        sa.sa_prefix_attn_decode(wide[:, n - 1:n, :h], kp, vp, wide[:, :, h:h + hk], wide[:, :, h + hk:], lengths, w, o1, lse1,
                                 ws, softmax_scale=0.2)
        status_ok()
        assert_close_attention(o1, lse1, (want[0][:, -1:], want[1][:, :, -1:], want[2][:, -1:]))


def test_prefix_batch_stride_is_not_used():
    """A prefix cut from a larger tensor, whose batch stride is not that of its rows."""
    torch = torch_cuda()
    (q, qf), (k, kf), (v, vf), (kv, kvf) = rand(0, 2, 5, 4, 64), rand(1, 2, 5, 2, 64), rand(2, 2, 5, 2, 64), rand(3, 3, 400, 2, 64)
    o, lse = sa.prefix_attn_fwd(q, kv[1:2, :129], kv[2:3, 7:136], k, v, 4)
    status_ok()
    assert_close_attention(o, lse, oc.prefix_attention(qf, kvf[1:2, :129], kvf[2:3, 7:136], kf, vf, 4))


@pytest.mark.parametrize("d", [32, 64, 128])
def test_prefix_attention_with_several_items_a_cta(d):
    """Persistent CTAs that take three work items and more, both plans, every row checked."""
    for b, n, p, h, hk, w in ((16, 120, 300, 35, 7, 50), (60, 6, 40, 24, 8, 3), (24, 150, 200, 20, 20, 9)):
        several_per_sm(b * hk * -(-n * (h // hk) // 128))
        (q, qf), (k, kf), (v, vf) = (rand(i, b, n, x, d) for i, x in enumerate((h, hk, hk)))
        (kp, kpf), (vp, vpf) = (rand(i, 1, p, hk, d) for i in (3, 4))
        o, lse = sa.prefix_attn_fwd(q, kp, vp, k, v, w)
        status_ok()
        assert_close_attention(o, lse, oc.prefix_attention(qf, kpf, vpf, kf, vf, w))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("h", [4, 24])
def test_nan_of_what_is_seen(h, d):
    """A NaN in a query, in a prefix key and in one own key: o and lse are NaN for the heads that see it, the
    weights of their key head too, and everything else is as without it."""
    torch = torch_cuda()
    b, hk, cap, p = 4, 2, 300, 500
    lengths = [1, 300, 300, 0]
    q, k, v = (rand(i, b, x, y, d)[0] for i, (x, y) in enumerate(((1, h), (cap, hk), (cap, hk))))
    kp, vp = (rand(i, 1, p, hk, d)[0] for i in (3, 4))
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    group = h // hk

    def both():
        cache = sa.ScoredCache(k, v, torch.zeros(b, hk, cap, device="cuda"), torch.zeros(b, hk, cap, dtype=torch.int32, device="cuda"))
        out = sa.prefix_attn_decode(q, kp, vp, k, v, n, cap), sa.scored_attn_decode(q, cache, n), cache.weights
        status_ok()
        return out

    clean = both()
    k[0, 0, 0, 5] = float("nan")                          # the only own key of key head 0
    k[1, 271, 1, d - 1] = float("nan")                    # one of 300 of key head 1
    q[2, 0, 1, 3] = float("nan")
    hit = torch.zeros(b, h, dtype=torch.bool, device="cuda")
    hit[0, :group] = hit[1, group:] = hit[2, 1] = True
    got = both()
    for (o, lse), (o1, lse1) in zip(got[:2], clean[:2]):
        assert torch.isnan(o[:, 0][hit]).all() and torch.isnan(lse[..., 0][hit]).all()
        assert torch.equal(o[:, 0][~hit], o1[:, 0][~hit]) and torch.equal(lse[..., 0][~hit], lse1[..., 0][~hit])
    assert torch.isneginf(got[1][1][3]).all() and not got[1][0][3].any()
    rows = torch.arange(cap, device="cuda") < n[:, None, None]
    heads = torch.tensor([[1, 0], [0, 1], [1, 0], [0, 0]], dtype=torch.bool, device="cuda")[:, :, None] & rows
    assert torch.isnan(got[2][heads]).all() and torch.equal(got[2][~heads], clean[2][~heads])
    # in the prefix: every query of key head 1
    kp[0, 130, 1, 0] = float("nan")
    (o, lse), (o1, lse1) = both()[0], got[0]
    assert torch.isnan(o[:, 0, group:]).all() and torch.isnan(lse[:, group:]).all()
    assert torch.equal(o[1, 0, :group], o1[1, 0, :group]) and torch.equal(lse[1, :group], lse1[1, :group])


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("h", [3, 20])
def test_scores_that_are_all_minus_infinity_add_no_weight(h, d):
    """Head 1's scores pass the fp32 range downwards, on every row or on some: rows without a finite score are as no rows (o 0, lse
    -inf), and add nothing to the weights that the other heads give."""
    torch = torch_cuda()
    b, cap, lengths = 4, 600, [1, 600, 70, 600]
    q, qf = rand(0, b, 1, h, d)
    (k, kf), (v, vf) = rand(1, b, cap, 1, d), rand(2, b, cap, 1, d)
    for t in (q, qf):
        t[..., 0] = 0.0
        t[:, :, 1] = 0.0
    q[:, :, 1, 0] = 3e38
    for t in (k, kf):
        t[..., 0] = -4.0
        t[3, ::7, :, 0] = 0.0                              # the last sequence has rows that head 1 sees, alike
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    old = torch.rand(b, 1, cap, device="cuda")
    cache = sa.ScoredCache(k, v, old.clone(), torch.zeros(b, 1, cap, dtype=torch.int32, device="cuda"))
    o, lse = sa.scored_attn_decode(q, cache, n, 0.5)
    status_ok()
    others = [e for e in range(h) if e != 1]
    of, lf, ob, want, bound = oc.scored_decode(qf[:, :, others], kf, vf, lengths, old.double().cpu().numpy(), 0.5)
    assert_close_attention(o[:, :, others], lse[:, others], (of, lf, ob))
    assert not o[:3, 0, 1].any() and torch.isneginf(lse[:3, 1]).all()
    rows = np.arange(0, cap, 7)
    want[3, 0, rows] += 1 / len(rows)
    bound[3, 0, rows] += oc.P_REL / len(rows)
    close(cache.weights, want, bound + 1e-30, "weights")
    mean = vf[3, rows, 0].mean(0)
    close(o[3, 0, 1], mean, 1.02 * ref.U * (np.abs(mean) + np.abs(vf[3, rows, 0]).mean(0)) + 1e-6, "o")
    assert abs(float(lse[3, 1]) - np.log(len(rows))) <= LSE_TOL


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("some", [False, True])
def test_prefix_scores_that_are_minus_infinity(d, some):
    """Head 1's scores pass the fp32 range downwards, on every key or on all but a few (whole tiles have no finite score): those few
    are seen alike, and without one o is 0 and lse -inf. Prompts and single tokens, few rows and many."""
    torch = torch_cuda()
    for b, n, p, h in ((2, 150, 1500, 2), (3, 5, 700, 4)):
        (q, qf), (k, kf), (v, vf) = (rand(i, b, n, x, d) for i, x in enumerate((h, 1, 1)))
        (kp, kpf), (vp, vpf) = (rand(i, 1, p, 1, d) for i in (3, 4))
        for t in (q, qf):
            t[..., 0] = 0.0
            t[:, :, 1] = 0.0
        q[:, :, 1, 0] = 3e38
        for t in (k, kf, kp, kpf):
            t[..., 0] = -4.0
        if some:
            for t in (kp, kpf):
                t[:, 130::400, :, 0] = 0.0
        others, w = [e for e in range(h) if e != 1], 100
        lengths = torch.full((b,), n, dtype=torch.int32, device="cuda")
        seen = vpf[0, 130::400, 0]
        mean, size = (seen.mean(0), np.abs(seen).mean(0)) if some else (0.0, 0.0)
        want = oc.prefix_attention(qf[:, :, others], kpf, vpf, kf, vf, w)
        for rows, (o, lse) in ((slice(0, n), sa.prefix_attn_fwd(q, kp, vp, k, v, w)),
                               (slice(n - 1, n), sa.prefix_attn_decode(q[:, -1:], kp, vp, k, v, lengths, w))):
            status_ok()
            assert_close_attention(o[:, :, others], lse[:, others], (want[0][:, rows], want[1][:, :, rows], want[2][:, rows]))
            mine = o[:, :, 1].double().cpu().numpy()
            close(mine, np.broadcast_to(mean, mine.shape), 1.02 * ref.U * (np.abs(mean) + size) + 1e-6, "o")
            assert ((lse[:, 1] - np.log(len(seen))).abs() <= LSE_TOL if some else torch.isneginf(lse[:, 1])).all()


@pytest.mark.parametrize("d", [32, 64, 128])
def test_sink_window_scores_that_are_minus_infinity(d):
    """The same of the sink-window forward: head 1 has a finite score on the first token (a sink) and on every 400th alone."""
    n, w, s = 1500, 300, 1
    (q, qf), (k, kf), (v, vf) = (rand(i, 1, n, x, d) for i, x in enumerate((2, 1, 1)))
    for t in (q, qf):
        t[..., 0] = 0.0
        t[:, :, 1] = 0.0
    q[:, :, 1, 0] = 3e38
    for t in (k, kf):
        t[..., 0] = -4.0
        t[:, ::400, :, 0] = 0.0
    for sinks in (s, 0):
        o, lse = sa.sink_attn_fwd(q, k, v, w, sinks)
        status_ok()
        want = ref.sink_attention(qf[:, :, :1], kf, vf, w, sinks)
        assert_close_attention(o[:, :, :1], lse[:, :1], want)
        mask = ref.sink_mask(n, w, sinks) & (np.arange(n) % 400 == 0)
        count = mask.sum(1)
        p = mask / np.maximum(count, 1)[:, None]
        mean, size = p @ vf[0, :, 0], p @ np.abs(vf[0, :, 0])
        close(o[0, :, 1], mean, 1.02 * ref.U * (np.abs(mean) + size) + 1e-6, "o")
        assert (count == 0).any() == (sinks == 0)
        got = lse[0, 1].double().cpu().numpy()
        assert np.array_equal(np.isneginf(got), count == 0) and np.abs(got[count > 0] - np.log(count[count > 0])).max() <= LSE_TOL


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("n,w,s", [(600, 599, 0), (300, 70, 2), (40, 3, 0)])
def test_sink_window_gradients_of_scores_that_are_minus_infinity(d, n, w, s):
    """A head without a finite score has no gradient, and the others' are as without it."""
    (q, qf), (k, kf), (v, vf), (g, gf) = (rand(i, 1, n, x, d) for i, x in enumerate((2, 1, 1, 2)))
    for t in (q, qf):
        t[..., 0] = 0.0
        t[:, :, 1] = 0.0
    q[:, :, 1, 0] = 3e38
    for t in (k, kf):
        t[..., 0] = -4.0
    o, lse = sa.sink_attn_fwd(q, k, v, w, s)
    dq, dk, dv = sa.sink_attn_bwd(q, k, v, o, lse, g, w, s)
    status_ok()
    (dqf, dkf, dvf), (bq, bk, bv) = ref.sink_attention_backward(qf[:, :, :1], kf, vf, gf[:, :, :1], w, s)
    assert not dq[:, :, 1].any()
    for x, y, bound in ((dq[:, :, :1], dqf, bq), (dk, dkf, bk), (dv, dvf, bv)):
        close(x, y, bound, "gradient")


@pytest.mark.parametrize("d", [32, 128])
def test_prefix_attention_keeps_nan_queries(d):
    torch = torch_cuda()
    q, k, v = (rand(i, 2, 40, x, d)[0] for i, x in enumerate((4, 2, 2)))
    kp, vp = (rand(i, 1, 300, 2, d)[0] for i in (3, 4))
    clean = sa.prefix_attn_fwd(q, kp, vp, k, v, 39)
    q[1, 7, 2, 1] = float("nan")
    o, lse = sa.prefix_attn_fwd(q, kp, vp, k, v, 39)
    status_ok()
    hit = torch.zeros(2, 40, 4, dtype=torch.bool, device="cuda")
    hit[1, 7, 2] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse.transpose(1, 2)[hit]).all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse.transpose(1, 2)[~hit], clean[1].transpose(1, 2)[~hit])


@pytest.mark.parametrize("scale", [1e-44, 1e-20, None])
@pytest.mark.parametrize("h,hk,d", [(4, 2, 32), (24, 2, 64), (4, 2, 128)])
def test_zero_queries_see_every_key_alike(h, hk, d, scale):
    torch = torch_cuda()
    b, cap, p, lengths = 3, 72, 200, [1, 13, 71]
    q, qf = rand(0, b, 1, h, d)
    q[:, :, 1] = 0.0
    qf[:, :, 1] = 0.0
    (k, kf), (v, vf) = (rand(i, b, cap, hk, d) for i in (1, 2))
    (kp, kpf), (vp, vpf) = (rand(i, 1, p, hk, d) for i in (3, 4))
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = sa.prefix_attn_decode(q, kp, vp, k, v, n, 100, scale)
    status_ok()
    assert_close_attention(*got, oc.prefix_decode(qf, kpf, vpf, kf, vf, lengths, 100, scale))
    cache = sa.ScoredCache(k, v, torch.zeros(b, hk, cap, device="cuda"), torch.zeros(b, hk, cap, dtype=torch.int32, device="cuda"))
    got = sa.scored_attn_decode(q, cache, n, 1.0, None, scale)
    status_ok()
    of, lf, ob, w, wb = oc.scored_decode(qf, kf, vf, lengths, np.zeros((b, hk, cap)), 1.0, scale)
    assert_close_attention(*got, (of, lf, ob))
    close(cache.weights, w, wb + 1e-30, "weights")


def test_lengths_outside_the_caches_are_cut():
    torch = torch_cuda()
    b, cap, hk, h, d = 3, 40, 2, 4, 64
    q, qf = rand(0, b, 1, h, d)
    (k, kf), (v, vf) = (rand(i, b, cap, hk, d) for i in (1, 2))
    (kp, kpf), (vp, vpf) = (rand(i, 1, 77, hk, d) for i in (3, 4))
    n = torch.tensor([-5, 1000, 40], dtype=torch.int32, device="cuda")
    got = sa.prefix_attn_decode(q, kp, vp, k, v, n, 20)
    status_ok()
    assert_close_attention(*got, oc.prefix_decode(qf, kpf, vpf, kf, vf, [0, 40, 40], 20))
    cache = sa.ScoredCache(k, v, torch.ones(b, hk, cap, device="cuda"), torch.zeros(b, hk, cap, dtype=torch.int32, device="cuda"))
    got = sa.scored_attn_decode(q, cache, n, 0.5)
    status_ok()
    of, lf, ob, w, wb = oc.scored_decode(qf, kf, vf, [0, 40, 40], np.ones((b, hk, cap)), 0.5)
    assert_close_attention(*got, (of, lf, ob))
    close(cache.weights, w, wb + 1e-30, "weights")
    k, v, w, pos = evict_inputs(b, cap, hk, d)
    check = oc.evict(bits(k).cpu().numpy(), bits(v).cpu().numpy(), w.cpu().numpy(), pos.cpu().numpy(), [-5, 1000, 40], 30, 2, 5)
    cache = sa.ScoredCache(k, v, w, pos)
    sa.scored_evict(cache, n, 30, 2, 5)
    status_ok()
    assert n.tolist() == check[4] == [0, 30, 30]
    assert all(np.array_equal(bits(x).cpu().numpy().view(y.dtype), y) for x, y in zip(cache, check))


# ------------------------------------------------------------------ sizes past 32 bits

def test_scored_cache_of_more_than_2_31_elements():
    """The last sequence's rows lie past 2^32 elements; its attention, weights and eviction against the oracle."""
    torch = torch_cuda()
    b, hk, h, d, cap, n = 9, 4, 8, 128, 1 << 20, 300
    k, v = (torch.empty(b, cap, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 1 << 32
    w, pos = torch.zeros(b, hk, cap, device="cuda"), torch.zeros(b, hk, cap, dtype=torch.int32, device="cuda")
    cache = sa.ScoredCache(k, v, w, pos)
    (rk, kf), (rv, vf), (q, qf) = rand(1, b, n, hk, d), rand(2, b, n, hk, d), rand(0, b, 1, h, d)
    start = torch.full((b,), -1, dtype=torch.int32, device="cuda")
    start[-1] = 0
    sa.scored_append(cache, rk, rv, start)
    lengths = torch.zeros(b, dtype=torch.int32, device="cuda")
    lengths[-1] = n
    o, lse = sa.scored_attn_decode(q, cache, lengths)
    status_ok()
    of, lf, ob, wf, wb = oc.scored_decode(qf[-1:], kf[-1:], vf[-1:], [n], np.zeros((1, hk, n)), 1.0)
    assert_close_attention(o[-1:], lse[-1:], (of, lf, ob))
    close(w[-1:, :, :n], wf, wb + 1e-30, "weights")
    want = oc.evict(bits(rk[-1:]).cpu().numpy(), bits(rv[-1:]).cpu().numpy(), w[-1:, :, :n].cpu().numpy(),
                    pos[-1:, :, :n].cpu().numpy(), [n], 200, 4, 50)
    sa.scored_evict(cache, lengths, 200, 4, 50)
    status_ok()
    assert np.array_equal(bits(k[-1:, :n]).cpu().numpy(), want[0]) and np.array_equal(bits(v[-1:, :n]).cpu().numpy(), want[1])
    assert np.array_equal(pos[-1:, :, :n].cpu().numpy(), want[3]) and lengths.tolist() == [0] * (b - 1) + [200]
    # a long list: every slot of one sequence in use
    lengths.zero_()
    lengths[0] = cap
    w[0] = torch.rand(hk, cap, device="cuda")
    pos[0] = torch.arange(cap, dtype=torch.int32, device="cuda")
    keep = cap - 5
    low = w[0, :, 4:cap - 9].sort(dim=-1, stable=True).indices[:, :5] + 4
    k[0, :, :, 0] = (torch.arange(cap, device="cuda") % 251).to(torch.bfloat16)[:, None]
    sa.scored_evict(cache, lengths, keep, 4, 9)
    status_ok()
    for e in range(hk):
        gone = sorted(x for x in low[e].tolist() if x < keep)
        moved = [x for x in range(keep, cap)]
        moved = [x for x in moved if x not in low[e].tolist()]
        assert pos[0, e, gone].tolist() == moved
        assert k[0, gone, e, 0].tolist() == [float(x % 251) for x in moved]
    assert int(lengths[0]) == keep


def test_prefix_of_more_than_2_31_elements():
    torch = torch_cuda()
    p, hk, h, d, b = (1 << 24) + 77, 2, 4, 128, 2
    kp, vp = (torch.zeros(1, p, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kp.numel() > 1 << 32
    ends = [rand(i, 1, 64, hk, d)[0] for i in (3, 4)]
    kp[:, -64:], vp[:, -64:] = ends[0] * 6, ends[1]
    q, k, v = (rand(i, b, 1, x, d)[0] for i, x in enumerate((h, hk, hk)))
    n = torch.ones(b, dtype=torch.int32, device="cuda")
    got = sa.prefix_attn_decode(q, kp, vp, k, v, n, 0), sa.prefix_attn_fwd(q, kp, vp, k, v, 0)
    status_ok()
    for s in range(b):
        for e in range(h):
            x = q[s, 0, e].double() * d ** -0.5
            near = torch.cat((kp[0, -64:, e // 2], k[s, :, e // 2])).double() @ x
            values = torch.cat((vp[0, -64:, e // 2], v[s, :, e // 2])).double()
            top = max(float(near.max()), 0.0)
            weight = (near - top).exp()
            total = float(weight.sum()) + (p - 64) * np.exp(-top)
            want, size = weight @ values / total, weight @ values.abs() / total
            for o, lse in got:
                # fp32 sums of 2^24 equal terms in some 10^5 parts: below 2^-12 of the total
                assert ((o[s, 0, e].double() - want).abs() <= 1.02 * ref.U * (want.abs() + size) + 2.0**-12 * size + 1e-6).all()
                assert abs(float(lse.view(b, h)[s, e]) - top - np.log(total)) <= LSE_TOL + 2.0**-12


# ------------------------------------------------------------------ around the outputs, graphs, streams, first calls

@pytest.mark.parametrize("n,d", [(1, 128), (133, 64), (30, 32)])
def test_nothing_is_written_around_the_outputs(n, d):
    torch = torch_cuda()
    b, h, hk, w, s, p = 2, 4, 2, 70, 9, 150
    f32, u8, i32 = torch.float32, torch.uint8, torch.int32
    q, k, v, g, gk = (rand(i, b, n, x, d)[0] for i, x in enumerate((h, hk, hk, h, hk)))
    kp, vp = (rand(i, 1, p, hk, d)[0] for i in (5, 6))
    guard = Guard()

    def rows(*shape):
        return guard(*shape, every_other_head=True)

    weight, freq = torch.ones(d, device="cuda"), 100.0 ** -np.arange(d // 2)
    pair, pos = [x % 2 for x in range(d // 2)], torch.ones(b, n, 2, dtype=i32, device="cuda")
    sa.sa_qk_norm_rope_axes_fwd(q, k, weight, weight, freq, pair, pos, rows(b, n, h, d), rows(b, n, hk, d))
    ws = guard(sa.sa_qk_norm_rope_bwd_workspace_size(d), dtype=u8)
    sa.sa_qk_norm_rope_axes_bwd(q, k, g, gk, weight, weight, freq, pair, pos, rows(b, n, h, d), rows(b, n, hk, d),
                                guard(d, dtype=f32), guard(d, dtype=f32), ws)
    ws = guard(sa.sa_prefix_attn_fwd_workspace_size(b, n, p, h, hk, d, w), dtype=u8)
    sa.sa_prefix_attn_fwd(q, kp, vp, k, v, w, rows(b, n, h, d), guard(b, h, n, dtype=f32), ws)
    lengths = torch.tensor([n, max(0, n - 3)], dtype=i32, device="cuda")
    ws = guard(sa.sa_prefix_attn_decode_workspace_size(b, p, h, hk, d), dtype=u8)
    sa.sa_prefix_attn_decode(q[:, :1], kp, vp, k, v, lengths, w, rows(b, 1, h, d), guard(b, h, 1, dtype=f32), ws)
    _, lse = sa.sink_attn_fwd(q, k, v, w, s)
    ws = guard(sa.sa_sink_attn_weights_workspace_size(), dtype=u8)
    sa.sa_sink_attn_weights(q, k, lse, w, s, guard(b, hk, n, dtype=f32), ws, first_query=n // 2)
    cache = sa.ScoredCache(rows(b, n + 2, hk, d), rows(b, n + 2, hk, d), guard(b, hk, n + 2, dtype=f32), guard(b, hk, n + 2, dtype=i32))
    sa.scored_append(cache, k, v, torch.tensor([0, 2], dtype=i32, device="cuda"))
    ws = guard(sa.sa_scored_attn_decode_workspace_size(b, n + 2, h, hk), dtype=u8)
    sa.sa_scored_attn_decode(q[:, :1], cache, lengths, rows(b, 1, h, d), guard(b, h, 1, dtype=f32), ws, 0.5,
                             guard(b, hk, n + 2, dtype=f32))
    sa.sa_scored_evict(cache, lengths, max(1, n // 2), 0, n // 4, guard(b, hk, n + 2, dtype=f32), guard(b, hk, n + 2, dtype=i32),
                       guard(b, dtype=i32))
    sa.scored_evict(cache, lengths, max(1, n // 2), 0, n // 4)
    status_ok()
    guard.check()


def chain_inputs(seed, b, n, p, h, hk, d):
    packed = rand(seed, b, n, h + 2 * hk, d)[0]
    return packed, rand(seed + 1, 1, p, 2 * hk, d)[0]


def test_captured_and_replayed_on_new_inputs():
    """One CUDA graph of every call, replayed after its inputs changed; its caches start anew in every replay."""
    torch = torch_cuda()
    b, n, p, h, hk, d, w = 2, 140, 300, 4, 2, 64, 60
    packed, both = chain_inputs(2, b, n, p, h, hk, d)
    wt = torch.ones(d, device="cuda")
    freq, pair = 100.0 ** (-np.arange(d // 2) / 32.0), [x % 3 for x in range(d // 2)]
    pos = torch.randint(0, 5000, (b, n, 3), dtype=torch.int32, device="cuda")
    full = torch.tensor([n, 131], dtype=torch.int32, device="cuda")
    cache = sa.scored_alloc(b, n + 4, hk, d)

    def chain():
        q, k, v = packed[:, :, :h], packed[:, :, h:h + hk], packed[:, :, h + hk:]
        q, k = sa.qk_norm_rope_axes_fwd(q, k, wt, wt, freq, pair, pos)
        back = sa.qk_norm_rope_axes_bwd(packed[:, :, :h], packed[:, :, h:h + hk], q, k, wt, wt, freq, pair, pos)
        _, lse = sa.sink_attn_fwd(q, k, v, w, 4)
        weights = sa.sink_attn_weights(q, k, lse, w, 4, 70)
        lengths = full.clone()
        for x in cache:
            x.zero_()
        sa.scored_append(cache, k, v)
        cache.weights[:, :, :n] = weights
        sa.scored_evict(cache, lengths, 100, 4, 20)
        last = q[:, -1:].contiguous()
        out = sa.scored_attn_decode(last, cache, lengths, 0.9)
        out += sa.prefix_attn_fwd(q, both[:, :, :hk], both[:, :, hk:], k, v, w)
        out += sa.prefix_attn_decode(last, both[:, :, :hk], both[:, :, hk:], cache.k, cache.v, lengths, n)
        return out + back + (weights, lengths) + tuple(x.clone() for x in cache)

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain()
    for seed in (21, 31):
        x, y = chain_inputs(seed, b, n, p, h, hk, d)
        packed.copy_(x)
        both.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        for x, y in zip(got, chain()):
            assert torch.equal(x, y)
    status_ok()


def test_two_streams_at_once():
    torch = torch_cuda()
    b, n, p, h, hk, d, cap = 4, 33, 3000, 8, 2, 128, 900
    lengths = torch.tensor([900, 500, 1, 0], dtype=torch.int32, device="cuda")
    sets = [(*chain_inputs(10 * i, b, n, p, h, hk, d), rand(10 * i + 5, b, cap, 2 * hk, d)[0]) for i in range(2)]

    def calls(packed, both, kv):
        q, k, v = packed[:, :, :h], packed[:, :, h:h + hk], packed[:, :, h + hk:]
        kp, vp = both[:, :, :hk], both[:, :, hk:]
        cache = sa.ScoredCache(kv[:, :, :hk].clone(), kv[:, :, hk:].clone(), torch.zeros(b, hk, cap, device="cuda"),
                               torch.arange(cap, dtype=torch.int32, device="cuda").expand(b, hk, cap).contiguous())
        m = lengths.clone()
        out = sa.prefix_attn_fwd(q, kp, vp, k, v, n) + sa.prefix_attn_decode(q[:, -1:], kp, vp, cache.k, cache.v, m, cap)
        out += sa.scored_attn_decode(q[:, -1:], cache, m) + sa.scored_evict(cache, m, 300, 2, 50)
        _, lse = sa.sink_attn_fwd(q, k, v, n, 0)
        return out + (sa.sink_attn_weights(q, k, lse, n, 0), cache.k, cache.v)

    want = [calls(*x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = calls(*sets[i])
    torch.cuda.synchronize()
    status_ok()
    for a, c in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, c))


FRESH = '''
import threading
import numpy as np, torch
import content_adaptive_sparse_gb300 as sa

b, n, p, h, hk, d, threads, calls = 2, 60, 300, 4, 2, 64, 8, 12
gen = torch.Generator(device="cuda").manual_seed(1)
q, k, v, kp, vp = (torch.randn(*x, d, generator=gen, device="cuda").bfloat16() for x in ((b, n, h), (b, n, hk), (b, n, hk), (1, p, hk), (1, p, hk)))
length = torch.tensor([n, 7], dtype=torch.int32, device="cuda")
pos = torch.randint(0, 900, (b, n, 2), dtype=torch.int32, device="cuda", generator=gen)

def chain(i):
    freq = (100.0 + i) ** (-np.arange(d // 2) / 32.0)
    qr, kr = sa.qk_norm_rope_axes_fwd(q, k, None, None, freq, [(x + i) % 2 for x in range(d // 2)], pos)
    cache = sa.scored_alloc(b, n, hk, d)
    sa.scored_append(cache, kr, v)
    _, lse = sa.sink_attn_fwd(qr, kr, v, n, 0)
    out = (qr, kr, sa.sink_attn_weights(qr, kr, lse, n, 0)) + sa.prefix_attn_fwd(qr, kp, vp, kr, v, n)
    out += sa.prefix_attn_decode(qr[:, -1:], kp, vp, cache.k, cache.v, length, n) + sa.scored_attn_decode(qr[:, -1:], cache, length)
    m = length.clone()
    return out + sa.scored_evict(cache, m, 20, 1, 4) + (cache.k[:, :7], cache.v[:, :7])
'''

THREADS = FRESH + '''
torch.cuda.synchronize()
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

CAPTURED = FRESH + '''
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = chain(0)
graph.replay(); torch.cuda.synchronize()
got = [x.clone() for x in outs]
assert all(torch.equal(x, y) for x, y in zip(got, chain(0)))
torch.cuda.synchronize(); assert sa.sa_device_status() == 0
'''


def test_first_calls_from_several_host_threads():
    in_a_fresh_process(THREADS)


def test_first_calls_inside_a_capture():
    in_a_fresh_process(CAPTURED)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("d", [64, 128])
def test_questions_about_a_video(d):
    """A video's patches (three axes) as the shared prefix, a question per sequence as a prompt behind it, then one token at a
    time: every output is that of one pass over prefix and own tokens."""
    torch = torch_cuda()
    b, p, n, more, h, hk = 5, 5 * 16, 9, 4, 6, 2
    freq, pair = 100.0 ** (-np.arange(d // 2) * 2.0 / d), [x % 3 for x in range(d // 2)]
    rng = np.random.default_rng(0)
    w = [np.float32(1 + 0.1 * rng.standard_normal(d)) for _ in range(2)]
    wt = [torch.from_numpy(x).cuda() for x in w]
    grid = torch.stack([torch.arange(p) // 16, torch.arange(p) % 16 // 4, torch.arange(p) % 4], -1).int()[None].cuda()
    video, _ = rand(1, 1, p, h + 2 * hk, d)
    text, _ = rand(2, b, n + more, h + 2 * hk, d)
    tpos = (5 + torch.arange(n + more, dtype=torch.int32, device="cuda"))[None, :, None].expand(b, -1, 3).contiguous()
    _, kp = sa.qk_norm_rope_axes_fwd(video[:, :, :h], video[:, :, h:h + hk], *wt, freq, pair, grid)
    vp = video[:, :, h + hk:].contiguous()
    q, k = sa.qk_norm_rope_axes_fwd(text[:, :, :h], text[:, :, h:h + hk], *wt, freq, pair, tpos)
    v = text[:, :, h + hk:]
    want = oc.prefix_attention(*(x.double().cpu().numpy() for x in (q, kp, vp, k, v)), n + more)
    o, lse = sa.prefix_attn_fwd(q[:, :n], kp, vp, k[:, :n], v[:, :n], n)
    status_ok()
    assert_close_attention(o, lse, (want[0][:, :n], want[1][:, :, :n], want[2][:, :n]))
    cache = [torch.full((b, n + more, hk, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache[0][:, :n], cache[1][:, :n] = k[:, :n], v[:, :n]
    lengths = torch.full((b,), n, dtype=torch.int32, device="cuda")
    for i in range(n, n + more):
        qi, ki = sa.qk_norm_rope_axes_fwd(text[:, i:i + 1, :h], text[:, i:i + 1, h:h + hk], *wt, freq, pair, tpos[:, i:i + 1].contiguous())
        cache[0][:, i:i + 1], cache[1][:, i:i + 1] = ki, v[:, i:i + 1]
        lengths += 1
        o, lse = sa.prefix_attn_decode(qi, kp, vp, *cache, lengths, n + more)
        status_ok()
        assert_close_attention(o, lse, (want[0][:, i:i + 1], want[1][:, :, i:i + 1], want[2][:, i:i + 1]), f"token {i} ")


@pytest.mark.parametrize("d", [32, 128])
def test_a_prompt_and_many_tokens_in_a_bounded_cache(d):
    """The prompt's weights, an eviction, then steps that append, attend, add weights and evict: attention and weights of every
    step against float64 over what the cache holds, every eviction against the oracle on the same weights, and
    the plain decoding call over the same rows."""
    torch = torch_cuda()
    b, n, h, hk, keep, steps, sinks, recent = 2, 150, 8, 2, 64, 12, 4, 16
    cap = n + 8
    (q, qf), (k, kf), (v, vf) = (rand(i, b, n + steps, x, d) for i, x in enumerate((h, hk, hk)))
    _, lse = sa.sink_attn_fwd(q[:, :n], k[:, :n], v[:, :n], n, 0)
    cache = sa.scored_alloc(b, cap, hk, d)
    sa.scored_append(cache, k[:, :n], v[:, :n])
    first = n - 32
    weights = sa.sink_attn_weights(q[:, :n], k[:, :n], lse, n, 0, first)
    status_ok()
    want, bound = oc.sink_weights(qf[:, :n], kf[:, :n], lse.double().cpu().numpy(), n, 0, first)
    close(weights, want, bound, "prompt weights")
    # every query's probabilities sum to one
    assert abs(float(weights.sum()) - b * h * 32) <= 1e-3 * b * h * 32
    cache.weights[:, :, :n] = weights
    lengths = torch.tensor([n, n - 20], dtype=torch.int32, device="cuda")
    for i in range(steps):
        before = [x.cpu().numpy() if x.dtype != torch.bfloat16 else bits(x).cpu().numpy() for x in cache]
        m = lengths.tolist()
        sa.scored_evict(cache, lengths, keep, sinks, recent)
        status_ok()
        after = oc.evict(*before, m, keep, sinks, recent)
        for x, y in zip(cache, after):
            assert np.array_equal(bits(x).cpu().numpy(), y.view(bits(x).cpu().numpy().dtype))
        assert lengths.tolist() == after[4]
        sa.scored_append(cache, k[:, n + i:n + i + 1], v[:, n + i:n + i + 1], lengths, torch.full_like(lengths, n + i))
        lengths += 1
        m = lengths.tolist()
        held = [x.double().cpu().numpy() for x in cache[:3]]
        qi, qif = q[:, n + i:n + i + 1].contiguous(), qf[:, n + i:n + i + 1]
        o, lse = sa.scored_attn_decode(qi, cache, lengths, 0.95)
        status_ok()
        of, lf, ob, wf, wb = oc.scored_decode(qif, held[0], held[1], m, held[2], 0.95)
        used = np.arange(cap) < np.array(m)[:, None, None]
        assert_close_attention(o, lse, (of, lf, ob), f"step {i} ")
        close(np.where(used, cache.weights.double().cpu().numpy(), wf), wf, wb, f"weights {i}")
        o2, lse2 = sa.sink_attn_decode(qi, cache.k, cache.v, lengths, cap, 0)
        assert_close_attention(o2, lse2, (of, lf, ob), f"plain {i} ")
