"""Shared contexts and bounded caches on the GPU against float64 (oracle/streaming.py, oracle/context.py):
norm and rotation with several axes, attention behind a shared prefix, the cache of slots with
accumulated weights, and runs of them together. Tolerances are the oracles' elementwise bounds."""
import numpy as np
import pytest

import content_adaptive_sparse_gb300 as sa
from gpu_helpers import torch_cuda
from oracle import streaming as ref
from test_gpu_streaming import Guard, close, in_a_fresh_process, rand, status_ok

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
