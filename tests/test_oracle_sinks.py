"""Pins of the oracle's local window with sinks (oracle/attention.py, oracle/tiles.py)."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import tiles as ot


@pytest.mark.parametrize("w,s", [(0, 0), (0, 2), (3, 1), (5, 4), (2, 40), (40, 3)])
def test_window_with_sinks_matches_autograd(w, s):
    """The oracle's sinks against a dense mask written out here and torch's float64 autograd."""
    cu = [0, 7, 8, 30]
    T, Hq, Hkv, d = 30, 4, 2, 8
    g = torch.Generator().manual_seed(100 * w + s)
    q, do = (torch.randn(T, Hq, d, generator=g, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(T, Hkv, d, generator=g, dtype=torch.float64) for _ in range(2))
    see = torch.zeros(T, T, dtype=torch.bool)
    for b, e in zip(cu, cu[1:]):
        for i in range(b, e):
            for j in range(b, i + 1):
                see[i, j] = i - j <= w or j - b < s
    x = [t.clone().requires_grad_(True) for t in (q, k, v)]
    sc = torch.einsum("ihd,jhd->hij", x[0], x[1].repeat_interleave(2, 1)) / math.sqrt(d)
    p = torch.softmax(sc.masked_fill(~see, -math.inf), -1)
    out = torch.einsum("hij,jhd->ihd", p, x[2].repeat_interleave(2, 1))
    out.backward(do)
    o, lse = oa.varlen_forward(q.numpy(), k.numpy(), v.numpy(), cu, window=w, sinks=s)
    gr = oa.varlen_backward(q.numpy(), k.numpy(), v.numpy(), o, lse, do.numpy(), cu, window=w, sinks=s)
    assert np.abs(o - out.detach().numpy()).max() < 1e-12
    assert np.abs(lse - torch.logsumexp(sc.masked_fill(~see, -math.inf), -1).detach().numpy()).max() < 1e-12
    for a, t in zip(gr, x):
        assert np.abs(a - t.grad.numpy()).max() < 1e-11


@pytest.mark.parametrize("w,s", [(0, 1), (100, 5), (128, 129), (300, 64), (700, 400)])
def test_sink_maps_cover_every_visible_pair_once(w, s):
    """Every visible (query, key) pair lies in exactly one listed tile, and no listed key or query
    block is without a visible pair."""
    cu = [0, 1, 130, 900]
    for BM, BN in ((256, 128), (128, 64)):
        seen = set()
        for b, m, _h, nb in ot.fwd_tile_map(cu, 1, BM, BN, True, 0, window=w, sinks=s).tolist():
            l = cu[b + 1] - cu[b]
            ns, k0 = ot.sink_blocks(m, l, BM, BN, w, s), ot.window_key_start(m, BM, BN, w)
            for n in range(nb):
                n = n if n < ns else k0 + n - ns
                pairs = {(b, i, j) for i in range(m * BM, min(l, m * BM + BM)) for j in range(n * BN, min(l, n * BN + BN))
                         if j <= i and (j >= i - w or j < s)}
                assert pairs and not (pairs & seen)
                seen |= pairs
        want = {(b, i, j) for b in range(3) for i in range(cu[b + 1] - cu[b]) for j in range(i + 1)
                if j >= i - w or j < s}
        assert seen == want
    BM, BN = 64, 128
    seen = set()
    for b, n, _h, nq in ot.bwd_tile_map(cu, 1, BM, BN, True, 0, window=w, sinks=s).tolist():
        l = cu[b + 1] - cu[b]
        for m in range(n * BN // BM, n * BN // BM + nq):
            pairs = {(b, i, j) for i in range(m * BM, min(l, m * BM + BM)) for j in range(n * BN, min(l, n * BN + BN))
                     if j <= i and (j >= i - w or j < s)}
            assert pairs and not (pairs & seen)
            seen |= pairs
    assert seen == want
