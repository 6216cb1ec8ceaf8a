"""Pins of the oracle's top-logit distillation: torch float64 autograd on the definition, and the
entry points' host-side refusals."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import loss as ol


@pytest.mark.parametrize("tau", [1.0, 0.5, 3.0])
def test_distillation_matches_autograd(tau):
    g = torch.Generator().manual_seed(int(10 * tau))
    T, V, K = 9, 23, 6
    z = torch.randn(T, V, generator=g, dtype=torch.float64, requires_grad=True)
    ids = torch.randint(0, V, (T, K), generator=g)                   # classes may repeat
    a = 3 * torch.randn(T, K, generator=g, dtype=torch.float64)
    ids[2, 3:] = -1
    ids[4] = -1
    has = torch.ones(T, dtype=torch.bool)
    has[5] = False
    total, n = 0.0, 0
    for t in range(T):
        keep = ids[t] >= 0
        if not has[t] or not keep.any():
            continue
        n += 1
        p = torch.softmax(a[t][keep] / tau, 0)
        total = total + tau ** 2 * (p * (p.log() - torch.log_softmax(z[t] / tau, 0)[ids[t][keep]])).sum()
    (total / n).backward()
    s, mean, N, grad = ol.top_logit_distillation(z.detach().numpy(), ids.numpy(), a.numpy(), has.numpy(), tau)
    assert N == n == 7
    assert abs(s - float(total)) < 1e-12 and abs(mean - float(total) / n) < 1e-12
    assert np.abs(grad - z.grad.numpy()).max() < 1e-14


def test_distillation_of_the_teacher_itself_is_zero():
    """All V classes listed with the student's own logits: loss 0, gradient 0."""
    z = np.random.default_rng(1).standard_normal((4, 11))
    ids = np.tile(np.arange(11), (4, 1))
    s, _, n, grad = ol.top_logit_distillation(z, ids, z, np.ones(4, bool), 2.0)
    assert n == 4 and abs(s) < 1e-13 and np.abs(grad).max() < 1e-15


@pytest.fixture(scope="module")
def lib():
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    return pkg._lib.load()


def test_host_side_refusals(lib):
    p, ok = ctypes.c_void_p(256), 1 << 20

    def call(logits=p, dtype=1, lrs=100, ids=p, irs=4, a=p, adt=0, ars=4, tg=None, T=8, V=100, K=4, tau=1.0, loss=p,
             count=p, grad=p, grs=100, ws=p, n=ok):
        return lib.varlen_token_distill(logits, dtype, lrs, ids, irs, a, adt, ars, tg, T, V, K, -100, tau, loss, count,
                                        grad, grs, ws, n, None)

    for kw in (dict(logits=None), dict(ids=None), dict(a=None), dict(loss=None), dict(count=None), dict(ws=None),
               dict(T=0), dict(V=0), dict(K=0), dict(dtype=2), dict(adt=3), dict(lrs=99), dict(irs=3), dict(ars=3),
               dict(grs=99), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")),
               dict(logits=ctypes.c_void_p(257)), dict(grad=ctypes.c_void_p(258), dtype=0),
               dict(ws=ctypes.c_void_p(264))):
        assert call(**kw) == 1, kw
    assert call(K=1025, irs=2000, ars=2000) == 2
    assert call(V=819201, lrs=819201, grs=819201) == 2 and call(V=409601, lrs=409601, grs=409601, dtype=0) == 2
    assert call(n=lib.varlen_token_distill_workspace_size(8) - 1) == 3
    assert lib.varlen_token_distill_workspace_size(-1) == 0


def test_temperature_range_and_sizes(lib):
    """Outside [1/64, 64] the fp32 loss would drown in the temperature's square; sizes stay below 2^30."""
    p = ctypes.c_void_p(256)
    for tau, T in ((64.5, 8), (1e-3, 8), (1e30, 8), (1e-40, 8), (1.0, 1 << 30)):
        assert lib.varlen_token_distill(p, 1, 100, p, 4, p, 0, 4, None, T, 100, 4, -100, tau, p, p, p, 100, p, 1 << 40,
                                        None) == 1, (tau, T)


def test_python_refusals_without_a_gpu(lib):
    import packed_sequence_varlen_gb300 as va
    with pytest.raises(ValueError):
        va.token_distill(torch.zeros(2, 5), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))
