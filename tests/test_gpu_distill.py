"""GPU parity of the distillation from a teacher's top logits against the float64 oracle."""
import math

import numpy as np
import pytest
import torch

from oracle import loss as ol

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
VA_ERR_BAD_TARGETS = 8


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    pkg._lib.load()
    return pkg


def inputs(T, V, K, dtype, seed, a_dtype=F32):
    g = torch.Generator().manual_seed(seed)
    z = (3 * torch.randn(T, V, generator=g)).to(dtype)
    ids = torch.randint(0, V, (T, K), generator=g, dtype=torch.int32)
    a = (2 * torch.randn(T, K, generator=g)).to(a_dtype)
    ids[torch.rand(T, K, generator=g) < 0.1] = -1
    ids[0, 0] = V - 1                                       # the last class; row 0 stays eligible
    tg = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    tg[torch.rand(T, generator=g) < 0.2] = -100
    tg[0] = 0
    return z, ids, a, tg


def check(va, z, ids, a, tg, tau, zd=None, gd=True):
    """Tolerances.  The base-2 exponents y = z log2(e) / tau are at most Y in magnitude, their
    log-sum-exp too (2 Y below covers both).  Each of the scale's rounding, the product's, the
    sum's and the log-sum-exp's own costs at most 2^-24 of 2 Y: an exponent is off by 2^-22 Y', Y' =
    2 Y, and ex2 / log2 add 2^-21; the row loss, a weighted sum of such exponents, is off by
    tau^2 times twice that (student and teacher).  The weights p_k are exponentials of such
    exponents and carry the same relative error into sum_k p_k |ln p_k - ln q_k|, which is the loss
    plus at most twice its negative part, the entropy of p (<= ln K); then two roundings to fp32 of
    the row's value and one of the sum.  A gradient value is tau / N (q - P): that
    relative error of q + P, then (bf16) half a step 2^-8 of the value."""
    zd = z.to(DEV) if zd is None else zd
    loss, count, grad = va.token_distill(zd, ids.to(DEV), a.to(DEV), None if tg is None else tg.to(DEV),
                                         temperature=tau, grad=gd, check_status=True)
    has = np.ones(len(z), bool) if tg is None else tg.numpy() != -100
    zz = z.double().numpy().copy()
    skip = ~has | ~((ids.numpy() >= 0) & (a.double().numpy() > -np.inf)).any(1)
    zz[skip] = 0
    rs, rmean, n, rg = ol.top_logit_distillation(zz, ids.numpy(), a.double().numpy(), has, tau)
    s, mean = loss.cpu().tolist()
    big = [np.abs(x[np.isfinite(x) & (np.abs(x) < 1e30)]).max(initial=1.0) for x in (zz, a.double().numpy())]
    Y = 2 * max(big) * 1.4427 / tau
    rel = 2.0 ** -22 * Y + 2.0 ** -21
    assert int(count.item()) == n
    assert abs(s - rs) <= (2.0 ** -22 + rel) * abs(rs) + (2 + 2 * math.log(ids.shape[1])) * rel * tau * tau * n
    assert abs(mean - rmean) <= (2.0 ** -22 + rel) * abs(rmean) + (2 + 2 * math.log(ids.shape[1])) * rel * tau * tau
    if grad is None:
        return loss, None
    g = grad.cpu().double().numpy()
    assert np.all(g[skip] == 0) and np.isfinite(g).all()
    # q + P in the same units: |grad| + 2 P bounds it
    P = np.zeros_like(rg)
    for t in range(len(z)):
        keep = (ids[t].numpy() >= 0) & (a[t].double().numpy() > -np.inf)
        if skip[t] or not keep.any():
            continue
        x = a[t].double().numpy()[keep] / tau
        np.add.at(P[t], ids[t].numpy()[keep], np.exp(x - x.max()) / np.exp(x - x.max()).sum() * tau / n)
    half = 2.0 ** -8 if z.dtype == BF else 2.0 ** -24
    tol = rel * (np.abs(rg) + 2 * P) + half * (1 + 2.0 ** -10) * np.abs(rg) + 1e-37
    assert (np.abs(g - rg) <= tol).all(), np.max(np.abs(g - rg) / tol)
    return loss, grad


# V: less than one 16-byte vector; below, at and past a warp's piece; odd (unaligned rows); slices
# over two, four and eight CTAs
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (3, 5, 2), (7, 17, 33), (130, 500, 64), (20, 2049, 1), (5, 4099, 1024),
                                   (40, 32768, 64), (33, 50003, 17), (9, 131072, 128), (2, 300001, 5)])
def test_parity(va, dtype, T, V, K):
    z, ids, a, tg = inputs(T, V, K, dtype, T + V + K)
    check(va, z, ids, a, tg, 1.0 if K != 64 else 2.0)


def test_many_rows_use_one_cta_each_and_wrap(va):
    """More rows than CTAs, eligible and skipped rows in every pattern."""
    z, ids, a, tg = inputs(3001, 600, 9, BF, 4)
    tg[1000:1040] = -100
    check(va, z, ids, a, tg, 0.7)


@pytest.mark.parametrize("a_dtype", [F32, BF])
@pytest.mark.parametrize("tau", [0.25, 1.0, 8.0])
def test_temperature_and_teacher_types(va, a_dtype, tau):
    z, ids, a, tg = inputs(50, 1000, 20, F32, 77, a_dtype)
    check(va, z, ids, a, None, tau)


def test_masked_entries_and_rows(va):
    """Absent entries (negative ids, -inf and NaN logits), rows without any, rows of NaN or inf
    logits that are skipped, the type's lowest value among logits and teacher logits."""
    z, ids, a, tg = inputs(12, 700, 8, BF, 5)
    tg[:] = 1
    ids[3] = -1                                             # nothing present: skipped
    a[4] = -math.inf                                        # likewise
    a[5, 2:] = -math.inf
    a[6, 1] = math.nan
    ids[7, :7] = -5
    tg[8] = -100
    z[3], z[4], z[8] = math.nan, math.inf, -math.inf
    z[9, 100:600] = torch.finfo(BF).min
    z[10, 5] = -math.inf                                    # a class without probability, not listed
    ids[10][ids[10] == 5] = 6
    a[11, 3] = torch.finfo(F32).min
    aa = a.clone()
    aa[6, 1] = -math.inf                                    # the oracle's spelling of absent
    zd, idd = z.to(DEV), ids.to(DEV)
    l1, _, g1 = va.token_distill(zd, idd, a.to(DEV), tg.to(DEV), check_status=True)
    l2, g2 = check(va, z, ids, aa, tg, 1.0)
    assert torch.equal(l1, l2) and torch.equal(g1, g2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_class_listed_several_times(va, dtype):
    z, ids, a, _ = inputs(6, 901, 40, dtype, 8)
    ids[0] = 13
    ids[1, ::2] = 900
    ids[2] = torch.arange(40, dtype=torch.int32) % 3        # the first, maybe unaligned elements
    ids[3, 5] = ids[3, 39]
    check(va, z, ids, a, None, 1.0)


def test_strides_alignment_and_in_place(va):
    """Padded rows, logits and gradient rows on different 16-byte phases, the gradient over the
    logits.  Where a row starts decides how its sum is grouped, so rows on another phase are held to
    the oracle; where the gradient goes and how the teacher's rows lie changes no bit."""
    z, ids, a, tg = inputs(37, 1003, 11, BF, 9)
    idd, ad, tgd = ids.to(DEV), a.to(DEV), tg.to(DEV)
    loss, grad = check(va, z, ids, a, tg, 1.0)
    big = torch.full((37, 1100), 7.0, dtype=BF, device=DEV)
    zd = torch.zeros(37, 1024, dtype=BF, device=DEV)[:, 3:1006]
    zd.copy_(z)
    loss3, grad3 = check(va, z, ids, a, tg, 1.0, zd=zd)
    for off in (0, 1, 3, 8):
        gd = big[:, off:off + 1003]
        l2, _, g2 = va.token_distill(zd, idd, ad, tgd, grad=gd)
        assert torch.equal(l2, loss3) and torch.equal(g2, grad3)
        assert (big[:, off + 1003:] == 7).all() and (big[:, :off] == 7).all()   # nothing beside the rows
        big.fill_(7.0)
    l3, _, g3 = va.token_distill(zd, idd, ad, tgd, grad=zd)
    assert torch.equal(l3, loss3) and torch.equal(zd, grad3) and g3.data_ptr() == zd.data_ptr()
    l4, _, none = va.token_distill(z.to(DEV), idd, ad, tgd, grad=False)
    assert none is None and torch.equal(l4, loss)
    wide = torch.zeros(37, 64, dtype=torch.int32, device=DEV)[:, 5:16]
    wide.copy_(idd)
    widea = torch.zeros(37, 64, device=DEV)[:, 1:12]
    widea.copy_(ad)
    l5, _, g5 = va.token_distill(z.to(DEV), wide, widea, tgd)
    assert torch.equal(l5, loss) and torch.equal(g5, grad)


def test_gradient_against_differences(va):
    """The mean loss of fp32 logits moved by h along a random direction, central differences in the
    kernel's own fp32 loss: its error per row as in check() (exponents within 2 * 16 * 1.44 / 2), over
    h, plus the third-order term."""
    z, ids, a, tg = inputs(8, 300, 16, F32, 12)
    u = torch.randn(z.shape, generator=torch.Generator().manual_seed(1))
    _, _, g = va.token_distill(z.to(DEV), ids.to(DEV), a.to(DEV), tg.to(DEV), temperature=2.0)
    h, f = 0.05, []
    for sgn in (-1, 1):
        f.append(va.token_distill((z + sgn * h * u).to(DEV), ids.to(DEV), a.to(DEV), tg.to(DEV), temperature=2.0,
                                  grad=False)[0][1].item())
    slope = float((g.cpu().double() * u.double()).sum())
    # third derivative of the log-sum-exp along u at temperature 2: below tau^2 max|u - mean|^3 / tau^3
    third = 4 * (2 * u.abs().max().item()) ** 3 / 8
    assert abs((f[1] - f[0]) / (2 * h) - slope) <= 4 * 2 * (2.0 ** -22 * 24 + 2.0 ** -21) / h + h * h / 6 * third


def test_device_errors_and_reuse(va):
    """A class >= V in an eligible row, or no eligible row: status, NaN loss, gradient untouched;
    the next call on the same workspace is right."""
    z, ids, a, tg = (x.to(DEV) for x in inputs(6, 50, 4, F32, 2))
    lib = va._lib.load()
    ws = torch.full((lib.varlen_token_distill_workspace_size(6),), 0x7f, dtype=torch.uint8, device=DEV)
    g = torch.full((6, 50), 3.0, device=DEV)
    for i, t in ((ids.clone(), tg), (ids, torch.full_like(tg, -100)), (torch.full_like(ids, -1), tg)):
        if t is tg and int(i.max()) >= 0:
            i[0, 1] = 50
        loss, _, _ = va.token_distill(z, i, a, t, workspace=ws, grad=g)
        assert va.read_status(ws) == VA_ERR_BAD_TARGETS
        assert all(math.isnan(x) for x in loss.cpu().tolist()) and (g == 3).all()
    skipped = ids.clone()
    skipped[1] = 99                                          # out of range, but the row is ignored
    t = tg.clone()
    t[1] = -100
    loss, _, _ = va.token_distill(z, skipped, a, t, workspace=ws, grad=g)
    assert va.read_status(ws) == 0 and all(math.isfinite(x) for x in loss.cpu().tolist())
    with pytest.raises(va.VarlenError):
        va.token_distill(z, torch.full_like(ids, -1), a, tg, check_status=True)


def test_refusals(va):
    z, ids, a, tg = (x.to(DEV) for x in inputs(6, 50, 4, F32, 3))
    for args in ((z.half(), ids, a, tg), (z.t(), ids, a, tg), (z, ids.long(), a, tg), (z, ids[:5], a[:5], tg),
                 (z, ids, a[:, :3], tg), (z, ids, a.half(), tg), (z, ids, a, tg.long()), (z, ids, a, tg[:5]),
                 (z, ids.cpu(), a, tg), (z, ids, a, tg.cpu())):
        with pytest.raises(ValueError):
            va.token_distill(*args)
    with pytest.raises(ValueError):
        va.token_distill(z, ids, a, tg, grad=torch.empty(6, 50, dtype=BF, device=DEV))
    for kw in (dict(temperature=0.0), dict(temperature=math.inf)):
        with pytest.raises(va.VarlenError) as e:
            va.token_distill(z, ids, a, tg, **kw)
        assert e.value.status == 1
    with pytest.raises(va.VarlenError):                      # one row seen six times: strides below the row
        va.token_distill(z[:1].expand(6, 50), ids, a, tg)


def test_graph_replay_on_a_side_stream(va):
    """A captured call on static buffers replays on new inputs bit-equal to eager calls."""
    z, ids, a, tg = (x.to(DEV) for x in inputs(70, 40000, 24, BF, 1))
    ws = torch.empty(va._lib.load().varlen_token_distill_workspace_size(70), dtype=torch.uint8, device=DEV)
    g = torch.empty_like(z)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        va.token_distill(z, ids, a, tg, grad=g, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        loss, count, _ = va.token_distill(z, ids, a, tg, grad=g, workspace=ws)
    for seed in (2, 3):
        for x, y in zip((z, ids, a, tg), inputs(70, 40000, 24, BF, seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        l2, c2, g2 = va.token_distill(z, ids, a, tg)
        assert torch.equal(loss, l2) and torch.equal(count, c2) and torch.equal(g, g2)


@pytest.mark.parametrize("T,V,K,dtype", [(250, 50257, 40, F32), (20, 50257, 40, F32), (130, 151936, 64, BF), (64, 128256, 9, F32),
                                         (24, 300007, 33, F32), (40, 100003, 1024, BF)])
def test_clusters_of_every_size(va, T, V, K, dtype):
    """Rows over clusters whose size is no power of two, more rows than clusters that fit at once."""
    z, ids, a, tg = inputs(T, V, K, dtype, V + T)
    check(va, z, ids, a, tg, 1.5)
    alone = va.token_distill(z.to(DEV), ids.to(DEV), a.to(DEV), tg.to(DEV), temperature=1.5)
    again = va.token_distill(z.to(DEV), ids.to(DEV), a.to(DEV), tg.to(DEV), temperature=1.5)
    assert all(torch.equal(x, y) for x, y in zip(alone, again))


def test_captured_call_whose_clusters_fill_the_gpu(va):
    z, ids, a, tg = (x.to(DEV) for x in inputs(400, 131072, 20, BF, 9))
    want = va.token_distill(z, ids, a, tg)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        va.token_distill(z, ids, a, tg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        got = va.token_distill(z, ids, a, tg)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
