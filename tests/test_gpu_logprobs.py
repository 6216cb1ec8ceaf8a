"""GPU parity of token log probabilities, entropies, top alternatives and their gradient against float64."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
INF = float("inf")


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    pkg._lib.load()
    return pkg


def reference(z, tok, k, tau):
    """float64: (logprob, entropy, lse, ids, top) of every row (tokens clamped)."""
    x = z.double() / tau
    lse = torch.logsumexp(x, 1)
    lq = torch.log_softmax(x, 1)
    H = -torch.xlogy(lq.exp(), lq.exp()).sum(1)
    order = (z.float() + 0.0).sort(dim=1, descending=True, stable=True).indices[:, :k]
    return lq.gather(1, tok.clamp(min=0).long()[:, None])[:, 0], H, lse, order, lq.gather(1, order)


def unit(z, tau):
    """Half a step of fp32 times the roundings a row's sums go through: V / 32 terms in turn at the worst
    (a thread's part of a short row or a warp's), the joins, the exponential's 2^-22 (4 half steps) and the
    exponents' own size."""
    V = z.shape[1]
    return (V / 32 + 64 + 4 * (88 + math.log(V))) * 2.0 ** -24


def check_rows(got, z, tok, k, tau, ignore=-100):
    lp, H, lse, ids, top = (None if t is None else t.cpu() for t in got)
    rlp, rH, rlse, rids, rtop = reference(z, tok, k, tau)
    on = tok != ignore
    u = unit(z, tau)

    def near(a, r, mag):
        if a.numel() == 0:                                   # every row ignored
            return
        a, r = a.double(), r.double()
        same = (a == r) | (a.isnan() & r.isnan())
        off = torch.where(same, 0.0, (a - r).abs() / (u * (1 + mag) + 2.0 ** -22 * r.abs()))
        assert float(off.max()) <= 1, float(off.max())
    near(lp[on], rlp[on], rlp[on].abs().nan_to_num(posinf=0))
    near(H[on], rH[on], 16 + rH[on].abs())
    near(lse[on], rlse[on], rlse[on].abs().nan_to_num(posinf=0, neginf=0))
    for t in (lp, H, lse):
        assert bool((t[~on] == 0).all())
    if k:
        assert torch.equal(ids[on].long(), rids[on])
        near(top[on], rtop[on], rtop[on].abs().nan_to_num(posinf=0))
        assert bool((ids[~on] == -1).all()) and bool((top[~on] == 0).all())
    else:
        assert ids is None and top is None


def check_gradient(got, z, tok, dl, dh, tau, ignore=-100):
    x = z.double() / tau
    lse = torch.logsumexp(x, 1, keepdim=True)
    lq = torch.log_softmax(x, 1)
    p = lq.exp()
    H = -torch.xlogy(p, p).sum(1, keepdim=True)
    on = (tok != ignore)[:, None]
    dl, dh = dl.double()[:, None], torch.zeros_like(dl.double())[:, None] if dh is None else dh.double()[:, None]
    l0 = torch.where(p > 0, lq, torch.zeros_like(lq))
    hot = torch.zeros_like(p).scatter_(1, tok.clamp(min=0).long()[:, None], 1.0)
    ref = torch.where(on, (dl * (hot - p) - dh * p * (l0 + H)) / tau, 0.0)
    # p is off by the roundings of its exponent ((|x| + |lse| of at most 256) 2^-24, or the row's own sums) and
    # the exponential's 2^-22
    rel = (12 + lse.abs().clamp(max=256) + l0.abs() + z.shape[1] / 32) * 2.0 ** -22
    tol = HALF[got.dtype] * (1 + 2.0 ** -7) * ref.abs() + \
        (rel * p * (dl.abs() + dh.abs() * (l0.abs() + H + 1)) + 2.0 ** -22 * hot * dl.abs()) / tau + 1e-36
    off = (got.cpu().double() - ref).abs() / tol
    assert float(off.max()) <= 1, float(off.max())


def draw(T, V, dt, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed + T + V)
    z = (spread * torch.randn(T, V, generator=g)).to(dt)
    tok = torch.randint(0, V, (T,), generator=g).to(torch.int32)
    tok[torch.rand(T, generator=g) < 0.15] = -100
    return z, tok, torch.randn(T, generator=g), 0.3 * torch.randn(T, generator=g)


SHAPES = [(1, 1, 1), (3, 2, 2), (5, 7, 3), (4, 100, 64), (9, 257, 128), (2, 2047, 5), (33, 2048, 20), (6, 5003, 128), (3, 32000, 1),
          (5, 50003, 8), (2, 131072, 33), (1, 262147, 100), (700, 300, 4), (40, 1000, 0)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,V,k", SHAPES)
def test_parity(va, T, V, k, dt):
    for tau in (1.0, 0.7, 3.0):
        z, tok, dl, dh = draw(T, V, dt, k)
        zd, td = z.to(DEV), tok.to(DEV)
        got = va.token_logprobs_fwd(zd, td, top_k=k, temperature=tau, check_status=True)
        check_rows(got, z, tok, k, tau)
        grad = va.token_logprobs_bwd(zd, td, got[2], got[1], dl.to(DEV), dh.to(DEV), tau)
        check_gradient(grad, z, tok, dl, dh, tau)
        check_gradient(va.token_logprobs_bwd(zd, td, got[2], None, dl.to(DEV), temperature=tau), z, tok, dl, None, tau)
        again = va.token_logprobs_fwd(zd, td, top_k=k, temperature=tau)
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


# rows enough that each has a warp, 128 or 256 threads to itself, alternatives on either side of what those are chosen by
MANY = [(1300, 500, 64), (1300, 1001, 33), (1300, 2048, 64), (1220, 3001, 32), (320, 4096, 65), (310, 4097, 8), (330, 5003, 100),
        (310, 8200, 64), (306, 20011, 9)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,V,k", MANY)
def test_many_rows(va, T, V, k, dt):
    z, tok, dl, dh = draw(T, V, dt, k)
    zd, td = z.to(DEV), tok.to(DEV)
    got = va.token_logprobs_fwd(zd, td, top_k=k, check_status=True)
    check_rows(got, z, tok, k, 1.0)
    check_gradient(va.token_logprobs_bwd(zd, td, got[2], got[1], dl.to(DEV), dh.to(DEV)), z, tok, dl, dh, 1.0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_ties_and_orders(va, dt):
    """Rows of one value, of two, sorted either way, peaks side by side, -0 against 0: the lower id first."""
    for V, k in ((300, 100), (5000, 20), (70000, 64)):
        i = torch.arange(V, dtype=torch.float32)
        rows = [torch.zeros(V), torch.full((V,), -3.5), (i % 2), -(i % 2), i / V, -i / V, (i % 7 == 3).float(),
                torch.where(i >= V - 50, 5.0, 0.0), torch.where(i < 50, 5.0, 0.0), torch.where(i % 3 == 0, -0.0, 0.0),
                torch.where((i >= 100) & (i < 164), 2.0, 1.0), torch.where(i % 256 == 8, 3.0, 0.0), 1e-6 * i]
        z = torch.stack(rows).to(dt)
        tok = torch.arange(len(rows), dtype=torch.int32)
        got = va.token_logprobs_fwd(z.to(DEV), tok.to(DEV), top_k=k)
        check_rows(got, z, tok, k, 1.0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_masked_logits(va, dt):
    """-inf and the type's lowest value: nothing of the vocabulary left but one, some, none; the token itself masked."""
    V, low = 3001, torch.finfo(dt).min
    for mask in (-INF, low):
        z, _, dl, dh = draw(8, V, dt, 3)
        z[0, 1:] = mask
        z[1, :-1] = mask
        z[2, ::2] = mask
        z[3, 5] = mask
        z[4, 1000:] = mask
        z[5, :2999] = mask
        z[6] = mask
        tok = torch.tensor([0, V - 1, 1, 5, 999, 0, 0, 1], dtype=torch.int32)
        got = va.token_logprobs_fwd(z.to(DEV), tok.to(DEV), top_k=9)
        if mask == -INF:
            lp, H, lse = (t.cpu() for t in got[:3])
            assert math.isnan(float(lp[6])) and math.isnan(float(H[6])) and float(lse[6]) == -INF
            assert torch.equal(got[3][6].cpu(), torch.arange(9, dtype=torch.int32))
            keep = torch.tensor([0, 1, 2, 3, 4, 5, 7])
            check_rows([t[keep.to(DEV)] for t in got], z[keep], tok[keep], 9, 1.0)
        else:
            # (a row of the lowest value alone is a uniform one)
            keep = torch.arange(8)
            lp, H = got[0].cpu().double(), got[1].cpu().double()
            assert abs(float(lp[6]) + math.log(V)) < 1e-4 and abs(float(H[6]) - math.log(V)) < 1e-4
            assert torch.equal(got[3][6].cpu(), torch.arange(9, dtype=torch.int32))
            rows = torch.tensor([0, 1, 2, 4, 7])             # (the others' tokens are masked: values near the lowest)
            check_rows([t[rows.to(DEV)] for t in got], z[rows], tok[rows], 9, 1.0)
        grad = va.token_logprobs_bwd(z.to(DEV), tok.to(DEV), got[2], got[1], dl.to(DEV), dh.to(DEV)).cpu()
        if mask == -INF:
            assert bool(grad[6].isnan().all())
        rows = torch.tensor([0, 1, 2, 3, 4, 5, 7] if mask == -INF else [0, 1, 2, 4, 6, 7])
        d2 = dh.clone()
        zr = z[rows].double()
        zr[zr == low] = torch.where((zr == low).all(1, keepdim=True), torch.zeros_like(zr), torch.full_like(zr, -INF))[zr == low]
        check_gradient(grad[rows], zr, tok[rows], dl[rows], d2[rows], 1.0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_not_finite(va, dt):
    """NaN and +inf give NaN in their row and nowhere else; ids stay in the row."""
    T, V = 6, 4001
    z, _, dl, dh = draw(T, V, dt, 5)
    tok = torch.arange(T, dtype=torch.int32)
    want = va.token_logprobs_fwd(z.to(DEV), tok.to(DEV), top_k=40)
    z[1, 77], z[2, 0], z[3, :], z[4, 4000] = float("nan"), INF, float("nan"), -float("nan")
    got = va.token_logprobs_fwd(z.to(DEV), tok.to(DEV), top_k=40)
    grad = va.token_logprobs_bwd(z.to(DEV), tok.to(DEV), got[2], got[1], dl.to(DEV), dh.to(DEV))
    for t in (1, 2, 3, 4):
        assert bool(got[0][t].isnan()) and bool(got[1][t].isnan()) and bool(grad[t].isnan().any())
    assert bool(((got[3] >= 0) & (got[3] < V)).all())
    for t in (0, 5):
        assert all(torch.equal(a[t], b[t]) for a, b in zip(got, want))
        assert bool(grad[t].isfinite().all())


def test_large_logits(va):
    """Logits around +-5000: the sums of a row whose log-sum-exp has lost its fraction are formed again."""
    for shift in (300.0, -5000.0, 4.0e4, -2.0e6):
        z, tok, dl, dh = draw(7, 3000, F32, 8)
        z = z + shift
        got = va.token_logprobs_fwd(z.to(DEV), tok.to(DEV), top_k=3)
        rlp, rH, _, rids, _ = reference(z, tok, 3, 1.0)
        on = tok != -100
        assert torch.equal(got[3][on.to(DEV)].cpu().long(), rids[on])
        assert float((got[0].cpu().double() - rlp)[on].abs().max()) <= 600 * 2.0 ** -24 * 16
        assert float((got[1].cpu().double() - rH)[on].abs().max()) <= 600 * 2.0 ** -24 * 24
        check_gradient(va.token_logprobs_bwd(z.to(DEV), tok.to(DEV), got[2], got[1], dl.to(DEV), dh.to(DEV)), z, tok, dl, dh, 1.0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_strides_in_place_and_bad_tokens(va, dt):
    T, V = 12, 700
    z, tok, dl, dh = draw(T, V, dt, 9)
    want = va.token_logprobs_fwd(z.to(DEV), tok.to(DEV), top_k=7)
    wgrad = va.token_logprobs_bwd(z.to(DEV), tok.to(DEV), want[2], want[1], dl.to(DEV), dh.to(DEV))
    for off, width in ((0, 704), (8, 720), (1, 701), (3, 713)):
        wide = torch.full((T, width), 5.0, device=DEV, dtype=dt)
        v = wide[:, off:off + V]
        v.copy_(z)
        got = va.token_logprobs_fwd(v, tok.to(DEV), top_k=7)
        check_rows(got, z, tok, 7, 1.0)
        out = va.token_logprobs_bwd(v, tok.to(DEV), got[2], got[1], dl.to(DEV), dh.to(DEV), grad=v)
        assert out.data_ptr() == v.data_ptr()
        check_gradient(v, z, tok, dl, dh, 1.0)
        assert bool((wide[:, :off] == 5).all()) and bool((wide[:, off + V:] == 5).all())
    # a token outside the vocabulary: its row alone, and reported when asked
    bad = tok.clone()
    bad[0], bad[1] = V, -5
    got = va.token_logprobs_fwd(z.to(DEV), bad.to(DEV), top_k=7)
    assert bool(got[0][:2].isnan().all()) and torch.equal(got[0][2:], want[0][2:])
    grad = va.token_logprobs_bwd(z.to(DEV), bad.to(DEV), got[2], got[1], dl.to(DEV), dh.to(DEV))
    assert bool(grad[:2].isnan().all()) and torch.equal(grad[2:], wgrad[2:])
    with pytest.raises(va.VarlenError) as e:
        va.token_logprobs_fwd(z.to(DEV), bad.to(DEV), check_status=True)
    assert e.value.status == 8


def test_ignored_rows_are_not_read(va):
    z, tok, dl, dh = draw(5, 900, F32, 2)
    tok[1:4] = -100
    tok[0] = tok[4] = 3
    z[1:4] = float("nan")
    got = va.token_logprobs_fwd(z.to(DEV), tok.to(DEV), top_k=2)
    check_rows(got, torch.where(z.isnan(), 0.0, z), tok, 2, 1.0)
    grad = va.token_logprobs_bwd(z.to(DEV), tok.to(DEV), got[2], got[1], dl.to(DEV), dh.to(DEV))
    assert bool((grad[1:4] == 0).all())


def test_autograd_and_differences(va):
    z, tok, dl, dh = draw(6, 40, F32, 11)
    leaf = z.to(DEV).requires_grad_(True)
    lp, H, ids, top = va.token_logprobs(leaf, tok.to(DEV), top_k=3, temperature=1.3)
    assert not ids.requires_grad and not top.requires_grad
    ((lp * dl.to(DEV)).sum() + (H * dh.to(DEV)).sum()).backward()

    def loss(z):
        rlp, rH, _, _, _ = reference(z, tok, 0, 1.3)
        on = tok != -100
        return float((rlp * dl.double())[on].sum() + (rH * dh.double())[on].sum())

    way = torch.randn(z.shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    diff = (loss(z.double() + 1e-6 * way) - loss(z.double() - 1e-6 * way)) / 2e-6
    got = leaf.grad.cpu().double() * way
    assert abs(float(got.sum()) - diff) <= 1e-5 * float(got.abs().sum()) + 1e-7
    leaf.grad = None
    va.token_logprobs(leaf, tok.to(DEV))[1].sum().backward()                 # the entropy alone
    check_gradient(leaf.grad, z, tok, torch.zeros(6), torch.ones(6), 1.0)


def test_graph_and_streams(va):
    z, tok, dl, dh = (t.to(DEV) for t in draw(50, 4000, BF, 4))

    def both():
        got = va.token_logprobs_fwd(z, tok, top_k=6)
        return got + (va.token_logprobs_bwd(z, tok, got[2], got[1], dl, dh),)
    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for _ in range(3):
        z.copy_(torch.randn_like(z))
        g.replay()
        torch.cuda.synchronize()
        want = both()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    got = []
    for s in [torch.cuda.Stream(), torch.cuda.Stream()]:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(both())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in got for a, b in zip(o, want))


def test_offsets_past_32_bits(va):
    """More than 2^31 logits: the last rows against the same rows alone, bit for bit."""
    T, V = 17000, 131072
    z = torch.empty(T, V, device=DEV, dtype=BF)
    z.normal_(generator=torch.Generator(DEV).manual_seed(1))
    tok = torch.randint(0, V, (T,), device=DEV, dtype=torch.int32)
    dl = torch.randn(T, device=DEV)
    got = va.token_logprobs_fwd(z, tok, top_k=4)
    last = va.token_logprobs_fwd(z[-3:].contiguous(), tok[-3:].contiguous(), top_k=4)
    check_rows([t[-3:] for t in got], z[-3:].cpu(), tok[-3:].cpu(), 4, 1.0)
    assert torch.equal(got[3][-3:], last[3])
    grad = va.token_logprobs_bwd(z, tok, got[2], got[1], dl, dl, grad=z.clone())
    check_gradient(grad[-3:], z[-3:].cpu(), tok[-3:].cpu(), dl[-3:].cpu(), dl[-3:].cpu(), 1.0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("tau", [1.0 / 64, 0.3, 1.0, 64.0])
@pytest.mark.parametrize("V", [900, 3001, 20000])
def test_logits_of_any_size(va, V, tau, dt):
    """Rows whose largest logit lies anywhere in the type's range, of one value and of several; rows of ordinary logits
    of which most are replaced by a large negative number, as masks do, and with one large positive number.  The type
    rounds the given numbers, the reference takes them as they are."""
    k = 9
    g = torch.Generator().manual_seed(V)
    rows, tok = [], []
    for size in (1e4, 1e5, 1e6, 1.1e7, 1.3e7, 3e7, 1e9, 1e10, 1e12, 1e20, 1e28, 2e29, 1e35):
        for sign in (1.0, -1.0):
            m = sign * size
            plain = 2 * torch.randn(V, generator=g)
            rows.append(torch.full((V,), m))                                  # one value
            rows.append(m * (1 + 0.1 * torch.rand(V, generator=g)))           # of one size
            rows.append(plain + m)                                            # side by side
            tok += [3, V - 1, 7]
            some = plain.clone()
            some[torch.rand(V, generator=g) < 0.97] = m                       # most of them masked (or most of them large)
            some[5] = 1.5
            whole = plain.clone()
            whole[40:] = m
            one = plain.clone()
            one[V // 2] = m
            rows += [some, whole, one]
            tok += [5, 11, V // 2]
    z, tok = torch.stack(rows).to(dt), torch.tensor(tok, dtype=torch.int32)
    dl, dh = torch.randn(len(tok), generator=g), 0.3 * torch.randn(len(tok), generator=g)
    got = va.token_logprobs_fwd(z.to(DEV), tok.to(DEV), top_k=k, temperature=tau, check_status=True)
    assert bool(torch.stack([t.isfinite().all() for t in got[:3]]).all())
    check_rows(got, z, tok, k, tau)
    grad = va.token_logprobs_bwd(z.to(DEV), tok.to(DEV), got[2], got[1], dl.to(DEV), dh.to(DEV), tau).cpu()
    # a p below 2^-126, fp32's least normal number, is 0 in the kernel: dz is off by at most 2^-126 times what it is
    # multiplied with, (|dl| + |dH| (|ln p| + H)) / tau, some 1e-35 at tau = 1/64, and not by the bound's 1e-36
    x = z.double() / tau
    lq = torch.log_softmax(x, 1)
    p = lq.exp()
    H = -torch.xlogy(p, p).sum(1, keepdim=True)
    by = torch.where(p > 0, (dl.double().abs()[:, None] + dh.double().abs()[:, None] * (lq.abs() + H)) / tau, 0.0)
    tiny = (p < 2.0 ** -126) & (torch.arange(V) != tok.long()[:, None])
    assert bool((grad.double().abs() <= 2.0 ** -126 * (1 + 2.0 ** -7) * by)[tiny].all())
    ref = -p * (dl.double()[:, None] + dh.double()[:, None] * (torch.where(p > 0, lq, 0.0) + H)) / tau
    check_gradient(torch.where(tiny, ref.to(dt), grad), z, tok, dl, dh, tau)


def test_results_may_change_in_place(va):
    """The differentiable results have memory of their own: one changed in place leaves the others, and the gradient is the
    one of what was done."""
    z, tok, dl, dh = draw(40, 500, F32, 12)
    zd, td, keep = z.to(DEV), tok.to(DEV), (torch.arange(40, device=DEV) % 3 > 0).float()
    leaf = zd.clone().requires_grad_(True)
    lp, H, ids, top = va.token_logprobs(leaf, td, top_k=3)
    entropies = H.detach().clone()
    lp.mul_(keep)
    lp.sub_(0.5)
    assert torch.equal(H.detach(), entropies)
    ((lp * dl.to(DEV)).sum() + (H * dh.to(DEV)).sum()).backward()
    check_gradient(leaf.grad, z, tok, dl * keep.cpu(), dh, 1.0)


def test_gradient_beside_and_on_the_logits(va):
    """The gradient in the other half of the logits' rows; on a part of the logits it is refused."""
    T, V = 9, 3000
    z, tok, dl, dh = draw(T, V, F32, 21)
    wide = torch.zeros(T, 2 * V, device=DEV)
    wide[:, :V] = z.to(DEV)
    got = va.token_logprobs_fwd(wide[:, :V], tok.to(DEV))
    grad = va.token_logprobs_bwd(wide[:, :V], tok.to(DEV), got[2], got[1], dl.to(DEV), dh.to(DEV), grad=wide[:, V:])
    check_gradient(grad, z, tok, dl, dh, 1.0)
    assert torch.equal(wide[:, :V].cpu(), z)
    for to in (wide[:, 4:V + 4], wide.view(2 * T, V)[:T]):
        with pytest.raises(va.VarlenError) as e:
            va.token_logprobs_bwd(wide[:, :V], tok.to(DEV), got[2], got[1], dl.to(DEV), dh.to(DEV), grad=to)
        assert e.value.status == 1
