"""GPU parity of the query / key norm with the position rotation, and of its gradient, against float64."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    pkg._lib.load()
    return pkg


def turn(x, pos, inv, interleaved, back=False):
    """x [T, H, d] float64, its first 2 len(inv) dims turned by pos * inv."""
    rot = 2 * len(inv)
    f = (pos.double()[:, None] * inv.double())[:, None]
    c, s = f.cos(), -f.sin() if back else f.sin()
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y = x.clone()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def reference(x, w, pos, inv, eps, interleaved, dy=None):
    """(y, bound of its fp32 error), and with dy (dx, bound, dw, bound)."""
    d = x.shape[-1]
    x = x.double()
    w = torch.ones(d, dtype=torch.float64) if w is None else w.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = x * r
    y = turn(n * w, pos, inv, interleaved)
    # a sum of d squares, a root, three products, an angle (2^-24 turns) and its functions, two products and a sum:
    # each pair's error is within (d / 2 + 32) half steps of fp32 of both its magnitudes
    def both(u):
        rot, m = 2 * len(inv), u.abs()
        i = torch.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        m[..., a], m[..., b] = m[..., a] + m[..., b], m[..., a] + m[..., b]
        return m
    ulp = (d / 2 + 32) * 2.0 ** -24
    if dy is None:
        return y, ulp * both(n * w)
    g = turn(dy.double(), pos, inv, interleaved, back=True)
    mean = (g * w * n).mean(-1, keepdim=True)
    dx = r * (g * w - n * mean)
    big = both(dy.double())
    ex = 4 * ulp * r * (big * w.abs() + n.abs() * (big * (w * n).abs()).mean(-1, keepdim=True))
    count = x.shape[0] * x.shape[1]
    return dx, ex, (g * n).sum((0, 1)), (count + d + 64) * 2.0 ** -24 * (big * n.abs()).sum((0, 1))


def close(got, ref, err):
    assert got.shape == ref.shape
    if got.numel() == 0:
        return
    tol = HALF[got.dtype] * (1 + 2.0 ** -7) * ref.abs() + err + 1e-37
    off = (got.cpu().double() - ref).abs() / tol
    assert float(off.max()) <= 1, float(off.max())


def make(T, Hq, Hkv, d, rot, dt, wdt, far=0, seed=0):
    g = torch.Generator().manual_seed(seed + T + d)
    mk = lambda *s: torch.randn(*s, generator=g)                             # noqa: E731
    inv = 10000.0 ** (-torch.arange(0, rot, 2).double() / max(rot, 1))
    pos = torch.randint(0, far + 1, (T,), generator=g).to(torch.int32) if far else torch.arange(T, dtype=torch.int32)
    return dict(q=(mk(T, Hq, d) * torch.exp(mk(T, Hq, 1))).to(dt), k=(3 * mk(T, Hkv, d)).to(dt), qw=(1 + 0.3 * mk(d)).to(wdt),
                kw=(mk(d)).to(wdt), inv=inv.float(), pos=pos, dq=mk(T, Hq, d).to(dt), dk=mk(T, Hkv, d).to(dt))


SHAPES = [(1, 1, 1, 64, 64), (446, 32, 8, 128, 128), (33, 7, 7, 80, 40), (65, 8, 2, 64, 32), (19, 3, 1, 8, 8),
          (130, 12, 1, 256, 256), (77, 5, 2, 96, 16), (40, 2, 2, 248, 240), (9, 1, 1, 16, 0), (700, 4, 4, 32, 32),
          (3000, 6, 1, 128, 64)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot", SHAPES)
def test_parity(va, T, Hq, Hkv, d, rot, dt, wdt, interleaved):
    m = make(T, Hq, Hkv, d, rot, dt, wdt)
    c = {n: x.to(DEV) for n, x in m.items()}
    qo, ko = va.qk_norm_rope_fwd(c["q"], c["k"], c["pos"], c["qw"], c["kw"], c["inv"], 1e-5, interleaved)
    close(qo, *reference(m["q"], m["qw"], m["pos"], m["inv"], 1e-5, interleaved))
    close(ko, *reference(m["k"], m["kw"], m["pos"], m["inv"], 1e-5, interleaved))
    got = va.qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], c["pos"], c["qw"], c["kw"], c["inv"], 1e-5, interleaved)
    for x, w, dy, dx, dw in ((m["q"], m["qw"], m["dq"], got[0], got[2]), (m["k"], m["kw"], m["dk"], got[1], got[3])):
        rx, ex, rw, ew = reference(x, w, m["pos"], m["inv"], 1e-5, interleaved, dy)
        close(dx, rx, ex)
        close(dw, rw, ew)
    again = va.qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], c["pos"], c["qw"], c["kw"], c["inv"], 1e-5, interleaved)
    assert all(torch.equal(a, b) for a, b in zip(got, again))                # the same bits every time


@pytest.mark.parametrize("far", [10 ** 5, 10 ** 6, 2 ** 31 - 1])
def test_far_positions(va, far):
    """A position of two thousand million is turned as accurately as the first."""
    m = make(50, 2, 1, 128, 128, F32, F32, far=far - 1)
    m["pos"][0], m["pos"][1] = far, -far
    c = {n: x.to(DEV) for n, x in m.items()}
    qo, ko = va.qk_norm_rope_fwd(c["q"], c["k"], c["pos"], c["qw"], c["kw"], c["inv"])
    # (float64 itself loses 2^-53 of up to far turns per unit of angle)
    extra = far * 2.0 ** -51
    for x, w, y in ((m["q"], m["qw"], qo), (m["k"], m["kw"], ko)):
        ref, err = reference(x, w, m["pos"], m["inv"], 1e-6, False)
        close(y, ref, err + extra * ref.abs().max())


def test_rows_and_scales(va):
    """A row of zeros stays zero with a finite gradient; large and small rows; no weights; no rotation."""
    T, H, d = 6, 2, 64
    x = torch.randn(T, H, d, generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1] *= 1e15
    x[2] *= 1e-12
    pos, dy = torch.arange(T, dtype=torch.int32), torch.randn(T, H, d, generator=torch.Generator().manual_seed(2))
    inv = torch.tensor([1.0, 0.5, 0.25, 0.125])
    qo, ko = va.qk_norm_rope_fwd(x.to(DEV), x.to(DEV), pos.to(DEV), None, None, inv.to(DEV))
    ref, err = reference(x, None, pos, inv, 1e-6, False)
    close(qo, ref, err)
    close(ko, ref, err)
    assert torch.equal(qo[0].cpu(), torch.zeros(H, d))
    dq, dk, dqw, dkw = va.qk_norm_rope_bwd(dy.to(DEV), dy.to(DEV), x.to(DEV), x.to(DEV), pos.to(DEV), None, None, inv.to(DEV))
    rx, ex, _, _ = reference(x, None, pos, inv, 1e-6, False, dy)
    close(dq, rx, ex)
    close(dk, rx, ex)
    assert dqw is None and dkw is None
    plain, _ = va.qk_norm_rope_fwd(x.to(DEV), x.to(DEV), pos.to(DEV))
    close(plain, *reference(x, None, pos, torch.zeros(0), 1e-6, False))
    w = torch.linspace(-1, 1, d)                                             # one weight alone
    got = va.qk_norm_rope_bwd(dy.to(DEV), dy.to(DEV), x.to(DEV), x.to(DEV), pos.to(DEV), None, w.to(DEV), inv.to(DEV))
    assert got[2] is None
    rx, ex, rw, ew = reference(x, w, pos, inv, 1e-6, False, dy)
    close(got[1], rx, ex)
    close(got[3], rw, ew)


def test_views_in_place_and_fused_gradient(va):
    """Views of a fused projection in, a fused gradient out, outputs over inputs; what lies between is left."""
    T, Hq, Hkv, d = 200, 4, 2, 64
    m = make(T, Hq, Hkv, d, d, BF, BF)
    c = {n: x.to(DEV) for n, x in m.items()}
    want = va.qk_norm_rope_fwd(c["q"], c["k"], c["pos"], c["qw"], c["kw"], c["inv"])
    wgrad = va.qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], c["pos"], c["qw"], c["kw"], c["inv"])
    qkv = torch.randn(T, Hq + 2 * Hkv, d, device=DEV).to(BF)
    qkv[:, :Hq], qkv[:, Hq:Hq + Hkv] = c["q"], c["k"]
    v = qkv[:, Hq + Hkv:].clone()
    dqkv = torch.full_like(qkv, 7)
    a = (c["pos"], c["qw"], c["kw"], c["inv"])
    got = va.qk_norm_rope_bwd(c["dq"], c["dk"], qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], *a, dq=dqkv[:, :Hq], dk=dqkv[:, Hq:Hq + Hkv])
    assert all(torch.equal(x, y) for x, y in zip(got, wgrad))
    assert bool((dqkv[:, Hq + Hkv:] == 7).all())
    va.qk_norm_rope_fwd(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], *a, q_out=qkv[:, :Hq], k_out=qkv[:, Hq:Hq + Hkv])
    assert torch.equal(qkv[:, :Hq], want[0]) and torch.equal(qkv[:, Hq:Hq + Hkv], want[1])
    assert torch.equal(qkv[:, Hq + Hkv:], v)
    heads_first = c["q"].transpose(0, 1).contiguous().transpose(0, 1)         # [H, T, d] in memory
    qo, _ = va.qk_norm_rope_fwd(heads_first, c["k"], *a)
    assert torch.equal(qo, want[0])
    dyq, dyk = c["dq"].clone(), c["dk"].clone()
    va.qk_norm_rope_bwd(dyq, dyk, c["q"], c["k"], *a, dq=dyq, dk=dyk)
    assert torch.equal(dyq, wgrad[0]) and torch.equal(dyk, wgrad[1])


def test_broadcast_heads(va):
    """One key head expanded to several, and one row of gradients for all tokens: as if they were copied."""
    T, Hq, d = 70, 4, 64
    m = make(T, Hq, 1, d, d, BF, BF)
    c = {n: x.to(DEV) for n, x in m.items()}
    a = (c["pos"], c["qw"], c["kw"], c["inv"])
    wide = c["k"].expand(T, 3, d)
    got = va.qk_norm_rope_fwd(c["q"], wide, *a)
    want = va.qk_norm_rope_fwd(c["q"], wide.contiguous(), *a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dk = c["dk"][:1].expand(T, 3, d)
    got = va.qk_norm_rope_bwd(c["dq"], dk, c["q"], wide, *a)
    want = va.qk_norm_rope_bwd(c["dq"], dk.contiguous(), c["q"], wide.contiguous(), *a)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    k = c["k"].clone().requires_grad_()
    out = va.qk_norm_rope(c["q"], k.expand(T, 3, d), *a)[1]
    out.backward(dk)
    near = want[1].float().sum(1, keepdim=True)                 # the sum's own rounding, and those of its terms
    tol = (want[1].float().abs().sum(1, keepdim=True) + near.abs()) * 2.0 ** -8 * 3
    assert bool(((k.grad.float() - near).abs() <= tol).all())


def test_no_tokens(va):
    q = torch.empty(0, 4, 64, device=DEV, dtype=BF)
    pos = torch.empty(0, dtype=torch.int32, device=DEV)
    w, inv = torch.ones(64, device=DEV, dtype=BF), torch.ones(32, device=DEV)
    qo, ko = va.qk_norm_rope_fwd(q, q, pos, w, w, inv)
    assert qo.shape == ko.shape == (0, 4, 64)
    _, _, dqw, dkw = va.qk_norm_rope_bwd(q, q, q, q, pos, w, w, inv)
    assert float(dqw.abs().sum()) == float(dkw.abs().sum()) == 0


def test_autograd_and_differences(va):
    T, Hq, Hkv, d = 9, 3, 1, 32
    m = make(T, Hq, Hkv, d, 16, F32, F32)
    c = {n: x.to(DEV) for n, x in m.items()}
    leaves = [c[n].clone().requires_grad_(True) for n in ("q", "k", "qw", "kw")]
    qo, ko = va.qk_norm_rope(leaves[0], leaves[1], c["pos"], leaves[2], leaves[3], c["inv"])
    ((qo * c["dq"]).sum() + (ko * c["dk"]).sum()).backward()

    def loss(q, k, qw, kw):
        a, _ = reference(q, qw, m["pos"], m["inv"], 1e-6, False)
        b, _ = reference(k, kw, m["pos"], m["inv"], 1e-6, False)
        return float((a * m["dq"].double()).sum() + (b * m["dk"].double()).sum())

    g = torch.Generator().manual_seed(3)
    for i, leaf in enumerate(leaves):
        way = torch.randn(leaf.shape, generator=g, dtype=torch.float64)
        at = [m[n].double() for n in ("q", "k", "qw", "kw")]
        h = 1e-6
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * way, at[i] - h * way
        diff = (loss(*up) - loss(*down)) / (2 * h)
        got = float((leaf.grad.cpu().double() * way).sum())
        # the differences' own error: h^2 of third derivatives and 2^-52 / h of the loss, some 1e-8 here
        scale = float((leaf.grad.cpu().double() * way).abs().sum())
        assert abs(got - diff) <= 1e-5 * scale + 1e-6


def test_graph_and_streams(va):
    """A captured forward and backward, replayed on new inputs, and two streams at once."""
    m = make(300, 8, 2, 128, 128, BF, BF)
    c = {n: x.to(DEV) for n, x in m.items()}

    def both():
        return va.qk_norm_rope_fwd(c["q"], c["k"], c["pos"], c["qw"], c["kw"], c["inv"]) + \
            va.qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], c["pos"], c["qw"], c["kw"], c["inv"])
    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for _ in range(3):
        c["q"].copy_(torch.randn_like(c["q"]))
        c["pos"].copy_(torch.randint_like(c["pos"], 5000))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, both()))
    want = both()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(both())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in got for a, b in zip(o, want))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d", [(3, 1, 128), (5, 1, 64), (1, 1, 64), (7, 2, 80), (1, 3, 256), (2, 1, 32)])
def test_no_eps(va, Hq, Hkv, d, dt):
    """eps = 0 with heads that leave lanes over: the norm of rows that are not zero, and every gradient."""
    m = make(60, Hq, Hkv, d, d, dt, dt)
    c = {n: x.to(DEV) for n, x in m.items()}
    a = (c["pos"], c["qw"], c["kw"], c["inv"], 0.0)
    qo, ko = va.qk_norm_rope_fwd(c["q"], c["k"], *a)
    close(qo, *reference(m["q"], m["qw"], m["pos"], m["inv"], 0.0, False))
    close(ko, *reference(m["k"], m["kw"], m["pos"], m["inv"], 0.0, False))
    got = va.qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], *a)
    for x, w, dy, dx, dw in ((m["q"], m["qw"], m["dq"], got[0], got[2]), (m["k"], m["kw"], m["dk"], got[1], got[3])):
        rx, ex, rw, ew = reference(x, w, m["pos"], m["inv"], 0.0, False, dy)
        close(dx, rx, ex)
        close(dw, rw, ew)


def test_gradients_off_their_boundaries(va):
    """The outputs' gradients as autograd may hand them over: contiguous parts of a larger one, off 16-byte boundaries."""
    m = make(20, 2, 1, 64, 64, BF, BF)
    c = {n: x.to(DEV) for n, x in m.items()}
    a = (c["pos"], c["qw"], c["kw"], c["inv"])
    want = va.qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], *a)
    q, k = (c[n].clone().requires_grad_(True) for n in ("q", "k"))
    qo, ko = va.qk_norm_rope(q, k, *a)
    flat = torch.cat([torch.zeros(3, device=DEV, dtype=BF), qo.reshape(-1), torch.zeros(2, device=DEV, dtype=BF), ko.reshape(-1)])
    up = torch.cat([torch.zeros(3, device=DEV, dtype=BF), c["dq"].reshape(-1), torch.zeros(2, device=DEV, dtype=BF), c["dk"].reshape(-1)])
    flat.backward(up)
    assert torch.equal(q.grad, want[0]) and torch.equal(k.grad, want[1])


def test_frozen_weights(va):
    """Weights that want no gradient have none formed: the others' gradients are the same bits, and with both frozen the
    launch that adds the weights' up is left out."""
    m = make(90, 3, 1, 64, 64, BF, BF)
    c = {n: x.to(DEV) for n, x in m.items()}
    a = (c["pos"], c["qw"], c["kw"], c["inv"])
    want = va.qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], *a)
    count = va._lib.load().varlen_launch_count
    for qg, kg in ((False, False), (True, False), (False, True), (True, True)):
        q, k = (c[n].clone().requires_grad_(True) for n in ("q", "k"))
        qw, kw = c["qw"].clone().requires_grad_(qg), c["kw"].clone().requires_grad_(kg)
        qo, ko = va.qk_norm_rope(q, k, c["pos"], qw, kw, c["inv"])
        before = count()
        torch.autograd.backward([qo, ko], [c["dq"], c["dk"]])
        assert count() - before == (2 if qg or kg else 1)
        assert torch.equal(q.grad, want[0]) and torch.equal(k.grad, want[1])
        assert torch.equal(qw.grad, want[2]) if qg else qw.grad is None
        assert torch.equal(kw.grad, want[3]) if kg else kw.grad is None
