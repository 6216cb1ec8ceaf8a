"""One packed distillation step through the operators together: metadata, embedding, attention with
a window and sinks, next-token targets, distillation from a teacher's top logits, and back to the
embedding table, against the same chain in float64 torch with a dense mask."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    pkg._lib.load()
    return pkg


def weights(V, D, Hq, Hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g).to(BF)                      # noqa: E731
    return dict(table=0.5 * mk(V, D), q=mk(Hq * d, D) / math.sqrt(D), k=mk(Hkv * d, D) / math.sqrt(D),
                v=mk(Hkv * d, D) / math.sqrt(D), o=mk(D, Hq * d) / math.sqrt(Hq * d), head=mk(V, D) / math.sqrt(D))


def reference(w, ids, lengths, tids, tlog, tau, window, sinks, scale, Hq, Hkv, d):
    """(mean loss, logits, gradients) in float64: the documents by a dense mask."""
    p = {n: x.double().requires_grad_(True) for n, x in w.items()}
    T = len(ids)
    x = scale * p["table"][ids]
    heads = lambda y, H: y.view(T, H, d).transpose(0, 1)                     # noqa: E731
    q, k, v = heads(x @ p["q"].T, Hq), heads(x @ p["k"].T, Hkv), heads(x @ p["v"].T, Hkv)
    see, ok, s = torch.zeros(T, T, dtype=torch.bool), torch.ones(T, dtype=torch.bool), 0
    for n in lengths:
        i = torch.arange(n)
        see[s:s + n, s:s + n] = (i[None] <= i[:, None]) & ((i[None] >= i[:, None] - window) | (i[None] < sinks))
        ok[s + n - 1] = False                                                # no target at a document's end
        s += n
    g = Hq // Hkv
    sc = (q @ k.repeat_interleave(g, 0).transpose(1, 2) / math.sqrt(d)).masked_fill(~see, -math.inf)
    att = (torch.softmax(sc, -1) @ v.repeat_interleave(g, 0)).transpose(0, 1).reshape(T, Hq * d)
    z = (x + att @ p["o"].T) @ p["head"].T
    t = torch.softmax(tlog.double() / tau, 1)
    lq = torch.log_softmax(z / tau, 1).gather(1, tids)
    loss = (tau * tau * (t * (t.log() - lq)).sum(1))[ok].sum() / int(ok.sum())
    loss.backward()
    return float(loss.detach()), z.detach(), {n: x.grad for n, x in p.items()}, int(ok.sum())


@pytest.mark.parametrize("Hq,Hkv,d,window,sinks,tau", [(2, 2, 64, 50, 3, 1.0), (4, 1, 128, 130, 140, 2.0)])
def test_packed_distillation_step(va, Hq, Hkv, d, window, sinks, tau):
    lengths, V, D, K = [300, 1, 17, 129, 65], 500, 96, 8
    T, scale = sum(lengths), 1.25
    w = weights(V, D, Hq, Hkv, d, 10 * Hq + d)
    g = torch.Generator().manual_seed(5)
    ids = torch.randint(0, V, (T,), generator=g)
    tids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)])
    tlog = 2 * torch.randn(T, K, generator=g)
    rl, rz, rg, n = reference(w, ids, lengths, tids, tlog, tau, window, sinks, scale, Hq, Hkv, d)

    p = {k: x.to(DEV).requires_grad_(True) for k, x in w.items()}
    idd = ids.to(DEV, torch.int32)
    cu, _, _, mx, st = va.build_metadata(torch.tensor(lengths, dtype=torch.int32, device=DEV), T_capacity=T)
    cu = cu[:len(lengths) + 1]
    x = va.embed(p["table"], idd, scale)
    q, k, v = ((x @ p[m].T).view(T, H, d) for m, H in (("q", Hq), ("k", Hkv), ("v", Hkv)))
    att = va.varlen_attn(q, k, v, cu, int(mx.item()), window=window, sinks=sinks)
    z = (x + att.reshape(T, Hq * d) @ p["o"].T) @ p["head"].T
    loss, count, gz = va.token_distill(z.detach(), tids.to(DEV, torch.int32), tlog.to(DEV), va.loss_targets(idd, cu),
                                       temperature=tau, check_status=True)
    z.backward(gz)

    # Every stage rounds to bf16 once (a relative 2^-8 at most): x, q / k / v, P, the attention's
    # output, its projection, the residual sum and the logits on the way there; the logits' error is
    # at most their sum over the path, 7 * 2^-8 of the norms involved.
    step = 2.0 ** -8
    assert int(count.item()) == n
    zd = z.detach().double().cpu()
    assert float((zd - rz).norm() / rz.norm()) <= 7 * step
    # the loss moves by at most twice the largest change of a logit over tau, times tau^2
    assert abs(float(loss[1]) - rl) <= 2 * tau * float((zd - rz).abs().max()) + 1e-5
    # and back: the logits' gradient (with the forward's error), its two products, dO, D, dS, dQ / dK /
    # dV, their products and the sum over a row's paths: 9 more
    for name, ref in rg.items():
        got = p[name].grad.double().cpu()
        assert float((got - ref).norm() / ref.norm()) <= 16 * step, name
    assert torch.equal(p["table"].grad.cpu()[rg["table"].abs().sum(1) == 0],
                       torch.zeros_like(p["table"].grad.cpu()[rg["table"].abs().sum(1) == 0]))


def test_two_streams_at_once(va):
    """Two steps on two streams with their own workspaces, interleaved: the results of each alone."""
    lengths = torch.tensor([700, 33, 512, 1], dtype=torch.int32, device=DEV)
    T, H, d, V, K = 1246, 8, 64, 4000, 12
    cu, _, _, _, _ = va.build_metadata(lengths, T_capacity=T)
    cu = cu[:5]
    sets = []
    for seed in (1, 2):
        g = torch.Generator(DEV).manual_seed(seed)
        sets.append(dict(q=torch.randn(T, H, d, device=DEV, generator=g).to(BF), do=torch.randn(T, H, d, device=DEV, generator=g).to(BF),
                         z=torch.randn(T, V, device=DEV, generator=g).to(BF),
                         ids=torch.randint(0, V, (T, K), device=DEV, generator=g, dtype=torch.int32),
                         a=torch.randn(T, K, device=DEV, generator=g), rows=torch.randn(T, 256, device=DEV, generator=g).to(BF),
                         tok=torch.randint(0, V, (T,), device=DEV, generator=g, dtype=torch.int32)))

    def step(s):
        o, lse = va.varlen_attn_fwd(s["q"], s["q"], s["q"], cu, 700, window=100, sinks=5)
        return (o, lse) + va.varlen_attn_bwd(s["q"], s["q"], s["q"], o, lse, s["do"], cu, 700, window=100, sinks=5) + \
            va.token_distill(s["z"], s["ids"], s["a"]) + (va.embed_bwd(s["rows"], s["tok"], V), va.embed_fwd(s["rows"], s["tok"] % T))

    alone = [step(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(step(s))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_calls_that_share_a_workspace(va):
    """Three captured calls on one workspace, replayed in turn on one stream: each starts from a
    workspace that another one has written, and gives what a call with its own gives."""
    torch.manual_seed(4)
    lengths = [200, 30, 150]
    T, V, K = sum(lengths), 900, 8
    cu = torch.tensor([0, 200, 230, 380], dtype=torch.int32, device=DEV)
    ids = torch.randint(0, V, (T,), dtype=torch.int32, device=DEV)
    z, a = torch.randn(T, V, device=DEV).to(torch.bfloat16), torch.randn(T, K, device=DEV)
    tid = torch.randint(0, V, (T, K), dtype=torch.int32, device=DEV)
    q, k, v, o, do = (torch.randn(T, 2, 64, device=DEV).to(torch.bfloat16) for _ in range(5))
    x = torch.randn(T, 64, device=DEV).to(torch.bfloat16)
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)

    def attend(ws=None):
        o, lse = va.varlen_attn_fwd(q, k, v, cu, 200, window=40, sinks=3, workspace=ws)
        return (o, lse) + va.varlen_attn_bwd(q, k, v, o, lse, do, cu, 200, window=40, sinks=3, workspace=ws)

    calls = [attend, lambda ws=None: va.token_distill(z, tid, a, workspace=ws),
             lambda ws=None: (va.embed_bwd(x, ids, V, 2.0, workspace=ws),)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for c in calls:
            c(ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=st):
            outs.append(c(ws))
    for order in ((0, 1, 2), (2, 0, 1), (1, 2, 0)):
        for t in (q, k, v, do, z, a, x):
            t.copy_(torch.randn_like(t))
        ids.copy_(torch.randint_like(ids, V))
        with torch.cuda.stream(st):
            st.wait_stream(torch.cuda.default_stream())
            for i in order:
                graphs[i].replay()
        torch.cuda.synchronize()
        for c, out in zip(calls, outs):
            for got, want in zip(out, c()):
                assert torch.equal(got, want)
