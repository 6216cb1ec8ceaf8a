"""One packed policy-gradient step of a hybrid decoder through the operators together: metadata, embedding, query /
key norm with rotation, attention, the gated recurrence over the same boundaries, log probabilities of the next
tokens with an entropy bonus, and back, against the same chain in float64 torch with a dense mask."""
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
    mk = lambda *s: torch.randn(*s, generator=g)                             # noqa: E731
    w = dict(table=mk(V, D), qkv=mk((Hq + 2 * Hkv) * d, D) / math.sqrt(D), qw=1 + 0.2 * mk(d), kw=1 + 0.2 * mk(d),
             o=mk(D, Hq * d) / math.sqrt(Hq * d), u=mk(D, D) / math.sqrt(D), gate=mk(D, D) / math.sqrt(D),
             r=mk(D, D) / math.sqrt(D), head=mk(V, D) / math.sqrt(D))
    return {n: x.to(BF) for n, x in w.items()}


def turn(x, pos, inv):
    f = pos[:, None, None].to(x.dtype) * inv.to(x.dtype)
    a, b = x[..., :len(inv)], x[..., len(inv):]
    return torch.cat([a * f.cos() - b * f.sin(), b * f.cos() + a * f.sin()], -1)


def reference(w, ids, lengths, inv, adv, bonus, Hq, Hkv, d):
    p = {n: x.double().requires_grad_(True) for n, x in w.items()}
    T = len(ids)
    x = p["table"][ids]
    qkv = (x @ p["qkv"].T).view(T, Hq + 2 * Hkv, d)
    pos = torch.cat([torch.arange(n) for n in lengths])
    norm = lambda y, wt: y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * wt   # noqa: E731
    q, k = turn(norm(qkv[:, :Hq], p["qw"]), pos, inv), turn(norm(qkv[:, Hq:Hq + Hkv], p["kw"]), pos, inv)
    see, on, targets, s = torch.zeros(T, T, dtype=torch.bool), torch.ones(T, dtype=torch.bool), ids.roll(-1), 0
    for n in lengths:
        see[s:s + n, s:s + n] = torch.ones(n, n, dtype=torch.bool).tril()
        on[s + n - 1] = False
        s += n
    g = Hq // Hkv
    sc = (q.transpose(0, 1) @ k.transpose(0, 1).repeat_interleave(g, 0).transpose(1, 2) / math.sqrt(d)).masked_fill(~see, -math.inf)
    att = (torch.softmax(sc, -1) @ qkv[:, Hq + Hkv:].transpose(0, 1).repeat_interleave(g, 0)).transpose(0, 1).reshape(T, -1)
    x = x + att @ p["o"].T
    u, ld = x @ p["u"].T, -torch.nn.functional.softplus(x @ p["gate"].T)
    rows, s = [], 0
    for n in lengths:
        h = torch.zeros(x.shape[1], dtype=torch.float64)
        for t in range(s, s + n):
            h = ld[t].exp() * h + u[t]
            rows.append(h)
        s += n
    z = (x + torch.stack(rows) @ p["r"].T) @ p["head"].T
    lq = torch.log_softmax(z, 1)
    lp, ent = lq.gather(1, targets[:, None])[:, 0], -(lq.exp() * lq).sum(1)
    loss = -(adv.double() * lp + bonus * ent)[on].sum() / int(on.sum())
    loss.backward()
    return float(loss.detach()), z.detach(), {n: y.grad for n, y in p.items()}, lp.detach(), on


@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 64), (4, 1, 128)])
def test_packed_policy_step(va, Hq, Hkv, d):
    lengths, V, D, bonus = [150, 1, 17, 129, 40], 500, 96, 0.1
    T = sum(lengths)
    w = weights(V, D, Hq, Hkv, d, 10 * Hq + d)
    g = torch.Generator().manual_seed(5)
    ids, adv = torch.randint(0, V, (T,), generator=g), torch.randn(T, generator=g)
    inv = (1e4 ** (-torch.arange(0, d, 2).double() / d)).float()
    rl, rz, rg, rlp, on = reference(w, ids, lengths, inv, adv, bonus, Hq, Hkv, d)

    p = {n: x.to(DEV).requires_grad_(True) for n, x in w.items()}
    idd = ids.to(DEV, torch.int32)
    cu, pos, _, mx, _ = va.build_metadata(torch.tensor(lengths, dtype=torch.int32, device=DEV), T_capacity=T)
    cu = cu[:len(lengths) + 1]
    x = va.embed(p["table"], idd)
    qkv = (x @ p["qkv"].T).view(T, Hq + 2 * Hkv, d)
    q, k = va.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], pos, p["qw"], p["kw"], inv.to(DEV))
    att = va.varlen_attn(q, k, qkv[:, Hq + Hkv:].contiguous(), cu, int(mx.item()))
    x = x + att.reshape(T, Hq * d) @ p["o"].T
    h, last = va.varlen_scan(x @ p["u"].T, -torch.nn.functional.softplus(x @ p["gate"].T), cu)
    z = (x + h @ p["r"].T) @ p["head"].T
    targets = va.loss_targets(idd, cu)
    lp, ent, top, _ = va.token_logprobs(z, targets, top_k=3)
    n = int((targets != va.IGNORE_INDEX).sum())
    loss = -(adv.to(DEV) * lp + bonus * ent).sum() / n
    loss.backward()

    # Every stage rounds to bf16 once (a relative 2^-8 at most): x, q / k / v, the norm, P, the attention's output, its
    # projection, the sum, u, the gate and its softplus (whose relative error is that of the decay's memory), h, its
    # projection, the sum and the logits: the logits' error is at most their sum over the path, 14 * 2^-8 of the norms.
    step = 2.0 ** -8
    zd = z.detach().double().cpu()
    assert n == int(on.sum())
    assert float((zd - rz).norm() / rz.norm()) <= 14 * step
    # a log probability moves by at most twice the largest change of a logit
    assert float((lp.detach().cpu().double() - rlp)[on].abs().max()) <= 2 * float((zd - rz).abs().max()) + 1e-5
    assert torch.equal(top.cpu()[on].long(), (z.detach().float().cpu()).sort(dim=1, descending=True, stable=True).indices[on][:, :3])
    # and back: the logits' gradient with the forward's error, and a rounding at each of the same stages
    for name, ref in rg.items():
        got = p[name].grad.double().cpu()
        assert float((got - ref).norm() / ref.norm()) <= 28 * step, name
    # the states that the recurrence leaves are the last rows of every document
    assert torch.equal(last.detach().to(BF).cpu(), h.detach().cpu()[torch.tensor(lengths).cumsum(0) - 1])


def test_single_token_step_follows_the_packed_one(va):
    """Norm, recurrence and scores of the next token, one token a sequence at a time, against the whole packed stream."""
    lengths, H, d, D, V = [9, 5, 12], 3, 64, 80, 700
    B, T = len(lengths), sum(lengths)
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)              # noqa: E731
    q, k, x, head = mk(T, H, d), mk(T, 1, d), mk(T, D), mk(V, D)
    ld = -torch.rand(T, D, generator=g).to(DEV)
    w, inv = mk(d), (1e4 ** (-torch.arange(0, d, 2).double() / d)).float().to(DEV)
    tok = torch.randint(0, V, (T,), generator=g).to(DEV, torch.int32)
    cu = torch.tensor([0] + lengths).cumsum(0).to(DEV, torch.int32)
    pos = torch.cat([torch.arange(n) for n in lengths]).to(DEV, torch.int32)
    qo, ko = va.qk_norm_rope_fwd(q, k, pos, w, w, inv)
    h, last = va.varlen_scan_fwd(x, ld, cu, h_last=True)
    lp, ent, lse, top, tlp = va.token_logprobs_fwd(h.to(BF) @ head.T, tok, top_k=4)
    state = torch.zeros(B, D, device=DEV)
    starts = torch.tensor([0] + lengths).cumsum(0)[:-1]
    for t in range(max(lengths)):
        live = [b for b in range(B) if t < lengths[b]]
        at = torch.tensor([int(starts[b]) + t for b in live], device=DEV)
        a, b_ = va.qk_norm_rope_fwd(q[at], k[at], torch.full((len(live),), t, dtype=torch.int32, device=DEV), w, w, inv)
        assert torch.equal(a, qo[at]) and torch.equal(b_, ko[at])
        s = state[live].contiguous()
        hs, s = va.varlen_scan_fwd(x[at], ld[at], torch.arange(len(live) + 1, dtype=torch.int32, device=DEV), s, h_last=s)
        state[live] = s
        # one decay after the other instead of a run's together: the sums' order differs, fp32 roundings of the states
        assert float((hs - h[at]).abs().max()) <= 64 * 2.0 ** -24 * float(h.abs().max()) * t + 1e-6
        again = va.token_logprobs_fwd(h[at].to(BF) @ head.T, tok[at].contiguous(), top_k=4)
        assert again[0].shape == (len(live),) and torch.equal(again[3].sort(1).values >= 0, torch.ones_like(again[3], dtype=torch.bool))
    assert float((state - last).abs().max()) <= 64 * 2.0 ** -24 * float(h.abs().max()) * max(lengths) + 1e-6


def test_single_token_scores_are_those_of_the_packed_stream(va):
    """Log probabilities, entropies and alternatives of one token a sequence at a time, from the recurrence's single-token form,
    against those of the packed stream."""
    lengths, D, V, k = [9, 5, 12, 1], 80, 700, 4
    B, T = len(lengths), sum(lengths)
    g = torch.Generator().manual_seed(2)
    x, head = (torch.randn(*s, generator=g).to(BF).to(DEV) for s in ((T, D), (V, D)))
    ld = -torch.rand(T, D, generator=g).to(DEV)
    tok = torch.randint(0, V, (T,), generator=g).to(DEV, torch.int32)
    cu = torch.tensor([0] + lengths).cumsum(0).to(DEV, torch.int32)
    h, _ = va.varlen_scan_fwd(x, ld, cu, h_last=True)
    z = h.double() @ head.double().T                          # logits of the fp32 states, rounded once
    lp, ent, lse, ids, top = va.token_logprobs_fwd(z.float(), tok, top_k=k)
    state, starts = torch.zeros(B, D, device=DEV), torch.tensor([0] + lengths).cumsum(0)[:-1]
    for t in range(max(lengths)):
        live = [b for b in range(B) if t < lengths[b]]
        at = torch.tensor([int(starts[b]) + t for b in live], device=DEV)
        hs, s = va.varlen_scan_fwd(x[at], ld[at], torch.arange(len(live) + 1, dtype=torch.int32, device=DEV), state[live].contiguous(),
                                   h_last=True)
        state[live] = s
        zs = hs.double() @ head.double().T
        one = va.token_logprobs_fwd(zs.float(), tok[at].contiguous(), top_k=k)
        # the states differ by fp32 roundings (two forms of one recurrence, as above), and the logits by what those make
        # and half a step of their own; a log probability and the lse move by at most the largest change of a logit, twice and once, an entropy
        # by it times the spread of ln p (at most lse - the smallest logit), a sum by 500 roundings of 2^-24
        off = float((zs - z[at]).abs().max()) + 2.0 ** -23 * float(z[at].abs().max())
        spread = float((lse[at, None] - z[at]).max())
        sums = 500 * 2.0 ** -24 * (1 + spread)
        assert float((hs - h[at]).abs().max()) <= 64 * 2.0 ** -24 * float(h.abs().max()) * t + 1e-6
        assert float((one[0] - lp[at]).abs().max()) <= 2 * off + sums
        assert float((one[1] - ent[at]).abs().max()) <= 2 * off * (1 + spread) + sums
        assert float((one[2] - lse[at]).abs().max()) <= off + sums
        # an alternative may change places with one whose logit is as near as that
        zi, zj = z[at].gather(1, one[3].long()), z[at].gather(1, ids[at].long())
        assert float((zi - zj).abs().max()) <= 2 * off
        assert float((one[4] - top[at]).abs().max()) <= 4 * off + sums
