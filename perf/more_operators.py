"""Cases of the operators around a packed decoder step: per-head norms of queries and keys with the
position rotation, the gated linear recurrence over packed documents, and log probabilities of given
tokens with entropy and top alternatives.

Each case runs one operator once.  ``own`` false: the operator in its plain form, elementary torch
operations in 32 bits (64 for angles and long sums), rounded once at the end.  ``own`` true: the
calls a training or scoring program makes of this package.

Operators (``"op"`` of a case):

``qk``        q [T, Hq, d], k [T, Hkv, d].  u = x / sqrt(mean(x^2) + eps) * weight over every head, then its
              first ``rot`` dims turned by position * inv_freq, in pairs (i, i + rot / 2) or, with
              ``interleaved``, (2 i, 2 i + 1).  Returns both, and with ``train`` dq, dk and the two weights'
              gradients.
``scan``      h_t = exp(g_t) h_(t-1) + x_t over x, g [T, D], restarted at every document from h0 (zero
              without ``state``).  Returns h (in the wider type of x and g) and with ``state`` the last h of
              every document; with ``train`` dx, dg (and dh0).
``logprobs``  logits z [T, V], one token a row, p = softmax(z / temperature): ln p[token], the entropy,
              the log-sum-exp, the ``k`` largest logits' ids (ties: the lower id) and their ln p; rows
              without a token are zero (ids -1).  With ``train`` also the logits' gradient for given
              gradients of ln p[token] and of the entropy.
"""
import math
import random

import numpy as np
import torch

own = False

IGNORE = -100
DEV = "cuda"


# ----------------------------------------------------------------- cases

def listed():
    return [
        # three short documents: a few microseconds of work, so launches count
        dict(name="qk three documents", op="qk", docs="list:300,17,129", Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", base=1e4, far=0, train=True),
        # a decoding step of 64 sequences, each far into its context
        dict(name="qk single tokens", op="qk", docs="uniform:64:1:1:0", Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", base=5e5, far=1000000, train=False),
        # a packed fine-tuning row
        dict(name="qk sft row", op="qk", docs="uniform:8192:32:2048:1", Hq=32, Hkv=32, d=128, rot=128, interleaved=False,
             dtype="bf16", base=1e4, far=0, train=True),
        # small heads, an odd length, half of a head turned, neighbouring pairs
        dict(name="qk odd d64", op="qk", docs="uniform:5003:1:700:3", Hq=8, Hkv=2, d=64, rot=32, interleaved=True,
             dtype="bf16", base=1e4, far=0, train=True),
        # one pass over long documents without gradients (evaluation, prefill)
        dict(name="qk long prefill", op="qk", docs="list:32768,16384,8192,4096,2048,1024,512,512", Hq=32, Hkv=8, d=128,
             rot=128, interleaved=False, dtype="bf16", base=5e5, far=0, train=False),
        # a decoding step of 256 sequences: every state moves on by one token
        dict(name="scan single tokens", op="scan", docs="uniform:256:1:1:0", D=4096, dtype="bf16", gate="fp32", state=True,
             train=False),
        # a packed fine-tuning row, all in bf16
        dict(name="scan sft row", op="scan", docs="uniform:8192:32:2048:1", D=4096, dtype="bf16", gate="bf16", state=False,
             train=True),
        # long-context training: one document is half of the stream; decays held in fp32
        dict(name="scan long", op="scan", docs="list:32768,16384,8192,4096,2048,1024,512,512", D=2048, dtype="bf16",
             gate="fp32", state=False, train=True),
        # the last positions of a few sequences: latency, 20 alternatives a token
        dict(name="logprobs 64 rows", op="logprobs", T=64, V=32000, k=20, dtype="bf16", temperature=1.0, train=False),
        # the fine-tuning row in a policy-gradient step
        dict(name="logprobs sft row", op="logprobs", T=8192, V=32768, k=5, dtype="bf16", temperature=1.0, train=True),
        # fp32 logits whose odd vocabulary leaves rows unaligned
        dict(name="logprobs odd fp32", op="logprobs", T=2047, V=50003, k=8, dtype="fp32", temperature=0.7, train=True),
        # a large vocabulary and a 16384 bin: offsets pass 2^31 elements
        dict(name="logprobs large", op="logprobs", T=16384, V=131072, k=1, dtype="bf16", temperature=1.0, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _docs(rng, T):
    kind = rng.choice(["uniform", "uniform", "lognormal", "one"])
    if kind == "one":
        return "list:%d" % T
    hi = _log(rng, 1, T)
    if kind == "uniform":
        return "uniform:%d:%d:%d:%d" % (T, rng.randint(1, hi), hi, rng.randrange(1000))
    return "lognormal:%d:%d:%d" % (T, max(16, hi // 8), rng.randrange(1000))


def draw(rng):
    op = rng.choice(["qk", "scan", "logprobs"])
    if op == "qk":
        Hq, Hkv = rng.choice([(32, 8), (32, 32), (16, 16), (8, 2), (12, 1), (7, 7)])
        d = rng.choice([64, 128, 128, 80, 96, 256])
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        T = _log(rng, 1, min(65536, (1 << 28) // ((Hq + Hkv) * d * (1 if dtype == "bf16" else 2))))
        return dict(op=op, docs=_docs(rng, T), Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2, 16]),
                    interleaved=rng.random() < 0.3, dtype=dtype, base=rng.choice([1e4, 5e5, 1e6]),
                    far=rng.choice([0, 0, 100000, 1000000]), train=rng.random() < 0.6)
    if op == "scan":
        dtype, gate = rng.choice([("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
        D = rng.choice([_log(rng, 1, 8192), 8 * _log(rng, 1, 1024)])
        T = _log(rng, 1, min(131072, (1 << (27 if gate == "bf16" else 26)) // D))
        train, state = rng.random() < 0.7, rng.random() < 0.4
        docs = "uniform:%d:1:1:0" % T if rng.random() < 0.15 else _docs(rng, T)
        return dict(op=op, docs=docs, D=D, dtype=dtype, gate=gate, state=state, train=train)
    V = _log(rng, 100, 131072)
    T = _log(rng, 1, min(16384, (1 << 30) // V))
    return dict(op=op, T=T, V=V, k=rng.choice([0, 1, 5, _log(rng, 1, 64)]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                temperature=rng.choice([0.7, 1.0, 1.0, 1.5]), train=rng.random() < 0.7)


def _lengths(case):
    """Document lengths (from the case alone)."""
    kind, *a = case["docs"].split(":")
    if kind == "list":
        return [int(x) for x in a[0].split(",")]
    T, a = int(a[0]), [int(x) for x in a[1:]]
    rng = random.Random(a[-1])
    out, left = [], T
    while left > 0:                      # the last document takes what is left of the row
        n = rng.randint(a[0], a[1]) if kind == "uniform" else max(16, int(rng.lognormvariate(math.log(a[0]), 1.0)))
        out.append(min(n, left))
        left -= out[-1]
    return out


def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    es = _size(case["dtype"])
    if case["op"] == "qk":
        n = sum(_lengths(case)) * (case["Hq"] + case["Hkv"]) * case["d"]
        # q, k in and out; with their gradients dout in and dq, dk out as well
        return {"bytes": float(n * es * (4 if case["train"] else 2) + 4 * sum(_lengths(case))),
                "flops": float(n) * (24 if case["train"] else 8)}
    if case["op"] == "scan":
        lens = _lengths(case)
        n, gs = sum(lens) * case["D"], _size(case["gate"])
        states = len(lens) * case["D"] * 4 if case["state"] else 0
        # x, g in, h out; dh in, dx, dg out; the states in and out and their gradients
        move = n * (es + gs + max(es, gs)) + 2 * states
        if case["train"]:
            move *= 2
        return {"bytes": float(move), "flops": float(n) * (8 if case["train"] else 3)}
    T, V = case["T"], case["V"]
    return {"bytes": float(T * V * es * (2 if case["train"] else 1) + T * (16 + 8 * case["k"])),
            "flops": float(T) * V * (12 if case["train"] else 5)}


# ----------------------------------------------------------------- inputs

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _wide(case):
    return _dtype("fp32" if "fp32" in (case["dtype"], case["gate"]) else "bf16")


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(int(seed))
    st, dt = dict(case), _dtype(case["dtype"])
    randn = lambda *s: torch.randn(*s, device=DEV, generator=g)                      # noqa: E731
    if case["op"] != "logprobs":
        lens = _lengths(case)
        T = sum(lens)
        st["cu"] = torch.from_numpy(np.cumsum([0] + lens).astype(np.int32)).to(DEV)
    if case["op"] == "qk":
        Hq, Hkv, d, rot = case["Hq"], case["Hkv"], case["d"], case["rot"]
        # a projection's output: queries, keys and values of a token side by side, their size differs by head
        qkv = (randn(T, Hq + 2 * Hkv, d) * torch.exp(0.5 * randn(Hq + 2 * Hkv, 1))).to(dt)
        st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        st["qw"], st["kw"] = ((1.0 + 0.2 * randn(d)).to(dt) for _ in range(2))
        st["inv_freq"] = (case["base"] ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)).float()
        pos = np.concatenate([np.arange(n) for n in lens])
        start = torch.randint(0, case["far"] + 1, (len(lens),), device=DEV, generator=g)
        seg = torch.from_numpy(np.repeat(np.arange(len(lens)), lens)).to(DEV)
        st["pos"] = (torch.from_numpy(pos).to(DEV) + start[seg]).to(torch.int32)
        if case["train"]:
            st["dq"], st["dk"] = randn(T, Hq, d).to(dt), randn(T, Hkv, d).to(dt)
    elif case["op"] == "scan":
        D = case["D"]
        # every channel forgets at a rate of its own, a token's gate moves it
        rate = torch.exp(torch.rand(D, device=DEV, generator=g) * math.log(1000.0)) * 1e-3
        st["g"] = (-rate * torch.sigmoid(randn(T, D))).to(_dtype(case["gate"]))
        st["x"] = (randn(T, D) * torch.sqrt(-torch.expm1(2 * st["g"].float()))).to(dt)
        st["h0"] = randn(len(lens), D) if case["state"] else None
        if case["train"]:
            st["dh"] = randn(T, D).to(_wide(case))
            st["dlast"] = randn(len(lens), D) if case["state"] else None
    else:
        T, V = case["T"], case["V"]
        # one likely token a row; the given token is that one as often as not
        like = torch.randint(0, V, (T, 1), device=DEV, generator=g)
        z = torch.empty(T, V, device=DEV, dtype=dt)
        rows = max(1, (1 << 28) // V)
        for r in range(0, T, rows):                     # in pieces: the fp32 draws would not be small
            z[r:r + rows] = 2.0 * randn(min(rows, T - r), V)
        z.scatter_(1, like, (12.0 + 2.0 * randn(T, 1)).to(dt))
        st["z"] = z
        other = torch.randint(0, V, (T,), device=DEV, generator=g)
        tok = torch.where(torch.rand(T, device=DEV, generator=g) < 0.5, like[:, 0], other)
        drop = torch.rand(T, device=DEV, generator=g) < 0.1            # prompts, document ends
        drop[0] = False
        st["tok"] = torch.where(drop, IGNORE, tok).to(torch.int32)
        if case["train"]:                               # advantages, and a small bonus for entropy
            st["dlp"], st["dent"] = randn(T) / T, -0.01 * torch.rand(T, device=DEV, generator=g) / T
    if own:
        import packed_sequence_varlen_gb300 as va
        st["va"] = va
    return st


# ----------------------------------------------------------------- one pass

def run(st):
    if st["op"] == "qk":
        return _own_qk(st) if own else _plain_qk(st)
    if st["op"] == "scan":
        return _own_scan(st) if own else _plain_scan(st)
    return _own_logprobs(st) if own else _plain_logprobs(st)


EPS = 1e-6


def _own_qk(st):
    va, a = st["va"], (st["pos"], st["qw"], st["kw"], st["inv_freq"])
    qo, ko = va.qk_norm_rope_fwd(st["q"], st["k"], *a, eps=EPS, interleaved=st["interleaved"])
    if not st["train"]:
        return qo, ko
    return (qo, ko) + tuple(va.qk_norm_rope_bwd(st["dq"], st["dk"], st["q"], st["k"], *a, eps=EPS,
                                                interleaved=st["interleaved"]))


def _own_scan(st):
    va = st["va"]
    h, last = va.varlen_scan_fwd(st["x"], st["g"], st["cu"], h0=st["h0"], h_last=st["state"])
    got = [h, last] if st["state"] else [h]
    if st["train"]:
        dx, dg, dh0 = va.varlen_scan_bwd(st["dh"], h, st["g"], st["cu"], h0=st["h0"], dh_last=st["dlast"],
                                         x_dtype=st["x"].dtype)
        got += [dx, dg, dh0] if st["state"] else [dx, dg]
    return got


def _own_logprobs(st):
    va = st["va"]
    lp, ent, lse, ids, top = va.token_logprobs_fwd(st["z"], st["tok"], top_k=st["k"], temperature=st["temperature"])
    got = [lp, ent, lse] + ([ids, top] if st["k"] else [])
    if st["train"]:
        got.append(va.token_logprobs_bwd(st["z"], st["tok"], lse, ent, st["dlp"], st["dent"],
                                         temperature=st["temperature"]))
    return got


def _turn(x, cos, sin, rot, interleaved):
    """The first ``rot`` of the last dim turned: (a, b) -> (a cos - b sin, b cos + a sin)."""
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    p, q = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = p, q
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = p, q
    return y


def _plain_qk(st):
    angle = st["pos"].double()[:, None, None] * st["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    got, grads, weights = [], [], []
    for x, w, dy in ((st["q"], st["qw"], st.get("dq")), (st["k"], st["kw"], st.get("dk"))):
        xf, wf = x.float(), w.float()
        r = (xf.square().mean(-1, keepdim=True) + EPS).rsqrt()
        n = xf * r
        got.append(_turn(n * wf, cos, sin, st["rot"], st["interleaved"]).to(x.dtype))
        if dy is not None:
            u = _turn(dy.float(), cos, -sin, st["rot"], st["interleaved"])
            weights.append((u * n).sum(1).double().sum(0).to(w.dtype))
            u *= wf
            grads.append((r * (u - n * (u * n).mean(-1, keepdim=True))).to(x.dtype))
    return got + grads + weights


def _blocks(x, C, fill=0.0):
    """[T, D] as [T / C, C, D], the last block filled up."""
    return torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % C), value=fill).view(-1, C, x.shape[1])


def _recur(a, x, carry):
    """h_t = a_t h_(t-1) + x_t over the first dim (``carry`` 0: nothing is carried into row t), block by
    block: all blocks together from zero, then their ends in turn.  In 64 bits: a decay near 1 sums
    over thousands of rows, and what rounding it to 32 bits loses adds up."""
    T, D = x.shape
    C = max(1, int(math.sqrt(T)))
    a = torch.where(carry[:, None], a, 0.0)
    A, X = _blocks(a, C), _blocks(x, C)
    H, P = torch.empty_like(X), torch.empty_like(X)
    H[:, 0], P[:, 0] = X[:, 0], A[:, 0]
    for t in range(1, C):
        torch.addcmul(X[:, t], A[:, t], H[:, t - 1], out=H[:, t])
        torch.mul(A[:, t], P[:, t - 1], out=P[:, t])
    end = torch.zeros(X.shape[0] + 1, D, device=x.device, dtype=x.dtype)
    for b in range(X.shape[0]):
        torch.addcmul(H[b, -1], P[b, -1], end[b], out=end[b + 1])
    return torch.addcmul(H, P, end[:-1, None]).view(-1, D)[:T]


def _plain_scan(st):
    cu = st["cu"].long()
    first, final = cu[:-1], cu[1:] - 1
    a, x = st["g"].double().exp(), st["x"].double()
    inner = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    inner[first] = False                                     # rows that carry their document's last h
    if st["state"]:
        x = x.index_add(0, first, a[first] * st["h0"].double())
    h = _recur(a, x, inner)
    got = [h.to(_wide(st))] + ([h[final].float()] if st["state"] else [])
    if not st["train"]:
        return got
    d = st["dh"].double()
    if st["state"]:
        d = d.index_add(0, final, st["dlast"].double())
    # e_t = dh_t + a_(t+1) e_(t+1): the same recurrence from behind, with the next row's decay
    later = torch.cat([a[1:], a[:1]]).flip(0)
    e = _recur(later, d.flip(0), torch.cat([inner[1:], inner[:1]]).flip(0)).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = st["h0"].double() if st["state"] else 0.0
    got += [e.to(st["x"].dtype), (e * a * before).to(st["g"].dtype)]
    return got + ([(a[first] * e[first]).float()] if st["state"] else [])


def _plain_logprobs(st):
    t, (T, V), k = st["temperature"], st["z"].shape, st["k"]
    ok = st["tok"] != IGNORE
    idx = st["tok"].clamp(min=0).long()[:, None]
    lp, ent, lse = (torch.empty(T, device=DEV) for _ in range(3))
    ids = torch.empty(T, k, device=DEV, dtype=torch.int32)
    top = torch.empty(T, k, device=DEV)
    grad = torch.empty_like(st["z"]) if st["train"] else None
    rank = (V - 1) - torch.arange(V, device=DEV)
    rows = max(1, (1 << 27) // V)
    for r in range(0, T, rows):
        s = slice(r, min(T, r + rows))
        z = st["z"][s].float() / t
        m = z.amax(1, keepdim=True)
        e = (z - m).exp()
        tot = e.sum(1, keepdim=True)
        ls = tot.log()
        x = z.sub(m).sub_(ls)                                # ln p
        p = e.div_(tot)
        H = -(p * x).sum(1, keepdim=True)
        o = ok[s, None]
        put = lambda to, v: to[s].copy_(torch.where(o, v, 0.0).view(to[s].shape))    # noqa: E731
        put(lp, x.gather(1, idx[s])), put(ent, H), put(lse, m + ls)
        if k:
            # one whole number a logit, ordered as the logits are and equal ones by their id
            i = (st["z"][s].float() + 0.0).view(torch.int32)
            key = torch.where(i < 0, i ^ 0x7fffffff, i).long() * (1 << 32) + rank
            j = (V - 1) - (key.topk(k, 1).values & 0xffffffff)
            ids[s] = torch.where(o, j, -1).to(torch.int32)
            put(top, x.gather(1, j))
        if grad is not None:
            dl, dh = (torch.where(ok[s], st[n][s], 0.0)[:, None] / t for n in ("dlp", "dent"))
            x.add_(H).mul_(dh).add_(dl).mul_(p).neg_()       # -p (dH (ln p + H) + dlp)
            grad[s] = torch.where(o, x.scatter_add_(1, idx[s], dl), 0.0).to(grad.dtype)
    return [lp, ent, lse] + ([ids, top] if k else []) + ([grad] if grad is not None else [])


# ----------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(st)
    if case["op"] == "scan":
        return _exact_scan(st)
    return _exact_logprobs(st)


def _exact_qk(st):
    """The turn as a product of complex numbers, the norm's gradient by its matrix."""
    rot, d = st["rot"], st["d"]
    phase = st["pos"].double()[:, None, None] * st["inv_freq"].double()
    z = torch.polar(torch.ones_like(phase), phase)
    at = torch.arange(rot, device=DEV)
    at = at.view(-1, 2) if st["interleaved"] else at.view(2, -1).T            # the pairs' dims

    def turn(x, z):
        y = x.clone()
        c = torch.complex(x[..., at[:, 0]], x[..., at[:, 1]]) * z
        y[..., at[:, 0]], y[..., at[:, 1]] = c.real, c.imag
        return y

    got, grads, weights = [], [], []
    for x, w, dy in ((st["q"], st["qw"], st.get("dq")), (st["k"], st["kw"], st.get("dk"))):
        x, w, T = x.double(), w.double(), x.shape[0]
        out, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(w)
        for r in range(0, T, 8192):
            s = slice(r, r + 8192)
            v = ((x[s] * x[s]).sum(-1, keepdim=True) / d + EPS)
            out[s] = turn(x[s] / v.sqrt() * w, z[s])
            if dy is not None:
                u = turn(dy[s].double(), z[s].conj())
                dw += (u * x[s] / v.sqrt()).sum((0, 1))
                # d(x_i v^-1/2) / dx_j = v^-1/2 [i == j] - v^-3/2 x_i x_j / d
                dx[s] = u * w / v.sqrt() - x[s] * ((u * w * x[s]).sum(-1, keepdim=True) / (d * v * v.sqrt()))
        got.append(out)
        if dy is not None:
            grads.append(dx), weights.append(dw)
    return got + grads + weights


def _exact_scan(st):
    """By doubling: after s steps row t holds the sum over its last 2^s rows of its document."""
    cu = st["cu"].long()
    T = st["x"].shape[0]
    first, final = cu[:-1], cu[1:] - 1
    decay = torch.exp(st["g"].double())

    def doubling(A, H):
        s = 1
        while s < T:
            H[s:] += A[s:] * H[:-s].clone()
            A[s:] = A[s:] * A[:-s].clone()
            A[:s] = 0
            s *= 2
        return H

    A, H = decay.clone(), st["x"].double()
    if st["state"]:
        H[first] += A[first] * st["h0"].double()
    A[first] = 0
    h = doubling(A, H)
    got = [h.clone() if st["train"] else h] + ([h[final]] if st["state"] else [])
    if not st["train"]:
        return got
    A, H = torch.zeros_like(decay), st["dh"].double()
    A[:-1] = decay[1:]
    A[final] = 0
    if st["state"]:
        H[final] += st["dlast"].double()
    e = doubling(A.flip(0), H.flip(0)).flip(0)
    h[1:] = h[:-1].clone()
    h[first] = st["h0"].double() if st["state"] else 0.0
    got += [e, e * decay * h]
    return got + ([(decay * e)[first]] if st["state"] else [])


def _exact_logprobs(st):
    t, (T, V), k = st["temperature"], st["z"].shape, st["k"]
    keep = torch.nonzero(st["tok"] != IGNORE)[:, 0]
    lp, ent, lse = (torch.zeros(T, device=DEV, dtype=torch.float64) for _ in range(3))
    top = torch.zeros(T, k, device=DEV, dtype=torch.float64)
    # beyond 2^28 values the 64-bit gradient is handed over in 32 bits
    grad = torch.zeros(T, V, device=DEV, dtype=torch.float64 if T * V <= 1 << 28 else torch.float32) if st["train"] else None
    rows = max(1, (1 << 26) // V)
    for r in range(0, len(keep), rows):
        s = keep[r:r + rows]
        lq = torch.log_softmax(st["z"][s].double() / t, 1)
        q, at = lq.exp(), torch.arange(len(s), device=DEV)
        tok = st["tok"][s].long()
        H = -torch.xlogy(q, q).sum(1)
        lp[s], ent[s], lse[s] = lq[at, tok], H, torch.logsumexp(st["z"][s].double() / t, 1)
        if k:
            top[s] = lq.topk(k, 1).values                     # equal logits have equal values
        if grad is not None:
            dl, dh = st["dlp"][s].double()[:, None], st["dent"][s].double()[:, None]
            gz = -dl * q - dh * q * (lq + H[:, None])
            gz[at, tok] += dl[:, 0]
            grad[s] = (gz / t).to(grad.dtype)
    return [lp, ent, lse] + ([None, top] if k else []) + ([grad] if grad is not None else [])
