"""Refusals of the query / key norm, the gated recurrence and the token log probabilities that need no GPU: the C
ABI checks its arguments before it touches the device, the Python face its tensors."""
import ctypes
import math

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = 1 << 20                                                   # an aligned address that nothing reads


@pytest.fixture(scope="module")
def va():
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    pkg._lib.load()
    return pkg


def qk_shape(va, **kw):
    s = va.VaQkShape()
    vals = dict(T=4, Hq=2, Hkv=1, d=64, rot=64, dtype=1, weight_dtype=1, interleaved=0, q_row_stride=128,
                q_head_stride=64, k_row_stride=64, k_head_stride=64, qo_row_stride=128, qo_head_stride=64,
                ko_row_stride=64, ko_head_stride=64)
    vals.update(kw)
    for n, v in vals.items():
        setattr(s, n, v)
    return s


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(T=1 << 30), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(dtype=2), INVALID),
    (dict(weight_dtype=-1), INVALID), (dict(d=60), UNSUPPORTED), (dict(d=264), UNSUPPORTED), (dict(d=0), UNSUPPORTED),
    (dict(rot=72), UNSUPPORTED), (dict(rot=4), UNSUPPORTED), (dict(rot=-8), UNSUPPORTED), (dict(q_row_stride=129), INVALID),
    (dict(k_head_stride=-64), INVALID), (dict(qo_row_stride=4), INVALID)])
def test_qk_shapes(va, change, status):
    lib, s, gs = va._lib.load(), qk_shape(va, **change), va.VaQkGradStrides(128, 64, 64, 64)
    f = lib.varlen_qk_norm_rope_fwd(P, P, P, P, P, P, ctypes.byref(s), 1e-6, P, P, None)
    b = lib.varlen_qk_norm_rope_bwd(P, P, P, P, P, P, P, P, ctypes.byref(s), ctypes.byref(gs), 1e-6, P, P, P, P, P, 1 << 30, None)
    assert f == b == status
    assert lib.varlen_last_error()


def test_qk_outputs_lie_apart(va):
    lib = va._lib.load()
    for kw in (dict(qo_head_stride=0), dict(qo_row_stride=0), dict(ko_row_stride=56)):
        s = qk_shape(va, **kw)
        assert lib.varlen_qk_norm_rope_fwd(P, P, P, P, P, P, ctypes.byref(s), 1e-6, P, P, None) == INVALID, kw
    s = qk_shape(va)
    for strides in ((0, 64, 64, 64), (128, 56, 64, 64), (128, 64, 0, 64)):
        gs = va.VaQkGradStrides(*strides)
        assert lib.varlen_qk_norm_rope_bwd(P, P, P, P, P, P, P, P, ctypes.byref(s), ctypes.byref(gs), 1e-6, P, P, P, P, P, 1 << 30,
                                           None) == INVALID, strides


def test_qk_arguments(va):
    lib, s, gs = va._lib.load(), qk_shape(va), va.VaQkGradStrides(128, 64, 64, 64)
    at = [P] * 6 + [ctypes.byref(s), 1e-6, P, P, None]
    for i, v in [(0, None), (1, None), (2, None), (5, None), (8, None), (9, None), (0, P + 8), (3, P + 1), (6, None)]:
        a = list(at)
        a[i] = v
        assert lib.varlen_qk_norm_rope_fwd(*a) == INVALID, i
    for eps in (-1e-6, float("inf"), float("nan")):
        assert lib.varlen_qk_norm_rope_fwd(*at[:7], eps, P, P, None) == INVALID
    bt = [P] * 8 + [ctypes.byref(s), ctypes.byref(gs), 1e-6, P, P, P, P, P, 1 << 30, None]
    for i, v, st in [(0, None, INVALID), (3, None, INVALID), (5, None, INVALID), (11, None, INVALID), (15, None, INVALID),
                     (15, P + 4, INVALID), (16, 100, WORKSPACE), (9, None, INVALID), (13, P + 1, INVALID)]:
        b = list(bt)
        b[i] = v
        assert lib.varlen_qk_norm_rope_bwd(*b) == st, i
    assert lib.varlen_qk_norm_rope_bwd_workspace_size(60) == 0 and lib.varlen_qk_norm_rope_bwd_workspace_size(264) == 0
    assert lib.varlen_qk_norm_rope_bwd_workspace_size(64) > 0


def scan_shape(va, **kw):
    s = va.VaScanShape()
    vals = dict(T=10, B=2, D=64, x_dtype=1, gate_dtype=1, x_row_stride=64, gate_row_stride=64, h_row_stride=64)
    vals.update(kw)
    for n, v in vals.items():
        setattr(s, n, v)
    return s


def scan_calls(va, s, ws=P, size=1 << 40, h0=None, last=None, gs=(64, 64, 64), x=P, h=P):
    lib = va._lib.load()
    g = va.VaScanGradStrides(*gs)
    return (lib.varlen_scan_fwd(x, P, P, ctypes.byref(s), h0, h, last, ws, size, None),
            lib.varlen_scan_bwd(x, h, P, P, ctypes.byref(s), ctypes.byref(g), h0, None, P, P, last, ws, size, None))


@pytest.mark.parametrize("change,status", [
    (dict(T=0), INVALID), (dict(T=1 << 30), INVALID), (dict(B=0), INVALID), (dict(B=11), INVALID), (dict(D=0), INVALID),
    (dict(D=(1 << 20) + 1, x_row_stride=1 << 21, gate_row_stride=1 << 21, h_row_stride=1 << 21), INVALID),
    (dict(x_dtype=2), INVALID), (dict(gate_dtype=-1), INVALID), (dict(x_dtype=0), UNSUPPORTED), (dict(gate_row_stride=63), INVALID),
    (dict(h_row_stride=63), INVALID)])
def test_scan_shapes(va, change, status):
    assert scan_calls(va, scan_shape(va, **change)) == (status, status)


def test_scan_arguments(va):
    s, lib = scan_shape(va), va._lib.load()
    assert scan_calls(va, s, ws=None) == (INVALID, INVALID)
    assert scan_calls(va, s, ws=P + 8) == (INVALID, INVALID)
    assert scan_calls(va, s, size=255) == (WORKSPACE, WORKSPACE)
    one = scan_shape(va, T=2)                                 # single tokens: the status word alone, or nothing
    assert scan_calls(va, one, size=255)[0] == WORKSPACE and scan_calls(va, one, ws=None, size=0)[1] == INVALID
    assert scan_calls(va, s, x=None) == (INVALID, INVALID)
    assert scan_calls(va, s, h=None) == (INVALID, INVALID)
    assert scan_calls(va, s, h=P + 1) == (INVALID, INVALID)
    assert scan_calls(va, s, h0=P + 2) == (INVALID, INVALID)
    # states over one another: the last row may be done before the first ones have been read again
    assert scan_calls(va, s, h0=P, last=P) == (INVALID, INVALID)
    assert scan_calls(va, s, h0=P, last=P + 64 * 4) == (INVALID, INVALID)
    assert scan_calls(va, scan_shape(va, x_row_stride=63))[0] == INVALID
    assert scan_calls(va, s, gs=(63, 64, 64))[1] == INVALID and scan_calls(va, s, gs=(64, 63, 64))[1] == INVALID
    assert scan_calls(va, s, gs=(64, 64, 63))[1] == INVALID
    for T, B, D in [(0, 1, 1), (1, 2, 1), (1, 0, 1), (1, 1, 0), (1 << 30, 1, 1), (1, 1, (1 << 20) + 1)]:
        assert lib.varlen_scan_workspace_size(T, B, D) == 0
    assert lib.varlen_scan_workspace_size(1, 1, 1) >= 256
    assert lib.varlen_scan_workspace_size((1 << 30) - 1, 1, 1 << 20) > 1 << 40      # sizes past 32 bits


@pytest.mark.parametrize("change,status", [
    (dict(z=None), INVALID), (dict(tok=None), INVALID), (dict(T=0), INVALID), (dict(T=1 << 30), INVALID), (dict(V=0), INVALID),
    (dict(V=1 << 30, rs=1 << 30), INVALID), (dict(dtype=2), INVALID), (dict(rs=99), INVALID), (dict(z=P + 1), INVALID),
    (dict(tau=0.0), INVALID), (dict(tau=65.0), INVALID), (dict(tau=float("nan")), INVALID), (dict(tau=-1.0), INVALID)])
def test_logprobs_arguments(va, change, status):
    a = dict(z=P, dtype=1, rs=100, tok=P, T=4, V=100, tau=1.0)
    a.update(change)
    lib = va._lib.load()
    f = lib.varlen_token_logprobs_fwd(a["z"], a["dtype"], a["rs"], a["tok"], a["T"], a["V"], 5, -100, a["tau"], P, P, P, P, P,
                                      None, None)
    b = lib.varlen_token_logprobs_bwd(a["z"], a["dtype"], a["rs"], a["tok"], P, P, P, P, a["T"], a["V"], -100, a["tau"], P,
                                      1 << 30, None)
    assert f == b == status


def test_logprobs_outputs(va):
    lib = va._lib.load()

    def fwd(k=5, V=100, lp=P, H=P, lse=P, ids=P, top=P):
        return lib.varlen_token_logprobs_fwd(P, 1, V, P, 4, V, k, -100, 1.0, lp, H, lse, ids, top, None, None)

    assert fwd(lp=None) == fwd(H=None) == fwd(lse=None) == fwd(ids=None) == fwd(top=None) == INVALID
    assert fwd(k=-1) == fwd(k=101) == INVALID and fwd(k=129, V=200) == UNSUPPORTED

    def bwd(lse=P, H=P, dl=P, dh=P, grad=P, rs=100):
        return lib.varlen_token_logprobs_bwd(P, 1, 100, P, lse, H, dl, dh, 4, 100, -100, 1.0, grad, rs, None)

    assert bwd(lse=None) == bwd(dl=None) == bwd(H=None) == bwd(grad=None) == bwd(rs=99) == bwd(grad=P + 1) == INVALID


def test_tensors_are_checked(va):
    q, pos = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        va.qk_norm_rope_fwd(q, q, pos)                        # not on a GPU
    x, cu = torch.zeros(4, 8), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        va.varlen_scan_fwd(x, x, cu)
    with pytest.raises(ValueError):
        va.varlen_scan_bwd(x, x, x, cu)
    with pytest.raises(ValueError):
        va.token_logprobs_fwd(x, pos)
    with pytest.raises(ValueError):
        va.token_logprobs_bwd(x, pos, x[:, 0], None, x[:, 0])


def test_plain_forms_agree_with_the_definitions():
    """The measured cases' plain forms and their 64-bit values, written apart, on small draws on the CPU."""
    import random

    import perf.more_operators as M
    device, M.DEV = M.DEV, "cpu"
    try:
        rng, seen = random.Random(3), {}
        while min(seen.get(op, 0) for op in ("qk", "scan", "logprobs")) < 6:
            case = M.draw(rng)
            if M.work(case)["bytes"] > 1e6:
                continue
            seen[case["op"]] = seen.get(case["op"], 0) + 1
            plain, exact = M.run(M.prepare(case, 1)), M.exact(case, 1)
            assert len(plain) == len(exact)
            for a, b in zip(plain, exact):
                if b is None:
                    continue
                assert a.shape == b.shape
                # half a step of the type at most each, and 2^-20 for what 32 bits lose on the way; a log probability
                # is a difference of numbers up to 32, whose half step in 32 bits is 2^-20, however near 0 it is itself
                half = torch.finfo(a.dtype).eps / 2
                lost = 2.0 ** -20 * math.sqrt(a.numel()) if case["op"] == "logprobs" and a.dim() < 2 or a.shape[-1:] == (case.get("k"),) else 0.0
                assert float((a.double() - b.double()).norm()) <= (half + 2.0 ** -20) * float(b.double().norm()) + lost + 1e-30, case
    finally:
        M.DEV = device


def meets(a, b):
    """Whether two lists of (first, past the last) share an element."""
    return any(x < v and u < y for x, y in a for u, v in b)


def test_qk_heads_on_one_another(va):
    """Strides that are each at least d, but let a token's heads lie on another token's, are refused; every other layout (heads
    first, tokens first, gaps that interleave) is not."""
    if torch.cuda.is_available():
        pytest.skip("calls that are not refused would launch")
    lib, d, seen = va._lib.load(), 16, set()
    for T, H in ((1, 3), (2, 2), (3, 4), (4, 3), (5, 2)):
        for rs in range(16, 97, 8):
            for hs in range(16, 97, 8):
                at = [(t * rs + h * hs, t * rs + h * hs + d) for t in range(T) for h in range(H)]
                bad = any(meets([x], at[i + 1:]) for i, x in enumerate(at))
                seen.add(bad)
                s = qk_shape(va, T=T, Hq=H, Hkv=1, d=d, rot=16, qo_row_stride=rs, qo_head_stride=hs, ko_row_stride=d)
                assert (lib.varlen_qk_norm_rope_fwd(P, P, P, P, P, P, ctypes.byref(s), 1e-6, 5 * P, 2 * P, None) == INVALID) == bad, (T, H, rs, hs)
                s, gs = qk_shape(va, T=T, Hq=1, Hkv=H, d=d, rot=16), va.VaQkGradStrides(64, 64, rs, hs)
                assert (lib.varlen_qk_norm_rope_bwd(P, P, P, P, P, P, P, P, ctypes.byref(s), ctypes.byref(gs), 1e-6, 2 * P, 3 * P, P, P,
                                                    4 * P, 1 << 30, None) == INVALID) == bad, (T, H, rs, hs)
    assert seen == {True, False}


def test_qk_outputs_over_inputs(va):
    """An output over its input has its strides."""
    lib = va._lib.load()
    for kw in (dict(qo_row_stride=256), dict(qo_head_stride=256), dict(ko_row_stride=192)):
        s = qk_shape(va, **kw)
        assert lib.varlen_qk_norm_rope_fwd(P, 2 * P, P, P, P, P, ctypes.byref(s), 1e-6, P, 2 * P, None) == INVALID, kw
    s = qk_shape(va)
    for strides in ((256, 64, 64, 64), (128, 64, 192, 64)):
        gs = va.VaQkGradStrides(*strides)
        for a, b in ((P, 2 * P), (3 * P, 4 * P)):             # over the outputs' gradients, over the inputs
            assert lib.varlen_qk_norm_rope_bwd(P, 2 * P, 3 * P, 4 * P, P, P, P, P, ctypes.byref(s), ctypes.byref(gs), 1e-6, a, b, P, P, 8 * P,
                                               1 << 30, None) == INVALID, strides


# the first row and the row stride of two arrays of T rows of D elements, in elements
SPANS = [(0, 8, 0, 8), (0, 8, 4, 8), (0, 16, 8, 16), (0, 16, 4, 16), (8, 16, 0, 16), (0, 16, 0, 8), (0, 16, 8, 32), (0, 24, 8, 16), (0, 32, 16, 16),
         (0, 8, 32, 8), (0, 8, 31, 8), (100, 8, 0, 8), (0, 16, 56, 16), (0, 16, 60, 16), (0, 16, 64, 16), (64, 16, 0, 16), (3, 16, 0, 16),
         (0, 64, 8, 16), (0, 9, 4, 18), (0, 20, 10, 40)]


@pytest.mark.parametrize("T", [1, 2, 4])
def test_outputs_on_a_part_of_the_inputs(va, T):
    """h, dx, dlog_decay and the logits' gradient: an input itself or apart from it, however the rows interleave."""
    if torch.cuda.is_available():
        pytest.skip("calls that are not refused would launch")
    lib, D, es, seen = va._lib.load(), 8, 4, set()
    far = [P + (i << 24) for i in range(8)]
    for a0, ra, b0, rb in SPANS:
        at = [[(f + t * r, f + t * r + D) for t in range(T)] for f, r in ((a0, ra), (b0, rb))]
        same = a0 == b0 and (T == 1 or ra == rb)
        meet = meets(*at)
        seen.add((same, meet))
        a, b = far[0] + a0 * es, far[0] + b0 * es
        both = dict(T=T, B=1, D=D, x_dtype=0, gate_dtype=0)
        status = []
        for x, rx, g, rg in ((b, rb, far[1], 64), (far[1], 64, b, rb)):                 # h on x, h on the decays
            s = scan_shape(va, x_row_stride=rx, gate_row_stride=rg, h_row_stride=ra, **both)
            status.append(lib.varlen_scan_fwd(x, g, P, ctypes.byref(s), None, a, None, far[2], 1 << 40, None))
        for dh, g, dx, dg in ((b, far[1], a, far[2]), (far[1], b, far[2], a), (far[1], b, a, far[2]), (b, far[1], far[2], a)):
            s = scan_shape(va, gate_row_stride=rb if g == b else 64, h_row_stride=64, x_row_stride=64, **both)
            gs = va.VaScanGradStrides(rb if dh == b else 64, ra if dx == a else 64, ra if dg == a else 64)
            status.append(lib.varlen_scan_bwd(dh, far[3], g, P, ctypes.byref(s), ctypes.byref(gs), None, None, dx, dg, None, far[4], 1 << 40,
                                              None))
        status.append(lib.varlen_token_logprobs_bwd(b, 0, rb, P, P, P, P, P, T, D, -100, 1.0, a, ra, None))
        assert [x == INVALID for x in status] == [meet and not same] * len(status), (a0, ra, b0, rb, status)
        for dx, rx, dg, rg, h, rh in ((a, ra, far[1], 64, b, rb), (far[1], 64, a, ra, b, rb), (a, ra, b, rb, far[1], 64)):
            s = scan_shape(va, gate_row_stride=64, h_row_stride=rh, x_row_stride=64, **both)   # on h, on one another: never
            gs = va.VaScanGradStrides(64, rx, rg)
            x = lib.varlen_scan_bwd(far[2], h, far[3], P, ctypes.byref(s), ctypes.byref(gs), None, None, dx, dg, None, far[4], 1 << 40, None)
            assert (x == INVALID) == meet, (a0, ra, b0, rb)
    assert {(True, True), (False, True), (False, False)} <= seen
