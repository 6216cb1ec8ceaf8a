"""Windows with sinks at the ends of their ranges."""
import ctypes
import math

import pytest
import torch

import seeded_inputs as si
from oracle import attention as oa
from oracle import packing as op
import _workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    pkg._lib.load()
    return pkg


def test_more_sink_tiles_than_16_bits_count(va):
    """2^22 sinks (32768 key tiles of 128) before a window of two keys: one key in the first sink tile
    and one in the last carry nearly all of the weight.

    Scores are 0 but for those two keys' 20, so of a query i past the sinks lse = ln(2 e^20 + n - 2), n
    its visible keys.  The row sum is up to 2^15 + 2 additions of positive numbers in fp32, each off by at
    most 2^-24 of the sum: 2^-8.9 altogether, on top of the usual tolerance of lse; O has that relative
    error on top of its own."""
    s = 1 << 22
    T, one = s + 700, (5, s - 100)
    q, k, v = (torch.zeros(T, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    q[..., 0] = 8
    for j, x in zip(one, (1.0, 3.0)):
        k[j, :, 0] = 20                                     # 8 * 20 / 8 = 20
        v[j] = x
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    o, lse = va.varlen_attn_fwd(q, k, v, cu, T, window=1, sinks=s, check_status=True)
    i = torch.arange(s, T, device=DEV)
    n = s + torch.where(i == s, 1, 2).double()              # the sinks, and i - 1 and i where they are none
    total = 2 * math.exp(20) + n - 2
    eps = 2.0 ** -8.9
    assert (lse[0, s:].double() - total.log()).abs().max().item() <= wl.LSE_MAX_ABS + eps
    ref = (4 * math.exp(20) / total)[:, None, None]
    assert (o[s:].double() - ref).abs().max().item() <= wl.O_MAX_ABS + 2 * eps


WHOLE = 300                                      # the longest segment below


def inputs(d):
    cu, _, _, mx = op.build_metadata([WHOLE, 17, WHOLE, 1, 129])
    assert mx == WHOLE
    t = si.tensors(int(cu[-1]), 2, 1, d, seed_offset=400 + d)
    return cu, torch.tensor(cu, dtype=torch.int32, device=DEV), t, [x.to(DEV) for x in t]


def step(va, x, cud, **kw):
    q, k, v, do = x
    o, lse = va.varlen_attn_fwd(q, k, v, cud, WHOLE, check_status=True, **kw)
    return (o, lse) + va.varlen_attn_bwd(q, k, v, o, lse, do, cud, WHOLE, check_status=True, **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("w,s", [(WHOLE - 3, 0), (WHOLE - 2, 0), (WHOLE - 1, 0), (WHOLE, 0), (WHOLE - 2, 1), (WHOLE - 1, 1),
                                 (WHOLE - 2, WHOLE - 2), (0, WHOLE - 3), (0, WHOLE - 2), (0, WHOLE - 1), (5, WHOLE), (0, 1)])
def test_at_the_longest_segments_length(va, w, s, d):
    """Where a window or the sinks begin to cover the longest segment (WHOLE - 1: the causal call's kernels;
    one less still hides at most a key), each against the oracle with the mask as defined."""
    cu, cud, host, dev = inputs(d)
    got = [t.double().cpu().numpy() for t in step(va, dev, cud, window=w, sinks=s)]
    qq, kk, vv, dd = (si.to_f64(x) for x in host)
    ro, rl = oa.varlen_forward(qq, kk, vv, cu, window=w, sinks=s)
    wl.assert_close_outputs(got[0], got[1], ro, rl)
    wl.assert_close_grads(tuple(got[2:]), oa.varlen_backward(qq, kk, vv, ro, rl, dd, cu, window=w, sinks=s))


@pytest.mark.parametrize("w,s", [(WHOLE - 1, 0), (WHOLE, 7), (2 ** 31 - 1, 2 ** 31 - 1), (3, WHOLE - 1)])
def test_whole_windows_are_the_causal_call(va, w, s):
    """The same bits as the call without a window."""
    _, cud, _, dev = inputs(128)
    for a, b in zip(step(va, dev, cud, window=w, sinks=s), step(va, dev, cud)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("w", [0, 77, WHOLE - 2])
def test_no_sinks_is_the_window_call(va, w):
    """sinks = 0 gives the bits of the library's window entry points."""
    cu, cud, _, (q, k, v, do) = inputs(64)
    o, lse, dq, dk, dv = step(va, (q, k, v, do), cud, window=w, sinks=0)
    lib, shape = va._lib.load(), va.make_shape(q, k, v, len(cu) - 1, WHOLE)
    out = [torch.full_like(x, 9) for x in (o, lse, dq, dk, dv)]
    ws = torch.empty(max(lib.varlen_attn_workspace_size(ctypes.byref(shape), b) for b in (0, 1)), dtype=torch.uint8, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    p = [x.data_ptr() for x in (q, k, v, cud, do)]
    r = [x.data_ptr() for x in out]
    assert lib.varlen_attn_fwd_window(p[0], p[1], p[2], p[3], ctypes.byref(shape), 0.125, 1, w, r[0], r[1], ws.data_ptr(),
                                      ws.numel(), st) == 0
    assert lib.varlen_attn_bwd_window(p[0], p[1], p[2], r[0], r[1], p[4], p[3], ctypes.byref(shape), 0.125, 1, w, r[2], r[3],
                                      r[4], ws.data_ptr(), ws.numel(), st) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, (o, lse, dq, dk, dv)))
