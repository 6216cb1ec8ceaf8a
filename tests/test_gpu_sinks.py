"""GPU parity of the local window with sinks (query i sees the keys j <= i with j >= i - w or
j < s of its segment) against the float64 oracle: tile maps bit-exact, O / LSE / dQ / dK / dV
within the attention tolerances, closed forms, strides, streams, graphs and refusals."""
import numpy as np
import pytest
import torch

import seeded_inputs as si
from oracle import attention as oa
from oracle import packing as op
from oracle import tiles as ot
import _workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EDGE = [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1, 383, 384, 385, 700]


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    pkg._lib.load()
    return pkg


def boundaries(lengths):
    cu, _, _, mx = op.build_metadata(lengths)
    return cu, torch.tensor(cu, dtype=torch.int32, device=DEV), mx


@pytest.mark.parametrize("w,s", [(0, 1), (1, 4), (63, 64), (128, 127), (200, 129), (512, 4), (100, 600), (5000, 4),
                                 (64, 5000)])
def test_sink_maps_bit_exact(va, w, s):
    for lengths, Hq, Hkv, d in ((EDGE, 4, 2, 128), (wl.pack("sft8k", 0), 32, 32, 128),
                                (wl.pack("tiny4k")[:300], 8, 8, 64), (wl.pack("long64k"), 16, 16, 128)):
        cu, cud, mx = boundaries(lengths)
        for kind in (0, 1, 2):
            BM, BN = va.tile_sizes(kind, d)
            ref = (ot.bwd_tile_map(cu, Hkv, BM, BN, True, 0, window=w, sinks=s) if kind == 1 else
                   ot.fwd_tile_map(cu, Hq, BM, BN, True, 0, window=w, sinks=s))
            tm, n = va.plan(cud, int(cu[-1]), Hq, Hkv, d, mx, kind, True, window=w, sinks=s)
            assert n == len(ref)
            assert np.array_equal(tm.cpu().numpy(), ref)


def run_both(va, q, k, v, do, cud, mx, w, s, ws=(None, None)):
    qd, kd, vd, dod = (x.to(DEV) for x in (q, k, v, do))
    o, lse = va.varlen_attn_fwd(qd, kd, vd, cud, mx, None, True, check_status=True, window=w, sinks=s, workspace=ws[0])
    g = va.varlen_attn_bwd(qd, kd, vd, o, lse, dod, cud, mx, None, True, check_status=True, window=w, sinks=s,
                           workspace=ws[1])
    torch.cuda.synchronize()
    return o.cpu().double().numpy(), lse.cpu().double().numpy(), tuple(x.cpu().double().numpy() for x in g)


def against_oracle(got, q, k, v, do, cu, w, s, kv_heads=None, chunked=True):
    qq, kk, vv, dd = (si.to_f64(x) for x in (q, k, v, do))
    ro, rl = oa.varlen_forward(qq, kk, vv, cu, window=w, sinks=s, kv_heads=kv_heads)
    rg = oa.varlen_backward(qq, kk, vv, ro, rl, dd, cu, window=w, sinks=s, kv_heads=kv_heads)
    o, lse, gr = got
    wl.assert_close_outputs(o, lse, ro, rl)
    wl.assert_close_grads(gr, rg)
    if chunked:
        wl.assert_close_grads_chunked(gr, rg)


# w = 0 leaves a query itself and the sinks; sinks inside one tile, at its edges, across several
@pytest.mark.parametrize("w,s", [(0, 1), (0, 130), (1, 4), (63, 64), (100, 7), (128, 127), (200, 129), (300, 300)])
@pytest.mark.parametrize("d,g", [(64, 1), (128, 2)])
def test_sink_parity_ragged(va, w, s, d, g):
    cu, cud, mx = boundaries(EDGE)
    T, Hkv = int(cu[-1]), 2
    q, k, v, do = si.tensors(T, Hkv * g, Hkv, d, seed_offset=700 + w + d + g + s)
    against_oracle(run_both(va, q, k, v, do, cud, mx, w, s), q, k, v, do, cu, w, s)


@pytest.mark.parametrize("Hq,Hkv,d", [(12, 1, 128), (8, 8, 64)])
def test_sink_parity_one_long_segment(va, Hq, Hkv, d):
    """A segment whose sink block is seen by many more queries than any other key block."""
    cu, cud, mx = boundaries([9001])
    q, k, v, do = si.tensors(9001, Hq, Hkv, d, seed_offset=60 + Hq)
    got = run_both(va, q, k, v, do, cud, mx, 130, 5)
    # dK of the sink rows is a sum over 9000 queries: compared by itself too
    qq, kk, vv, dd = (si.to_f64(x) for x in (q, k, v, do))
    heads = None if Hkv == 1 else [2, 7]
    ro, rl = oa.varlen_forward(qq, kk, vv, cu, window=130, sinks=5, kv_heads=heads)
    rg = oa.varlen_backward(qq, kk, vv, ro, rl, dd, cu, window=130, sinks=5, kv_heads=heads)
    wl.assert_close_outputs(got[0], got[1], ro, rl)
    wl.assert_close_grads(got[2], rg)
    hs = [0] if Hkv == 1 else heads
    for i in (1, 2):
        assert wl.rel_l2(got[2][i][:5, hs], rg[i][:5, hs]) <= wl.GRAD_REL_L2


def test_sinks_degenerate_forms(va):
    """sinks = 0 and a window or sink count over the whole segment give the results of the
    window and of the plain causal call on the same inputs."""
    cu, cud, mx = boundaries(EDGE)
    q, k, v, do = si.tensors(int(cu[-1]), 4, 2, 128, seed_offset=11)
    for (w, s), (w2, s2) in (((77, 0), (77, 0)), ((5000, 3), (5000, 0)), ((10, 5000), (5000, 0)),
                             ((2 ** 31 - 1, 2 ** 31 - 1), (5000, 0))):
        a, b = run_both(va, q, k, v, do, cud, mx, w, s), run_both(va, q, k, v, do, cud, mx, w2, s2)
        if (w, s) == (w2, s2):
            assert np.array_equal(a[0], b[0])
        assert np.abs(a[0] - b[0]).max() <= wl.O_MAX_ABS and np.abs(a[1] - b[1]).max() <= wl.LSE_MAX_ABS
        for x, y in zip(a[2], b[2]):
            assert wl.rel_l2(x, y) <= wl.GRAD_REL_L2


def test_sinks_only_the_sinks_carry_weight(va):
    """Large positive scores on the sinks: O is their mean value for every later query."""
    cu, cud, mx = boundaries([1000])
    T, s = 1000, 4
    q, k, v = torch.zeros(T, 1, 64), torch.zeros(T, 1, 64), torch.randn(T, 1, 64, generator=torch.Generator().manual_seed(3))
    q[..., 0] = 32.0
    k[:s, :, 0] = 32.0                                   # scores 128 against 0
    q, k, v = (x.bfloat16() for x in (q, k, v))
    o, lse = va.varlen_attn_fwd(q.to(DEV), k.to(DEV), v.to(DEV), cud, mx, window=50, sinks=s, check_status=True)
    ref = v[:s].double().mean(0).numpy()
    o = o.cpu().double().numpy()
    assert np.abs(o[s:] - ref).max() <= wl.O_MAX_ABS
    assert np.abs(lse.cpu().double().numpy()[:, s:] - (128 + np.log(4))).max() <= wl.LSE_MAX_ABS


def test_sink_workload_packs(va):
    """An sft8k pack and a gqa16k bin, all heads on the GPU, some against the oracle."""
    for name, idx, w, s, heads in (("sft8k", 1, 511, 4, [3, 20]), ("gqa16k", 0, 1023, 66, [5])):
        w_ = si.WORKLOADS[name]
        cu, cud, mx = boundaries(wl.pack(name, idx))
        q, k, v, do = si.tensors(int(cu[-1]), w_.Hq, w_.Hkv, w_.d, seed_offset=911)
        against_oracle(run_both(va, q, k, v, do, cud, mx, w, s), q, k, v, do, cu, w, s, heads, chunked=False)


def test_sinks_strided_side_stream_and_graph(va):
    """Views into one fused projection, on a side stream, captured and replayed on new inputs:
    bit-equal to contiguous eager calls; a workspace left dirty by another call does not matter."""
    cu, cud, mx = boundaries([300, 17, 640, 1])
    T, Hq, Hkv, d = int(cu[-1]), 4, 2, 128
    q, k, v, do = (x.to(DEV) for x in si.tensors(T, Hq, Hkv, d, seed_offset=21))
    fused = torch.empty(T, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device=DEV)
    fq, fk, fv = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    dof = torch.empty(T, Hq, d, dtype=torch.bfloat16, device=DEV)
    o = torch.empty(T, Hq, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(Hq, T, device=DEV)
    kw = dict(window=70, sinks=9)
    n = max(va.workspace_size(T, 4, Hq, Hkv, d, mx, b, **kw) for b in (False, True))
    ws = torch.full((n,), 0x7f, dtype=torch.uint8, device=DEV)

    def step():
        va.varlen_attn_fwd(fq, fk, fv, cud, mx, out=o, lse=lse, workspace=ws, **kw)
        return va.varlen_attn_bwd(fq, fk, fv, o, lse, dof, cud, mx, workspace=ws, **kw)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
        graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        got = step()
    for off in (0, 5):
        q, k, v, do = (x.to(DEV) for x in si.tensors(T, Hq, Hkv, d, seed_offset=21 + off))
        fq.copy_(q), fk.copy_(k), fv.copy_(v), dof.copy_(do)
        graph.replay()
        torch.cuda.synchronize()
        o2, lse2 = va.varlen_attn_fwd(q, k, v, cud, mx, **kw)
        ref = va.varlen_attn_bwd(q, k, v, o2, lse2, do, cud, mx, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert va.read_status(ws) == 0


def test_sinks_autograd_differences_and_refusals(va):
    """Autograd through varlen_attn: against the oracle's gradient, and the directional
    derivative of the float64 oracle forward (central differences)."""
    cu, cud, mx = boundaries([70, 5, 200])
    T = int(cu[-1])
    q, k, v, do = si.tensors(T, 2, 2, 64, seed_offset=5)
    qd, kd, vd = (x.to(DEV).requires_grad_(True) for x in (q, k, v))
    out = va.varlen_attn(qd, kd, vd, cud, mx, window=33, sinks=3)
    out.backward(do.to(DEV))
    got = tuple(x.grad.cpu().double().numpy() for x in (qd, kd, vd))
    qq, kk, vv, dd = (si.to_f64(x) for x in (q, k, v, do))
    ro, rl = oa.varlen_forward(qq, kk, vv, cu, window=33, sinks=3)
    wl.assert_close_grads(got, oa.varlen_backward(qq, kk, vv, ro, rl, dd, cu, window=33, sinks=3))
    rng = np.random.default_rng(0)
    base = [qq, kk, vv]
    for a in range(3):
        u = rng.standard_normal(base[a].shape)
        f = [0.0, 0.0]
        for sgn in (0, 1):
            x = list(base)
            x[a] = base[a] + (1e-4 if sgn else -1e-4) * u
            f[sgn] = float((oa.varlen_forward(*x, cu, window=33, sinks=3)[0] * dd).sum())
        # the kernel's gradient has a relative L2 error of at most 1e-2, so along u its error is at
        # most that times |grad| |u|
        assert abs((f[1] - f[0]) / 2e-4 - (got[a] * u).sum()) <= \
            wl.GRAD_REL_L2 * np.linalg.norm(got[a]) * np.linalg.norm(u)
    q, k, v = (x.detach() for x in (qd, kd, vd))
    for kw in (dict(sinks=3), dict(window=3, sinks=-1), dict(window=3, sinks=2, causal=False)):
        with pytest.raises(va.VarlenError) as e:
            va.varlen_attn_fwd(q, k, v, cud, mx, **kw)
        assert e.value.status == 1
    bad = torch.tensor([0, 70, 70, 275], dtype=torch.int32, device=DEV)     # an empty segment
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    va.varlen_attn_fwd(q, k, v, bad, mx, window=3, sinks=2, workspace=ws)
    assert va.read_status(ws) == 5


def _align256(x):
    return (x + 255) // 256 * 256


def piece_of(T, Hq, Hkv, w, s, mx):
    """The backward's rule for cutting a sink block's q range (q blocks per piece, 0: never)."""
    g, w, s = Hq // Hkv, min(w, mx), min(s, mx)
    share = Hq * (T // 128 + 1) * (w // 64 + 2) // 152
    if s == 0 or g * (mx // 64 + 1) <= max(share, 64):
        return 0
    P = max(8, -(-(share // 4) // g)) * ((-(-s // 128) + 1) // 2)
    return P if 64 * P < mx else 0


# both planning paths (up to 32 segments, more), one and several blocks with sinks, split and not
@pytest.mark.parametrize("w,s", [(0, 1), (100, 4), (1000, 130), (5000, 9), (64, 0), (700, 0), (300, 400)])
@pytest.mark.parametrize("lengths,Hq,Hkv,d", [(EDGE, 4, 2, 128), ([9001, 1, 3000, 2689, 2690], 12, 1, 128),
                                              (EDGE * 3 + [5000], 24, 2, 64), ([40], 8, 8, 64),
                                              (EDGE[:9] * 5, 4, 2, 64)])
def test_call_maps_bit_exact(va, lengths, Hq, Hkv, d, w, s):
    """The maps the attention calls build for themselves, read back from their workspaces."""
    cu, cud, mx = boundaries(lengths)
    T, B = int(cu[-1]), len(lengths)
    q, k, v, do = (torch.zeros(T, h, d, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv, Hq))
    kw = dict(window=w, sinks=s)
    # a window or sinks over the longest segment: the causal call's maps
    whole = w >= mx - 1 or s >= mx - 1
    w, s = (None, 0) if whole else (w, s)
    piece = 0 if whole else piece_of(T, Hq, Hkv, w, s, mx)
    blocks = -(-min(s, mx) // 128)
    ws_f, ws_b = (torch.full((va.workspace_size(T, B, Hq, Hkv, d, mx, x, **kw),), 0x5a, dtype=torch.uint8, device=DEV)
                  for x in (False, True))
    o, lse = va.varlen_attn_fwd(q, k, v, cud, mx, workspace=ws_f, check_status=True, **kw)
    va.varlen_attn_bwd(q, k, v, o, lse, do, cud, mx, workspace=ws_b, check_status=True, **kw)
    BN_kv = va.tile_sizes(1, d)[1]
    kvmap = _align256(256 + Hq * T * 4)
    cap = (T // BN_kv + B) * Hkv + (blocks * (T // (64 * piece) + 1) * Hkv if piece else 0)
    qmap = _align256(kvmap + cap * 16)
    for ws, kind, at in ((ws_f, 0, 256), (ws_b, 1, kvmap), (ws_b, 2, qmap)):
        BM, BN = va.tile_sizes(kind, d)
        short = 64 if T < 256 * B and (whole or B > 32) and (kind == 0 or not piece) else 0      # token tiles
        ref = (ot.bwd_tile_map(cu, Hkv, BM, BN, True, short, window=w, sinks=s, piece=piece, window_tokens=True)
               if kind == 1 else ot.fwd_tile_map(cu, Hq, BM, BN, True, short, window=w, sinks=s, window_tokens=True))
        raw = ws.cpu().numpy()
        assert int(raw[4 + 4 * kind:8 + 4 * kind].view(np.int32)[0]) == len(ref)
        got = raw[at:at + 16 * len(ref)].view(np.int32).reshape(-1, 4)
        assert np.array_equal(got, ref), kind


def test_split_sink_blocks_parity(va):
    """Several segments long enough to be cut, next to short ones, sinks over three key blocks, 12 q
    heads on one kv head; the gradient of every row and of the sink rows alone; the same bits twice."""
    lengths = [2100, 5, 4400, 129, 3333, 1400]
    cu, cud, mx = boundaries(lengths)
    T, w, s = int(cu[-1]), 90, 261
    assert 0 < piece_of(T, 12, 1, w, s, mx) * 64 < 1400
    q, k, v, do = si.tensors(T, 12, 1, 64, seed_offset=77)
    got = run_both(va, q, k, v, do, cud, mx, w, s)
    against_oracle(got, q, k, v, do, cu, w, s)
    again = run_both(va, q, k, v, do, cud, mx, w, s)
    assert all(np.array_equal(a, b) for a, b in zip(got[2], again[2]))
    qq, kk, vv, dd = (si.to_f64(x) for x in (q, k, v, do))
    ro, rl = oa.varlen_forward(qq, kk, vv, cu, window=w, sinks=s)
    rg = oa.varlen_backward(qq, kk, vv, ro, rl, dd, cu, window=w, sinks=s)
    for b, n in zip(cu[:-1], lengths):
        for i in (1, 2):
            rows = slice(int(b), int(b) + min(n, s))
            assert wl.rel_l2(got[2][i][rows], rg[i][rows]) <= wl.GRAD_REL_L2


def test_window_and_sinks_past_32_bits(va):
    """A window or sink count beyond 32 bits is the whole segment, not its low word."""
    cu, cud, mx = boundaries([300, 40])
    q, k, v, do = si.tensors(int(cu[-1]), 2, 1, 64, seed_offset=21)
    a = run_both(va, q, k, v, do, cud, mx, 5, 2 ** 32)
    b = run_both(va, q, k, v, do, cud, mx, 2 ** 32 + 5, 0)
    ref = run_both(va, q, k, v, do, cud, mx, 5000, 0)
    for x in (a, b):
        assert np.abs(x[0] - ref[0]).max() <= wl.O_MAX_ABS and np.abs(x[1] - ref[1]).max() <= wl.LSE_MAX_ABS
        for y, z in zip(x[2], ref[2]):
            assert wl.rel_l2(y, z) <= wl.GRAD_REL_L2


@pytest.mark.parametrize("w,s", [(0, 1), (1, 0), (3, 2), (7, 70), (20, 5), (63, 1), (100, 30)])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 128), (2, 2, 64)])
def test_runs_of_short_segments(va, w, s, Hq, Hkv, d):
    """Token tiles under a window: runs of segments of 1 to 64 tokens between longer ones."""
    rng = np.random.default_rng(w + 10 * s)
    lengths = [1, 64, 2, 63, 65, 300] + rng.integers(1, 65, size=40).tolist() + [130, 1, 1, 1, 90] + \
        rng.integers(1, 20, size=60).tolist()
    cu, cud, mx = boundaries(lengths)
    q, k, v, do = si.tensors(int(cu[-1]), Hq, Hkv, d, seed_offset=31)
    got = run_both(va, q, k, v, do, cud, mx, w, s)
    qq, kk, vv, dd = (si.to_f64(x) for x in (q, k, v, do))
    ro, rl = oa.varlen_forward(qq, kk, vv, cu, window=w, sinks=s)
    wl.assert_close_outputs(got[0], got[1], ro, rl)
    wl.assert_close_grads(got[2], oa.varlen_backward(qq, kk, vv, ro, rl, dd, cu, window=w, sinks=s))
