"""GPU parity of the embedding lookup and its gradient by sorted tokens against float64."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
VA_ERR_BAD_IDS = 9


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    pkg._lib.load()
    return pkg


def draw_ids(T, V, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        ids = torch.randint(0, V, (T,), generator=g)
    elif kind == "zipf":
        ids = (torch.exp(torch.rand(T, generator=g, dtype=torch.float64) * math.log(V + 1)) - 1).long().clamp(0, V - 1)
    elif kind == "one":
        ids = torch.full((T,), V - 1)
    elif kind == "pad":
        ids = torch.full((T,), -1)
    else:                                                    # every id once, backwards
        ids = torch.arange(T).flip(0) % V
    if kind in ("uniform", "zipf"):
        ids[torch.rand(T, generator=g) < 0.05] = -7
    return ids.to(torch.int32)


def reference_gradient(dout, ids, V, scale):
    """(gradient, n, sum of magnitudes) in float64: n terms per row."""
    d, keep = dout.double().numpy(), ids.numpy() >= 0
    ref, mag, n = np.zeros((V, d.shape[1])), np.zeros((V, d.shape[1])), np.zeros(V)
    np.add.at(ref, ids.numpy()[keep], d[keep])
    np.add.at(mag, ids.numpy()[keep], np.abs(d[keep]))
    np.add.at(n, ids.numpy()[keep], 1)
    return ref * scale, n[:, None], mag * abs(scale)


def check_gradient(got, dout, ids, V, scale, base=None):
    """A sum of n fp32 terms in any order is off by at most n 2^-24 of its magnitudes' sum; the
    scale (itself fp32) and the product round once each, then the type of the table once."""
    scale = float(np.float32(scale))
    ref, n, mag = reference_gradient(dout, ids, V, scale)
    half = HALF[got.dtype]
    if base is not None:
        ref, mag = ref + base.double().numpy(), mag + np.abs(base.double().numpy())
    tol = (n + 3) * 2.0 ** -24 * mag + half * (1 + 2.0 ** -8) * np.abs(ref) + 1e-37
    g = got.cpu().double().numpy()
    assert (np.abs(g - ref) <= tol).all(), np.max(np.abs(g - ref) / tol)
    if base is None:
        assert np.all(g[n[:, 0] == 0] == 0)
    else:
        assert np.array_equal(g[n[:, 0] == 0], base.double().numpy()[n[:, 0] == 0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (5, 7, 8), (33, 100, 24), (446, 32000, 512), (300, 1000, 130),
                                   (1000, 50, 16), (70, 600, 4096), (9, 40, 5000), (3, 50, 16392)])
def test_forward(va, dtype, T, V, D):
    g = torch.Generator().manual_seed(T + D)
    table = torch.randn(V, D, generator=g).to(dtype)
    ids = draw_ids(T, V, "uniform", T)
    for scale in (1.0, math.sqrt(D), -0.3):
        out = va.embed_fwd(table.to(DEV), ids.to(DEV), scale, check_status=True).cpu()
        ref = table.double().numpy()[ids.clamp(min=0).numpy()] * float(np.float32(scale))
        ref[ids.numpy() < 0] = 0
        tol = (HALF[dtype] * (1 + 2.0 ** -8) + (2.0 ** -24 if dtype == BF else 0)) * np.abs(ref)
        assert (np.abs(out.double().numpy() - ref) <= tol).all()
        if scale == 1.0:
            assert np.array_equal(out.double().numpy(), ref)


# one digit and several; chunks that end inside runs; runs over many chunks; every thread mapping
@pytest.mark.parametrize("kind", ["uniform", "zipf", "one", "pad", "each"])
@pytest.mark.parametrize("T,V,D", [(1, 1, 8), (2, 3, 1), (31, 5, 24), (300, 1000, 130), (1000, 300, 512), (8192, 2000, 64),
                                   (20011, 3000, 40), (515, 513, 2056), (129, 40000, 16), (64, 300, 4096)])
def test_gradient(va, kind, T, V, D):
    g = torch.Generator().manual_seed(T + D)
    ids = draw_ids(T, V, kind, T + 1)
    for din, dtab in ((BF, BF), (F32, F32), (BF, F32), (F32, BF)):
        if (din, dtab) != (BF, BF) and T * D > 600000 and kind != "zipf":
            continue
        dout = torch.randn(T, D, generator=g).to(din)
        out = torch.full((V, D), 5.0, dtype=dtab, device=DEV)
        got = va.embed_bwd(dout.to(DEV), ids.to(DEV), V, 0.7, dtable=out, check_status=True)
        assert got.data_ptr() == out.data_ptr()
        check_gradient(got, dout, ids, V, 0.7)


def test_gradient_many_tokens_and_large_vocabulary(va):
    """Three radix digits, more rows than 16-bit numbers, runs of thousands of tokens."""
    T, V, D = 140000, 300000, 32
    ids = draw_ids(T, V, "zipf", 3)
    ids[::5] = 77777
    dout = torch.randn(T, D, generator=torch.Generator().manual_seed(1)).to(BF)
    a = va.embed_bwd(dout.to(DEV), ids.to(DEV), V, 2.0, check_status=True)
    check_gradient(a, dout, ids, V, 2.0)
    b = va.embed_bwd(dout.to(DEV), ids.to(DEV), V, 2.0)
    assert torch.equal(a, b)                                 # the same bits every time


@pytest.mark.parametrize("dtab", [BF, F32])
def test_accumulate(va, dtab):
    """Added to what the tensor holds; rows of absent ids keep their bits."""
    T, V, D = 2000, 500, 72
    ids = draw_ids(T, V, "zipf", 9)
    dout = torch.randn(T, D, generator=torch.Generator().manual_seed(2)).to(BF)
    base = torch.randn(V, D, generator=torch.Generator().manual_seed(3)).to(dtab)
    got = va.embed_bwd(dout.to(DEV), ids.to(DEV), V, 0.5, dtable=base.to(DEV), accumulate=True, check_status=True)
    check_gradient(got, dout, ids, V, 0.5, base=base)


def test_ids_past_the_table(va):
    """Status VA_ERR_BAD_IDS, NaN rows in the lookup, no gradient; nothing else changes."""
    table = torch.randn(10, 16, device=DEV)
    ids = torch.tensor([1, 10, 3, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    with pytest.raises(va.VarlenError) as e:
        va.embed_fwd(table, ids, check_status=True)
    assert e.value.status == VA_ERR_BAD_IDS
    out = va.embed_fwd(table, ids)
    assert torch.isnan(out[[1, 3]]).all() and (out[4] == 0).all() and torch.equal(out[[0, 2]], table[[1, 3]])
    dout = torch.randn(5, 16, device=DEV)
    ws = torch.full((va._lib.load().varlen_embed_bwd_workspace_size(5, 16),), 0x7f, dtype=torch.uint8, device=DEV)
    d = va.embed_bwd(dout, ids, 10, workspace=ws)
    assert va.read_status(ws) == VA_ERR_BAD_IDS
    assert torch.equal(d[1], dout[0]) and torch.equal(d[3], dout[2]) and int((d != 0).any(1).sum()) == 2
    va.embed_bwd(dout, ids.clamp(0, 9), 10, workspace=ws)
    assert va.read_status(ws) == 0


def test_empty_stream(va):
    table = torch.randn(10, 16, device=DEV)
    ids = torch.empty(0, dtype=torch.int32, device=DEV)
    assert va.embed_fwd(table, ids).shape == (0, 16)
    d = torch.full((10, 16), 3.0, device=DEV)
    va.embed_bwd(torch.empty(0, 16, device=DEV), ids, 10, dtable=d, accumulate=True, check_status=True)
    assert (d == 3).all()
    va.embed_bwd(torch.empty(0, 16, device=DEV), ids, 10, dtable=d, check_status=True)
    assert (d == 0).all()


def test_strides_and_alignment(va):
    """Column slices of wider tensors on and off 16-byte boundaries: the bits of contiguous calls,
    nothing beside the rows written."""
    T, V, D = 700, 90, 48
    ids = draw_ids(T, V, "zipf", 4).to(DEV)
    table, dout = torch.randn(V, D, device=DEV).to(BF), torch.randn(T, D, device=DEV).to(BF)
    out, dt = va.embed_fwd(table, ids, 3.0), va.embed_bwd(dout, ids, V, 3.0)
    for off in (0, 1, 8):
        wt, wo = torch.zeros(V, 80, dtype=BF, device=DEV), torch.full((T, 80), 9.0, dtype=BF, device=DEV)
        wt[:, off:off + D] = table
        o = va.embed_fwd(wt[:, off:off + D], ids, 3.0, out=wo[:, off:off + D])
        assert torch.equal(o, out) and (wo[:, off + D:] == 9).all() and (wo[:, :off] == 9).all()
        wd, wg = torch.zeros(T, 80, dtype=BF, device=DEV), torch.full((V, 80), 9.0, dtype=BF, device=DEV)
        wd[:, off:off + D] = dout
        g = va.embed_bwd(wd[:, off:off + D], ids, V, 3.0, dtable=wg[:, off:off + D])
        assert torch.equal(g, dt) and (wg[:, off + D:] == 9).all() and (wg[:, :off] == 9).all()


def test_autograd_differences_and_broadcast_gradient(va):
    """The operator is linear in the table: <dout, embed(u)> = <embed's gradient, u> exactly up to
    fp32 sums; a broadcast (stride 0) gradient of sum() and two backward passes of one graph."""
    V, T, D = 60, 200, 40
    ids = draw_ids(T, V, "uniform", 6)
    table = torch.randn(V, D, device=DEV).requires_grad_(True)
    out = va.embed(table, ids.to(DEV), 1.5)
    dout, u = torch.randn(T, D, device=DEV), torch.randn(V, D, device=DEV)
    out.backward(dout, retain_graph=True)
    check_gradient(table.grad, dout.cpu(), ids, V, 1.5)
    lhs = float((va.embed_fwd(u, ids.to(DEV), 1.5).double() * dout.double()).sum())
    rhs = float((table.grad.double() * u.double()).sum())
    # each side's terms carry a few fp32 roundings: at most 30 tokens share an id
    assert abs(lhs - rhs) <= 34 * 2.0 ** -24 * 1.5 * float((u[ids.clamp(min=0).to(DEV).long()] * dout).abs().sum())
    table.grad = None
    out.sum().backward()
    check_gradient(table.grad, torch.ones(T, D), ids, V, 1.5)


def test_refusals(va):
    t, i = torch.zeros(4, 8, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    for args in ((t.half(), i), (t.t(), i), (t[0], i), (t, i.long()), (t, i[None]), (t, i.cpu()),
                 (t, torch.zeros(6, dtype=torch.int32, device=DEV)[::2])):
        with pytest.raises(ValueError):
            va.embed_fwd(*args)
    with pytest.raises(ValueError):
        va.embed_fwd(t, i, out=torch.empty(3, 8, dtype=BF, device=DEV))
    d = torch.zeros(3, 8, device=DEV)
    for kw in (dict(dout=d[:2]), dict(dtable=torch.zeros(5, 8, device=DEV)), dict(accumulate=True),
               dict(dtable=torch.zeros(4, 8, device=DEV).half()), dict(ids=i.long())):
        a = dict(dout=d, ids=i, num_rows=4)
        a.update(kw)
        with pytest.raises(ValueError):
            va.embed_bwd(**a)
    with pytest.raises(va.VarlenError) as e:
        va.embed_fwd(t, i, math.nan)
    assert e.value.status == 1
    with pytest.raises(va.VarlenError):                      # rows that overlap
        va.embed_bwd(d[:1].expand(3, 8), i, 4)


def test_graph_replay_on_a_side_stream(va):
    T, V, D = 900, 700, 256
    ids, dout = draw_ids(T, V, "zipf", 1).to(DEV), torch.randn(T, D, device=DEV).to(BF)
    table = torch.randn(V, D, device=DEV).to(BF)
    ws = torch.empty(va._lib.load().varlen_embed_bwd_workspace_size(T, D), dtype=torch.uint8, device=DEV)
    dt = torch.empty(V, D, dtype=BF, device=DEV)
    out = torch.empty(T, D, dtype=BF, device=DEV)

    def step():
        va.embed_fwd(table, ids, 2.0, out=out)
        va.embed_bwd(dout, ids, V, 2.0, dtable=dt, workspace=ws)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    for seed in (2, 3):
        ids.copy_(draw_ids(T, V, "zipf", seed))
        dout.copy_(torch.randn(T, D))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, va.embed_fwd(table, ids, 2.0)) and torch.equal(dt, va.embed_bwd(dout, ids, V, 2.0))


def test_second_derivative_is_refused(va):
    table = torch.randn(5, 8, device=DEV).requires_grad_(True)
    out = va.embed(table, torch.tensor([1, 3, 1], dtype=torch.int32, device=DEV))
    w = torch.randn(3, 8, device=DEV).requires_grad_(True)
    (g,) = torch.autograd.grad(out, table, w, create_graph=True)
    with pytest.raises(RuntimeError):
        g.square().sum().backward()


def test_sizes_past_the_arguments(va):
    i = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):                          # would wrap to 4 rows
        va.embed_bwd(torch.ones(2, 1, device=DEV), i, 2 ** 32 + 4)
