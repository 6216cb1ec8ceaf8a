"""GPU parity of the gated recurrence over packed segments, and of its gradient, against float64."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
TYPES = [(BF, BF), (BF, F32), (F32, F32)]


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    pkg._lib.load()
    return pkg


def decay_error(g):
    """Relative error of a row's decay: an exponential of 2^-22, its argument's product, and its share of the rounding
    of a sum over a run of at most 32 rows."""
    return 2.0 ** -21 + 40 * 2.0 ** -24 * g.abs().clamp(max=1e30)


def reference(x, g, lengths, h0=None, dh=None, dlast=None):
    """Row by row in float64.  Forward: (h, bound of the fp32 error, last); with dh: (dx, bound, dg, bound, dh0, bound)."""
    x, g = x.double(), g.double()
    a, c = g.exp(), decay_error(g)
    T, D = x.shape
    z = torch.zeros(D, dtype=torch.float64)
    h, eh, before, ebefore = (torch.empty(T, D, dtype=torch.float64) for _ in range(4))
    t = 0
    for b, n in enumerate(lengths):
        s = z if h0 is None else h0[b].double()
        e, m = z, s.abs()
        for _ in range(n):
            before[t], ebefore[t] = s, e
            lost = torch.where(a[t] > 0, a[t] * (e + c[t] * m), z)
            m = torch.where(a[t] > 0, a[t] * m, z) + x[t].abs()
            s = torch.where(a[t] > 0, a[t] * s, z) + x[t]
            e = lost + 2.0 ** -22 * m
            h[t], eh[t] = s, e
            t += 1
    last = torch.tensor(lengths).cumsum(0) - 1
    if dh is None:
        return h, eh, h[last], eh[last]
    hd = HALF[torch.promote_types(dh.dtype, F32 if dh.dtype == F32 else BF)]
    dx, ex, dg, eg = (torch.empty(T, D, dtype=torch.float64) for _ in range(4))
    dh0, e0 = (torch.zeros(len(lengths), D, dtype=torch.float64) for _ in range(2))
    t = T - 1
    for b in range(len(lengths) - 1, -1, -1):
        f = z if dlast is None else dlast[b].double()
        e, m = z, f.abs()
        for _ in range(lengths[b]):
            v, m = dh[t].double() + f, dh[t].double().abs() + m
            e = e + 2.0 ** -22 * m
            dx[t], ex[t] = v, e
            f, e, m = a[t] * v, a[t] * (e + c[t] * m), a[t] * m
            dg[t] = f * before[t]
            # the row before's h as it was stored: rounded to its type
            eg[t] = e * before[t].abs() + (f.abs() + e) * (ebefore[t] + hd * (1 + 2.0 ** -7) * before[t].abs()) + 2.0 ** -23 * dg[t].abs()
            t -= 1
        dh0[b], e0[b] = f, e
    return dx, ex, dg, eg, dh0, e0


def close(got, ref, err):
    assert got.shape == ref.shape
    tol = HALF[got.dtype] * (1 + 2.0 ** -7) * ref.abs() + err * (1 + 2.0 ** -6) + 1e-37
    off = (got.cpu().double() - ref).abs() / tol
    assert float(off.max()) <= 1, float(off.max())


def make(lengths, D, xt, gt, seed=0, slow=1e-3):
    T = sum(lengths)
    g = torch.Generator().manual_seed(seed + T + D)
    mk = lambda *s: torch.randn(*s, generator=g)                             # noqa: E731
    rate = slow ** torch.rand(D, generator=g)
    ht = torch.promote_types(xt, gt)
    return dict(x=mk(T, D).to(xt), g=(-rate * torch.sigmoid(mk(T, D))).to(gt), dh=mk(T, D).to(ht), h0=2 * mk(len(lengths), D),
                dlast=mk(len(lengths), D), cu=torch.tensor([0] + lengths).cumsum(0).to(torch.int32))


def check(va, lengths, D, xt, gt, state, seed=0, m=None):
    m = make(lengths, D, xt, gt, seed) if m is None else m
    c = {n: x.to(DEV) for n, x in m.items()}
    h0, dl = (c["h0"], c["dlast"]) if state else (None, None)
    h, last = va.varlen_scan_fwd(c["x"], c["g"], c["cu"], h0, h_last=True, check_status=True)
    assert h.dtype == torch.promote_types(xt, gt) and last.dtype == F32
    rh, eh, rl, el = reference(m["x"], m["g"], lengths, m["h0"] if state else None)
    close(h, rh, eh)
    close(last, rl, el)
    got = va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"], h0, dl, x_dtype=xt, check_status=True)
    assert got[0].dtype == xt and got[1].dtype == gt
    dx, ex, dg, eg, d0, e0 = reference(m["x"], m["g"], lengths, m["h0"] if state else None, m["dh"], m["dlast"] if state else None)
    close(got[0], dx, ex)
    close(got[1], dg, eg)
    if state:
        close(got[2], d0, e0)
    else:
        assert got[2] is None
    # the same bits every time, whatever finishes first
    for _ in range(2):
        again = va.varlen_scan_fwd(c["x"], c["g"], c["cu"], h0, h_last=True)
        assert torch.equal(h, again[0]) and torch.equal(last, again[1])
        for a, b in zip(got, va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"], h0, dl, x_dtype=xt)):
            assert a is None or torch.equal(a, b)


# one row, rows around the runs and tiles, boundaries on them, many short segments, single tokens
LENGTHS = [[1], [2], [15], [16], [17], [127], [128], [129], [300, 1, 17, 129, 65], [128, 128, 1, 127, 129], [1] * 70,
           [16] * 20, [3, 1, 2] * 60, [255, 257], [5000]]


@pytest.mark.parametrize("xt,gt", TYPES)
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda x: "-".join(map(str, x[:4])) + "x%d" % len(x))
def test_parity(va, lengths, state, xt, gt):
    check(va, lengths, 40 if sum(lengths) > 1000 else 130, xt, gt, state)


@pytest.mark.parametrize("D", [1, 2, 3, 31, 33, 64, 65, 127, 200, 515])
def test_channels(va, D):
    for xt, gt in TYPES:
        check(va, [100, 30, 200], D, xt, gt, True)


def test_long_segments_cross_groups_of_tiles(va):
    """Segments that run over several groups of 32 tiles, that end on one and inside one."""
    for lengths in ([20000], [4096, 8192, 5000], [4095, 1, 4097, 9000], [10, 12289, 3]):
        check(va, lengths, 6, F32, F32, True)
        check(va, lengths, 3, BF, BF, False)


@pytest.mark.parametrize("D", [8192, 8191])
def test_offsets_past_32_bits(va, D):
    """A stream of more than 2^32 bytes: its last rows against the recurrence of those rows alone."""
    T = 300000
    x = torch.empty(T, D, device=DEV, dtype=BF)
    x.normal_(generator=torch.Generator(DEV).manual_seed(1))
    g = torch.full((1, D), -0.25, device=DEV, dtype=BF).expand(T, D).contiguous()
    cu = torch.tensor([0, 299000, T], dtype=torch.int32, device=DEV)
    h, _ = va.varlen_scan_fwd(x, g, cu, check_status=True)
    rh, eh, _, _ = reference(x[299000:, :64].cpu(), g[299000:, :64].cpu(), [1000])
    close(h[299000:, :64], rh, eh)
    # a decay of 1 / 4 a row: 200 rows before are nothing (e^-50), so the row's own past gives it
    rh, eh, _, _ = reference(x[298700:299000, -64:].cpu(), g[298700:299000, -64:].cpu(), [300])
    close(h[298900:299000, -64:], rh[200:], eh[200:] + 1e-20)
    dx, dg, _ = va.varlen_scan_bwd(x, h, g, cu, check_status=True)
    dr = reference(x[299000:, :64].cpu(), g[299000:, :64].cpu(), [1000], dh=x[299000:, :64].cpu())
    close(dx[299000:, :64], dr[0], dr[1])
    close(dg[299000:, :64], dr[2], dr[3])


def test_decays_at_their_ends(va):
    """g = 0 (a plain sum), -inf (nothing passes), very small and very large ones, in every mix."""
    lengths = [40, 300, 7]
    m = make(lengths, 64, F32, F32)
    kinds = torch.tensor([0.0, -float("inf"), -1e-8, -50.0, -1e30, -0.1])
    g = torch.Generator().manual_seed(2)
    m["g"] = kinds[torch.randint(0, 6, m["g"].shape, generator=g)]
    m["g"][:, :8] = 0.0
    m["g"][:, 8:16] = -1e-8
    check(va, lengths, 64, F32, F32, True, m=m)


def test_nothing_crosses_a_boundary(va):
    """Infinities and NaN of one segment stay in it, forward and backward, states included."""
    lengths = [100, 150, 1, 400, 60]
    m = make(lengths, 70, F32, F32)
    c = {n: x.to(DEV) for n, x in m.items()}
    bad = {n: x.clone() for n, x in c.items()}
    s, e = 100, 250                                          # the second segment, and the fourth
    for name in ("x", "g", "dh"):
        bad[name][s:e, 0], bad[name][s:e, 1], bad[name][e - 1, 2] = float("nan"), float("inf"), float("nan")
        bad[name][251 + 399, 3] = bad[name][251, 4] = float("inf")
    bad["h0"][1], bad["dlast"][3] = float("nan"), float("inf")
    clean = torch.ones(sum(lengths), dtype=torch.bool)
    clean[s:e] = clean[251:651] = False
    for x in (c, bad):
        x["h"], x["last"] = va.varlen_scan_fwd(x["x"], x["g"], x["cu"], x["h0"], h_last=True)
        x["got"] = va.varlen_scan_bwd(x["dh"], x["h"], x["g"], x["cu"], x["h0"], x["dlast"])
    for a, b in ((c["h"], bad["h"]), (c["got"][0], bad["got"][0]), (c["got"][1], bad["got"][1])):
        assert torch.equal(a[clean], b[clean])
    for a, b in ((c["last"], bad["last"]), (c["got"][2], bad["got"][2])):
        assert torch.equal(a[[0, 2, 4]], b[[0, 2, 4]])


def test_single_tokens(va):
    """T == B: the state moves on in place, step after step, as the whole sequence does."""
    B, D, steps = 37, 200, 9
    g = torch.Generator().manual_seed(4)
    x, ld = torch.randn(steps, B, D, generator=g).to(BF), -torch.rand(steps, B, D, generator=g)
    state = torch.zeros(B, D, device=DEV)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    seen = []
    for t in range(steps):
        h, last = va.varlen_scan_fwd(x[t].to(DEV), ld[t].to(DEV), cu, state, h_last=state, check_status=True)
        assert last.data_ptr() == state.data_ptr()
        seen.append(h)
    whole = x.transpose(0, 1).reshape(B * steps, D).contiguous()
    decays = ld.transpose(0, 1).reshape(B * steps, D).contiguous()
    rh, eh, rl, el = reference(whole, decays, [steps] * B)
    close(torch.stack(seen, 1).reshape(B * steps, D), rh, eh)
    close(state, rl, el)
    h, last = va.varlen_scan_fwd(x[0].to(DEV), ld[0].to(DEV), cu, h_last=True)  # without a state: x itself
    assert torch.equal(h.cpu(), x[0].float()) and torch.equal(last.cpu(), x[0].float())


def test_split_sequences(va):
    """A sequence cut in two with its state carried over is the whole one: states and gradients."""
    T, D, at = 700, 66, 333
    m = make([T], D, F32, F32)
    c = {n: x.to(DEV) for n, x in m.items()}
    cu1, cu2 = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (at, T - at))
    h, last = va.varlen_scan_fwd(c["x"], c["g"], c["cu"], c["h0"], h_last=True)
    a, la = va.varlen_scan_fwd(c["x"][:at], c["g"][:at], cu1, c["h0"], h_last=True)
    b, lb = va.varlen_scan_fwd(c["x"][at:], c["g"][at:], cu2, la, h_last=True)
    rh, eh, rl, el = reference(m["x"], m["g"], [T], m["h0"])
    close(torch.cat([a, b]), rh, 2 * eh)
    close(lb, rl, 2 * el)
    xb, gb, s = va.varlen_scan_bwd(c["dh"][at:], b, c["g"][at:], cu2, la, c["dlast"])
    xa, ga, s0 = va.varlen_scan_bwd(c["dh"][:at], a, c["g"][:at], cu1, c["h0"], s)
    dx, ex, dg, eg, d0, e0 = reference(m["x"], m["g"], [T], m["h0"], m["dh"], m["dlast"])
    close(torch.cat([xa, xb]), dx, 2 * ex)
    close(torch.cat([ga, gb]), dg, 2 * eg)
    close(s0, d0, 2 * e0)


def test_strides_and_in_place(va):
    """Views of wider rows, odd offsets, h over x, gradients over their inputs."""
    lengths, D = [200, 90], 50
    m = make(lengths, D, F32, F32)
    c = {n: x.to(DEV) for n, x in m.items()}
    rh, eh, _, _ = reference(m["x"], m["g"], lengths)
    dx, ex, dg, eg, _, _ = reference(m["x"], m["g"], lengths, dh=m["dh"])
    for off, width in ((0, 64), (1, 64), (2, 61), (3, 53), (0, 50), (2, 66)):
        wide = torch.full((6, 290, width), 9.0, device=DEV)
        xv, gv, hv, dv, ov, qv = (wide[i, :, off:off + D] for i in range(6))
        xv.copy_(c["x"]), gv.copy_(c["g"]), dv.copy_(c["dh"])
        va.varlen_scan_fwd(xv, gv, c["cu"], out=hv)
        close(hv, rh, eh)
        va.varlen_scan_bwd(dv, hv, gv, c["cu"], dx=ov, dlog_decay=qv)
        close(ov, dx, ex)
        close(qv, dg, eg)
        # over the inputs: the same bits (which other strides need not give: runs may be cut otherwise)
        va.varlen_scan_fwd(xv, gv, c["cu"], out=xv)
        assert torch.equal(xv, hv)
        va.varlen_scan_bwd(dv, hv, gv, c["cu"], dx=dv, dlog_decay=gv)
        assert torch.equal(dv, ov) and torch.equal(gv, qv)
        assert bool((wide[:, :, :off] == 9).all()) and bool((wide[:, :, off + D:] == 9).all())


@pytest.mark.parametrize("D", [63, 64, 65, 130])
@pytest.mark.parametrize("xt,gt", TYPES)
def test_rows_off_their_boundaries(va, xt, gt, D):
    """Each tensor with an offset and a row stride of its own, some on 16 bytes and others not, outputs on odd elements;
    nothing beside the rows changes."""
    lengths = [70, 1, 129, 64]
    m = make(lengths, D, xt, gt)
    T, ht = sum(lengths), torch.promote_types(xt, gt)
    cu = m["cu"].to(DEV)
    rh, eh, rl, el = reference(m["x"], m["g"], lengths, m["h0"])
    dx, ex, dg, eg, d0, e0 = reference(m["x"], m["g"], lengths, m["h0"], m["dh"], m["dlast"])
    for offs in ((0, 0, 0, 0, 0, 0), (0, 8, 0, 1, 3, 0), (1, 0, 16, 0, 2, 7), (5, 3, 1, 7, 0, 1)):
        wides, views = [], []
        for i, (off, dt) in enumerate(zip(offs, (xt, gt, ht, ht, xt, gt))):
            w = torch.full((T, D + off + (0, 3, 8)[i % 3]), 9.0, device=DEV, dtype=dt)
            wides.append((w, off))
            views.append(w[:, off:off + D])
        xv, gv, hv, dv, ov, qv = views
        xv.copy_(m["x"]), gv.copy_(m["g"]), dv.copy_(m["dh"])
        _, last = va.varlen_scan_fwd(xv, gv, cu, m["h0"].to(DEV), h_last=True, out=hv, check_status=True)
        close(hv, rh, eh)
        close(last, rl, el)
        _, _, s0 = va.varlen_scan_bwd(dv, hv, gv, cu, m["h0"].to(DEV), m["dlast"].to(DEV), dx=ov, dlog_decay=qv, check_status=True)
        close(ov, dx, ex)
        close(qv, dg, eg)
        close(s0, d0, e0)
        for w, off in wides:
            assert bool((w[:, :off] == 9).all()) and bool((w[:, off + D:] == 9).all())


@pytest.mark.parametrize("cu", [[0, 5, 5, 90], [0, 50, 40, 90], [1, 50, 60, 90], [0, 50, 60, 89], [0, 50, 2 ** 31 - 1, 90],
                                [0, -7, 60, 90]])
def test_bad_boundaries(va, cu):
    """Reported, with nothing written, and the next call is right."""
    m = make([30, 30, 30], 64, F32, F32)
    c = {n: x.to(DEV) for n, x in m.items()}
    out = torch.full((90, 64), 3.0, device=DEV)
    bad = torch.tensor(cu, dtype=torch.int32, device=DEV)
    with pytest.raises(va.VarlenError) as e:
        va.varlen_scan_fwd(c["x"], c["g"], bad, out=out, check_status=True)
    assert e.value.status == 5
    assert bool((out == 3).all())
    h, _ = va.varlen_scan_fwd(c["x"], c["g"], c["cu"], check_status=True)
    with pytest.raises(va.VarlenError) as e:
        va.varlen_scan_bwd(c["dh"], h, c["g"], bad, dx=out, check_status=True)
    assert e.value.status == 5
    assert bool((out == 3).all())
    rh, eh, _, _ = reference(m["x"], m["g"], [30, 30, 30])
    close(h, rh, eh)
    one = torch.tensor([0, 2, 2], dtype=torch.int32, device=DEV)
    with pytest.raises(va.VarlenError) as e:
        va.varlen_scan_fwd(c["x"][:2], c["g"][:2], one, check_status=True)
    assert e.value.status == 5


def test_autograd_and_differences(va):
    lengths, D = [5, 1, 20], 6
    m = make(lengths, D, F32, F32, slow=0.1)
    c = {n: x.to(DEV) for n, x in m.items()}
    leaves = [c[n].clone().requires_grad_(True) for n in ("x", "g", "h0")]
    h, last = va.varlen_scan(leaves[0], leaves[1], c["cu"], leaves[2])
    ((h * c["dh"]).sum() + (last * c["dlast"]).sum()).backward()

    def loss(x, g, h0):
        h, _, last, _ = reference(x, g, lengths, h0)
        return float((h * m["dh"].double()).sum() + (last * m["dlast"].double()).sum())

    gen = torch.Generator().manual_seed(3)
    at = [m[n].double() for n in ("x", "g", "h0")]
    for i, leaf in enumerate(leaves):
        way = torch.randn(leaf.shape, generator=gen, dtype=torch.float64)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + 1e-6 * way, at[i] - 1e-6 * way
        diff = (loss(*up) - loss(*down)) / 2e-6
        got = leaf.grad.cpu().double() * way
        assert abs(float(got.sum()) - diff) <= 1e-5 * float(got.abs().sum()) + 1e-6
    y = va.varlen_scan(leaves[0], leaves[1], c["cu"])[1].sum()               # the states alone
    y.backward()


def test_graph_streams_and_shared_workspace(va):
    m = make([300, 17, 500], 96, BF, F32)
    c = {n: x.to(DEV) for n, x in m.items()}
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)

    def both(ws=None):
        h, last = va.varlen_scan_fwd(c["x"], c["g"], c["cu"], c["h0"], h_last=True, workspace=ws)
        return (h, last) + va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"], c["h0"], c["dlast"], x_dtype=BF, workspace=ws)

    both(ws)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                       # two graphs on one workspace, replayed in turn
        graphs.append([torch.cuda.CUDAGraph()])
        with torch.cuda.graph(graphs[-1][0]):
            graphs[-1].append(both(ws))
    for _ in range(3):
        c["x"].copy_(torch.randn_like(c["x"]))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = both()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(both())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in got for a, b in zip(o, want))


def test_many_blocks_on_streams_at_once(va):
    """Calls that each fill the GPU, on three streams at once: blocks of one that wait for others of it share the SMs
    with the other calls' blocks."""
    sets = []
    for seed, lengths in ((1, [9000, 200, 3000]), (2, [12200]), (3, [40] * 305)):
        m = make(lengths, 2048, BF, BF, seed)
        sets.append({n: x.to(DEV) for n, x in m.items()})

    def both(c):
        h, last = va.varlen_scan_fwd(c["x"], c["g"], c["cu"], c["h0"], h_last=True)
        return (h, last) + va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"], c["h0"], c["dlast"])

    want = [both(c) for c in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, c in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(both(c))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


# many tiles for each block and few, copied rows and rows read in place
@pytest.mark.parametrize("T,D,xt,gt", [(3000, 64, F32, F32), (20000, 512, BF, BF), (20000, 511, BF, F32), (300, 6, F32, F32)])
def test_bounded_wait_runs_out_and_reports_timeout(va, T, D, xt, gt):
    """The test hook keeps the first tile's map back: the others' waits run out after a few milliseconds, the call
    reports it, and the next one is ordinary.  No GPU fault is involved."""
    m = make([T], D, xt, gt)
    c = {n: x.to(DEV) for n, x in m.items()}
    lib = va._lib.load()
    ws = torch.empty(lib.varlen_scan_workspace_size(T, 1, D), dtype=torch.uint8, device=DEV)
    h, _ = va.varlen_scan_fwd(c["x"], c["g"], c["cu"], check_status=True)
    want = va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"], x_dtype=xt, check_status=True)
    assert lib.varlen_test_stall_next_scan(5_000_000) == 0
    va.varlen_scan_fwd(c["x"], c["g"], c["cu"], workspace=ws)
    torch.cuda.synchronize()
    assert va.read_status(ws) == 6
    assert torch.equal(va.varlen_scan_fwd(c["x"], c["g"], c["cu"], workspace=ws, check_status=True)[0], h)
    assert lib.varlen_test_stall_next_scan(5_000_000) == 0
    va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"], x_dtype=xt, workspace=ws)
    torch.cuda.synchronize()
    assert va.read_status(ws) == 6
    again = va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"], x_dtype=xt, workspace=ws, check_status=True)
    assert all(x is y is None or torch.equal(x, y) for x, y in zip(again, want))
    assert lib.varlen_test_stall_next_scan(10) == 1 and lib.varlen_test_stall_next_scan(5_000_000_000) == 1


@pytest.mark.parametrize("D", [64, 66, 67])
@pytest.mark.parametrize("xt,gt", TYPES)
def test_states_that_only_decay(va, xt, gt, D):
    """Nothing but the states in: decays of 0.45 to 0.11 a row carry them over runs and tiles, where what a run keeps of
    a state is 1e-3 to 1e-15; a gradient at the last states alone goes back the same way.  Each row's value keeps its relative
    precision (the reference's own bound of it)."""
    lengths = [40, 1, 300, 129]
    m = make(lengths, D, xt, gt, seed=7)
    rates = torch.tensor([-0.8, -1.0, -1.2, -2.2, -0.4, -0.03])
    m["g"] = rates[torch.arange(D) % 6].expand(sum(lengths), D).contiguous().to(gt)
    m["x"].zero_()
    m["dh"].zero_()
    check(va, lengths, D, xt, gt, True, m=m)
    m["x"][:] = torch.randn(m["x"].shape, generator=torch.Generator().manual_seed(1)).to(xt)
    m["x"][:, ::2] = 0
    m["x"][45:48] = 1000                                     # large rows, then nothing
    m["dh"][300:303] = -1000
    check(va, lengths, D, xt, gt, True, m=m)


@pytest.mark.parametrize("D", [64, 67])
def test_outputs_over_the_other_input(va, D):
    """h over the decays, dx over the decays and their gradient over dh; views side by side in one buffer.  A row further
    on in the same rows is refused, and so is a gradient on h."""
    lengths = [300, 77]
    m = make(lengths, D, F32, F32)
    c = {n: x.to(DEV) for n, x in m.items()}
    T = sum(lengths)
    h, _ = va.varlen_scan_fwd(c["x"], c["g"], c["cu"])
    dx, dg, _ = va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"])
    over = c["g"].clone()
    va.varlen_scan_fwd(c["x"], over, c["cu"], out=over)
    assert torch.equal(over, h)
    dh, g = c["dh"].clone(), c["g"].clone()
    va.varlen_scan_bwd(dh, h, g, c["cu"], dx=g, dlog_decay=dh)
    assert torch.equal(g, dx) and torch.equal(dh, dg)
    one = torch.zeros(T, 4 * D, device=DEV)
    x, g, out = one[:, :D], one[:, D:2 * D], one[:, 2 * D:3 * D]
    x.copy_(c["x"]), g.copy_(c["g"])
    va.varlen_scan_fwd(x, g, c["cu"], out=out)
    rh, eh, _, _ = reference(m["x"], m["g"], lengths)
    close(out, rh, eh)
    assert bool((one[:, 3 * D:] == 0).all())
    long = torch.zeros(T + 1, D, device=DEV)
    for call in (lambda: va.varlen_scan_fwd(long[:T], c["g"], c["cu"], out=long[1:]),
                 lambda: va.varlen_scan_fwd(c["x"], long[1:], c["cu"], out=long[:T]),
                 lambda: va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"], dx=h),
                 lambda: va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"], dlog_decay=h),
                 lambda: va.varlen_scan_bwd(long[1:], h, c["g"], c["cu"], dx=long[:T])):
        with pytest.raises(va.VarlenError) as e:
            call()
        assert e.value.status == 1


@pytest.mark.parametrize("D", [64, 67, 130])
@pytest.mark.parametrize("lengths", [[1], [300, 1, 17, 129, 65], [1] * 40, [3, 1, 2] * 30, [2500]],
                         ids=lambda x: "-".join(map(str, x[:4])) + "x%d" % len(x))
def test_fp32_states_of_bf16_inputs(va, lengths, D):
    """bf16 x and decays with h, and dh, in fp32: h and dx as exact as with fp32 decays, and a dg that loses nothing by h's
    rounding (the reference's bound knows of none then)."""
    m = make(lengths, D, BF, BF)
    m["dh"] = torch.randn(m["dh"].shape, generator=torch.Generator().manual_seed(5))
    c = {n: x.to(DEV) for n, x in m.items()}
    h, last = va.varlen_scan_fwd(c["x"], c["g"], c["cu"], c["h0"], h_last=True, check_status=True, h_dtype=F32)
    assert h.dtype == F32
    rh, eh, rl, el = reference(m["x"], m["g"], lengths, m["h0"])
    close(h, rh, eh)
    close(last, rl, el)
    out = torch.empty_like(h)
    assert va.varlen_scan_fwd(c["x"], c["g"], c["cu"], c["h0"], out=out)[0] is out and torch.equal(out, h)
    narrow = va.varlen_scan_fwd(c["x"], c["g"], c["cu"], c["h0"])[0]
    assert narrow.dtype == BF and torch.equal(narrow, h.to(BF))             # the same states, rounded when stored
    got = va.varlen_scan_bwd(c["dh"], h, c["g"], c["cu"], c["h0"], c["dlast"], x_dtype=BF, check_status=True)
    assert got[0].dtype == got[1].dtype == BF
    dx, ex, dg, eg, d0, e0 = reference(m["x"], m["g"], lengths, m["h0"], m["dh"], m["dlast"])
    close(got[0], dx, ex)
    close(got[1], dg, eg)
    close(got[2], d0, e0)
    leaves = [c[n].clone().requires_grad_(True) for n in ("x", "g", "h0")]
    h, last = va.varlen_scan(leaves[0], leaves[1], c["cu"], leaves[2], h_dtype=F32)
    ((h * c["dh"]).sum() + (last * c["dlast"]).sum()).backward()
    assert all(torch.equal(a.grad, b) for a, b in zip(leaves, got))
    with pytest.raises(ValueError):
        va.varlen_scan_fwd(c["x"], c["g"].float(), c["cu"], h_dtype=BF)
    with pytest.raises(ValueError):
        va.varlen_scan_bwd(c["dh"].to(BF), c["dh"].to(BF), c["g"].float(), c["cu"], x_dtype=BF)


@pytest.mark.parametrize("D", [64, 67])
def test_states_that_grow(va, D):
    """Log decays above 0: a state that grows to e^20 of itself, and one next to 1 on either side."""
    lengths = [200, 40, 17]
    m = make(lengths, D, F32, F32, seed=3)
    m["g"] = torch.tensor([0.1, 0.05, 1e-3, -1e-3, 1e-7, -1e-7, 0.0215, -0.0217])[torch.arange(D) % 8].expand(sum(lengths), D).contiguous()
    check(va, lengths, D, F32, F32, True, m=m)
