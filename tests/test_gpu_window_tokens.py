"""Which calls with a window take token tiles, and their results where they do.

Token tiles pay for packs of many segments of at most 64 tokens.  In packs of longer ones, and in
small calls, they made the window's calls slower than one tile per segment.
"""
import numpy as np
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


def boundaries(lengths):
    cu, _, _, mx = op.build_metadata(lengths)
    return cu, torch.tensor(cu, dtype=torch.int32, device=DEV), int(mx)


def uniform(mean, n):
    rng = np.random.default_rng(mean * 1000 + n)
    return rng.integers(mean // 2, mean * 3 // 2 + 1, size=n).tolist()


def token_records(va, lengths, Hq, Hkv, d, w, s):
    """Token records (negative segment entries) in the forward's own map, and its record count."""
    cu, cud, mx = boundaries(lengths)
    T = int(cu[-1])
    q, k, v = (torch.zeros(T, h, d, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    ws = torch.zeros(va.workspace_size(T, len(lengths), Hq, Hkv, d, mx, False, window=w, sinks=s), dtype=torch.uint8,
                     device=DEV)
    va.varlen_attn_fwd(q, k, v, cud, mx, window=w, sinks=s, workspace=ws, check_status=True)
    raw = ws.cpu().numpy()
    n = int(raw[4:8].view(np.int32)[0])
    return int((raw[256:256 + 16 * n].view(np.int32).reshape(-1, 4)[:, 0] < 0).sum()), n


# no segment of at most 64 tokens, or few; many of them in a small call; few segments
@pytest.mark.parametrize("lengths,Hq,Hkv,d", [(uniform(160, 60), 8, 2, 64), (uniform(160, 190), 32, 8, 128),
                                              (uniform(80, 100), 8, 2, 64), (uniform(240, 40), 32, 8, 128),
                                              (uniform(40, 36), 2, 1, 64), (uniform(10, 32), 8, 2, 64)])
@pytest.mark.parametrize("w,s", [(16, 0), (20, 3)])
def test_medium_segments_and_small_calls_take_whole_tiles(va, lengths, Hq, Hkv, d, w, s):
    if max(lengths) - 1 <= w:
        w = max(lengths) - 2                     # (a window over the longest segment is the causal call)
    assert token_records(va, lengths, Hq, Hkv, d, w, s)[0] == 0


@pytest.mark.parametrize("lengths,Hq,Hkv,d", [(uniform(12, 400), 8, 2, 64), (uniform(40, 100), 32, 8, 128),
                                              (uniform(24, 300) + [900], 4, 2, 64)])
@pytest.mark.parametrize("w,s", [(5, 0), (9, 3)])
def test_many_short_segments_take_token_tiles(va, lengths, Hq, Hkv, d, w, s):
    assert token_records(va, lengths, Hq, Hkv, d, w, s)[0] > 0


@pytest.mark.parametrize("w,s", [(0, 1), (1, 0), (7, 70), (20, 5), (63, 1), (100, 30)])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (8, 8, 64)])
def test_runs_of_short_segments(va, w, s, Hq, Hkv, d):
    """Runs of segments of 1 to 64 tokens between longer ones, against the oracle."""
    rng = np.random.default_rng(w + 10 * s)
    lengths = [1, 64, 2, 63, 65, 300] + rng.integers(1, 65, size=40).tolist() + [130, 1, 1, 1, 90] + \
        rng.integers(1, 20, size=60).tolist()
    assert token_records(va, lengths, Hq, Hkv, d, w, s)[0] > 0
    cu, cud, mx = boundaries(lengths)
    q, k, v, do = si.tensors(int(cu[-1]), Hq, Hkv, d, seed_offset=31)
    qd, kd, vd, dod = (x.to(DEV) for x in (q, k, v, do))
    o, lse = va.varlen_attn_fwd(qd, kd, vd, cud, mx, window=w, sinks=s, check_status=True)
    got = va.varlen_attn_bwd(qd, kd, vd, o, lse, dod, cud, mx, window=w, sinks=s, check_status=True)
    qq, kk, vv, dd = (si.to_f64(x) for x in (q, k, v, do))
    ro, rl = oa.varlen_forward(qq, kk, vv, cu, window=w, sinks=s)
    wl.assert_close_outputs(o.double().cpu().numpy(), lse.double().cpu().numpy(), ro, rl)
    wl.assert_close_grads(tuple(x.double().cpu().numpy() for x in got),
                          oa.varlen_backward(qq, kk, vv, ro, rl, dd, cu, window=w, sinks=s))
