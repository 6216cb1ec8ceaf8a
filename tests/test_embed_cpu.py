"""Host-side refusals of the embedding entry points (no device work)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    return pkg._lib.load()


P = ctypes.c_void_p(256)


def test_forward_refusals(lib):
    def call(table=P, dtype=1, trs=64, ids=P, T=8, V=100, D=64, scale=1.0, out=P, ors=64):
        return lib.varlen_embed_fwd(table, dtype, trs, ids, T, V, D, scale, out, ors, None, None)

    for kw in (dict(table=None), dict(ids=None), dict(out=None), dict(dtype=2), dict(trs=63), dict(ors=63), dict(T=-1),
               dict(T=1 << 30), dict(V=0), dict(V=2 ** 31 - 1), dict(D=0), dict(scale=float("nan")),
               dict(scale=float("-inf")), dict(table=ctypes.c_void_p(257)), dict(out=ctypes.c_void_p(258), dtype=0)):
        assert call(**kw) == 1, kw
    assert call(T=0, ids=None) == 0                          # nothing to do, nothing launched


def test_backward_refusals(lib):
    n = lib.varlen_embed_bwd_workspace_size(8, 64)

    def call(dout=P, dtype=1, irs=64, ids=P, T=8, V=100, D=64, scale=1.0, dtable=P, odt=0, ors=64, ws=P, nws=n):
        return lib.varlen_embed_bwd(dout, dtype, irs, ids, T, V, D, scale, dtable, odt, ors, 0, ws, nws, None)

    for kw in (dict(dout=None), dict(ids=None), dict(dtable=None), dict(ws=None), dict(dtype=-1), dict(odt=2),
               dict(irs=63), dict(ors=1), dict(T=-1), dict(V=0), dict(D=0), dict(scale=float("inf")),
               dict(ws=ctypes.c_void_p(264)), dict(dtable=ctypes.c_void_p(258))):
        assert call(**kw) == 1, kw
    assert call(nws=n - 1) == 3
    assert lib.varlen_embed_bwd_workspace_size(-1, 64) == 0 and lib.varlen_embed_bwd_workspace_size(8, 0) == 0


def test_python_refusals_without_a_gpu(lib):
    import packed_sequence_varlen_gb300 as va
    with pytest.raises(ValueError):
        va.embed_fwd(torch.zeros(4, 8), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        va.embed_bwd(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32), 4)
