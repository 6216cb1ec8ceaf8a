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


def test_sizes_past_the_kernels_indexes(lib):
    """Sizes that the 32-bit arguments would wrap, or whose columns exceed the gradient's grid."""
    import packed_sequence_varlen_gb300 as va
    assert lib.varlen_embed_fwd(P, 1, 1 << 31, P, 8, 100, (1 << 26) + 1, 1.0, P, 1 << 31, None, None) == 1
    assert lib.varlen_embed_bwd(None, 0, 1 << 31, None, 0, 1 << 30, 64, 1.0, P, 0, 1 << 31, 0, P, 1 << 40, None) == 1
    assert lib.varlen_embed_bwd(None, 0, 1 << 31, None, 0, 4, 1 << 29, 1.0, P, 0, 1 << 31, 0, P, 1 << 40, None) == 1
    with pytest.raises(ValueError):
        va._check_sizes(num_rows=2 ** 32 + 4)
    assert va._int32(2 ** 32) == 2 ** 31 - 1 and va._int32(2 ** 32 + 5) == 2 ** 31 - 1 and va._int32(-2 ** 40) == -2 ** 31
    assert va._int32(-1) == -1 and va._int32(512) == 512
    # 2^32 sinks are all tokens (a wrapped count would be none, with a smaller or other workspace)
    big = dict(T=65536, B=1, Hq=12, Hkv=1, d=128, max_seqlen=65536, for_bwd=True)
    assert va.workspace_size(**big, window=1023, sinks=2 ** 32) == va.workspace_size(**big, window=1023, sinks=65536)
    assert va.workspace_size(**big, window=1023, sinks=2 ** 32 + 4) != va.workspace_size(**big, window=1023, sinks=4)
