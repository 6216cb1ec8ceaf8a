"""Calls straight after one another, each reading what the one before it wrote.

The library's kernels may become resident while the kernel before them still runs, so whatever a
call reads of another's results has to be read after that one has ended.
"""
import pytest
import torch

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


@pytest.mark.parametrize("T,V,D", [(700, 50, 64), (5003, 300, 40), (20000, 1000, 128)])
def test_gradients_in_one_workspace_with_new_ids_each_time(va, T, V, D):
    """Sixteen gradients in a row through one workspace, whose sorted pairs every call overwrites: bit-equal
    to the same gradients each on its own."""
    g = torch.Generator(device=DEV).manual_seed(T)
    ids = [torch.randint(0, V, (T,), device=DEV, generator=g, dtype=torch.int32) for _ in range(16)]
    dout = torch.randn(T, D, device=DEV, generator=g)
    ws = torch.zeros(va._lib.load().varlen_embed_bwd_workspace_size(T, D), dtype=torch.uint8, device=DEV)
    ref = []
    for x in ids:
        ref.append(va.embed_bwd(dout, x, V, check_status=True))
        torch.cuda.synchronize()
    for accumulate in (False, True):
        outs = [torch.zeros(V, D, device=DEV) for _ in ids]
        torch.cuda.synchronize()
        for x, o in zip(ids, outs):
            va.embed_bwd(dout, x, V, dtable=o, accumulate=accumulate, workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
