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


def test_targets_written_just_before_the_distillation(va):
    """Next-token targets into one buffer and the distillation over them, again and again: each sees its own."""
    T, V, K = 3000, 64, 4
    g = torch.Generator(device=DEV).manual_seed(1)
    z, a = torch.randn(T, V, device=DEV, generator=g), torch.randn(T, K, device=DEV, generator=g)
    tid = torch.randint(0, V, (T, K), device=DEV, generator=g, dtype=torch.int32)
    cus = [torch.tensor(sorted({0, *range(7 + i, T, 11 + 3 * i), T}), dtype=torch.int32, device=DEV) for i in range(12)]
    ids = torch.randint(0, V, (T,), device=DEV, generator=g, dtype=torch.int32)
    torch.cuda.synchronize()
    got = [va.token_distill(z, tid, a, va.loss_targets(ids, cu)) for cu in cus]
    torch.cuda.synchronize()
    for cu, (loss, count, grad) in zip(cus, got):
        tg = va.loss_targets(ids, cu)
        torch.cuda.synchronize()
        l2, c2, g2 = va.token_distill(z, tid, a, tg, check_status=True)
        assert torch.equal(loss, l2) and torch.equal(count, c2) and torch.equal(grad, g2)
        assert int(count.item()) == T - (cu.numel() - 1)
