"""The distillation's failure path: a bounded wait that runs out.

The test hook varlen_test_stall_next_distill lets the first CTA of every row's cluster load nothing, so
its waits, and those of the CTAs that want its sums, run out after a few milliseconds.  No GPU
fault is involved; the call reports VA_ERR_TIMEOUT and the next one is ordinary.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
VA_ERR_TIMEOUT = 6


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_sequence_varlen_gb300 import build as b
    b.build()
    import packed_sequence_varlen_gb300 as pkg
    pkg._lib.load()
    return pkg


# rows in one CTA (one and several rows each, with and without a gradient), in clusters of five and of eight
@pytest.mark.parametrize("T,V,K,dtype,with_grad", [(5, 500, 4, torch.float32, True), (3001, 600, 9, torch.bfloat16, True),
                                                   (3001, 600, 9, torch.bfloat16, False),
                                                   (301, 151936, 8, torch.bfloat16, True),
                                                   (40, 300001, 5, torch.float32, True)])
def test_bounded_wait_runs_out_and_reports_timeout(va, T, V, K, dtype, with_grad):
    g = torch.Generator(device=DEV).manual_seed(T + V)
    z = torch.randn(T, V, device=DEV, generator=g).to(dtype)
    ids = torch.randint(0, V, (T, K), device=DEV, generator=g, dtype=torch.int32)
    a = torch.randn(T, K, device=DEV, generator=g)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    ref = va.token_distill(z, ids, a, grad=with_grad, check_status=True)
    lib = va._lib.load()
    assert lib.varlen_test_stall_next_distill(5_000_000) == 0        # 5 ms
    loss, _, _ = va.token_distill(z, ids, a, grad=with_grad, workspace=ws)
    torch.cuda.synchronize()
    assert va.read_status(ws) == VA_ERR_TIMEOUT
    assert all(math.isnan(x) for x in loss.tolist())
    # the hook is one-shot and the context is still usable
    again = va.token_distill(z, ids, a, grad=with_grad, workspace=ws, check_status=True)
    assert all(x is y is None or torch.equal(x, y) for x, y in zip(again, ref))


def test_stall_hook_rejects_limits_outside_its_range(va):
    lib = va._lib.load()
    assert lib.varlen_test_stall_next_distill(10) == 1
    assert lib.varlen_test_stall_next_distill(5_000_000_000) == 1
