"""Windows with sinks at the ends of their ranges."""
import math

import pytest
import torch

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
