"""The library called from several host threads at once, each with a stream of its own."""
import threading

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


def distill_job(va, T, V, K, seed):
    """One library call that repeats a distillation into the same tensors, and what it has to give."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = torch.randn(T, V, device=DEV, generator=g).bfloat16()
    ids = torch.randint(0, V, (T, K), device=DEV, generator=g, dtype=torch.int32)
    a = torch.randn(T, K, device=DEV, generator=g)
    loss, count = torch.empty(2, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    grad, ws = torch.empty_like(z), torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    out = (loss, count, grad)
    call = va._lib.load().varlen_token_distill

    def step(stream):
        return call(z.data_ptr(), 1, V, ids.data_ptr(), K, a.data_ptr(), 0, K, None, T, V, K, -100, 1.0,
                    loss.data_ptr(), count.data_ptr(), grad.data_ptr(), V, ws.data_ptr(), ws.numel(), stream)

    ref = va.token_distill(z, ids, a)
    return step, out, ref


def test_distillations_of_different_sizes_at_once(va):
    """Calls whose kernels are the same and whose shared memory differs (rows in five CTAs' slices of
    61 KB, in one CTA's of 1 KB with few and with many teacher entries): none may see another's
    launch settings.  The bindings release the interpreter's lock during a call."""
    jobs = [distill_job(va, *size) for size in ((2, 151936, 8, 1), (2, 500, 4, 2), (2, 700, 1024, 3), (2, 151936, 4, 4))]
    torch.cuda.synchronize()
    gate, codes = threading.Barrier(len(jobs)), [set() for _ in jobs]

    def run(i):
        stream = torch.cuda.Stream(DEV)
        step, raw = jobs[i][0], stream.cuda_stream
        gate.wait()
        for n in range(4000):
            codes[i].add(step(raw))
            if n % 200 == 199:
                stream.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}] * len(jobs), codes
    for _, out, ref in jobs:
        assert all(torch.equal(x, y) for x, y in zip(out, ref))
