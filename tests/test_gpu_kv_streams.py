"""Attention calls share scratch: they follow one another whatever streams they run on, streams of one
handle among them (the per-thread stream of two host threads that take turns)."""
import concurrent.futures as futures

import pytest
import torch

import adapter_linear_gb300 as al
import _kv_reference as R

pytestmark = pytest.mark.gpu

PER_THREAD = 2      # cudaStreamPerThread: each host thread's own stream under one handle


@pytest.mark.parametrize("new", [[1, 1], [90, 60]])
def test_per_thread_streams_share_a_cache(new):
    lens = [20000, 15000]
    p, q = (R.Paged(al, al.LORA_KV_INT8, lens, new, 2, 128, 16, seed=230) for _ in range(2))
    Qs = [torch.randn(p.T, 8, 128, device="cuda").to(torch.bfloat16) for _ in range(2)]
    alone = [q.cache.attention(x, q.batch) for x in Qs]
    got = [[(torch.empty_like(x), torch.empty(p.T, 8, device="cuda")) for _ in range(20)] for x in Qs]
    torch.cuda.synchronize()

    def call(thread, i):
        torch.cuda.set_device(0)
        O, lse = got[thread][i]
        p.cache.attention(Qs[thread], p.batch, O=O, lse=lse, stream=PER_THREAD)

    with futures.ThreadPoolExecutor(1) as a, futures.ThreadPoolExecutor(1) as b:
        for i in range(20):
            for thread, pool in enumerate((a, b)):
                pool.submit(call, thread, i).result()
        assert p.cache.check_errors() == al.LORA_OK          # waits for all of them
        for thread in range(2):
            for O, lse in got[thread]:
                assert torch.equal(O.view(torch.int16), alone[thread][0].view(torch.int16))
                assert torch.equal(lse, alone[thread][1])


def test_check_errors_waits_for_writes_on_per_thread_streams():
    """A bad table entry written through by the first of two threads is reported, whichever wrote last."""
    p = R.Paged(al, al.LORA_KV_INT8, [6000], [5000], 8, 128, 16, seed=240)
    K, V = (torch.randn(p.T, 8, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    bad = p.table.clone()
    bad[0, 374] = p.cache.num_pages          # the last tokens'
    wrong = al.KvBatch(bad, p.batch.start, p.batch.kv_len, p.T, 5000)
    small = al.KvBatch(p.table, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), p.batch.kv_len, 1, 1)
    torch.cuda.synchronize()
    with futures.ThreadPoolExecutor(1) as a, futures.ThreadPoolExecutor(1) as b:
        for _ in range(10):
            a.submit(p.cache.write, K, V, wrong, PER_THREAD).result()
            b.submit(p.cache.write, K[:1], V[:1], small, PER_THREAD).result()
            assert p.cache.check_errors() == al.LORA_ERR_RANGE
            assert p.cache.check_errors() == al.LORA_OK


@pytest.mark.parametrize("as_handle", [False, True])
def test_memory_of_a_call_on_another_stream(as_handle):
    """Outputs belong to the stream that writes them, and inputs dropped after the call are not handed
    out again while it runs."""
    p = R.Paged(al, al.LORA_KV_INT8, [300, 200], [50, 30], 2, 128, 16, seed=250)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_handle else side
    rows = [torch.randn(p.T, h, 128, device="cuda").to(torch.bfloat16) for h in (8, 2, 2)]
    p.cache.write(rows[1], rows[2], p.batch)                 # (kernels loaded, scratch there)
    p.cache.attention(rows[0], p.batch)
    p.cache.read(p.batch)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)                       # some 200 ms
    O, lse = p.cache.attention(rows[0], p.batch, stream=stream)
    p.cache.write(rows[1], rows[2], p.batch, stream=stream)
    K, V = p.cache.read(p.batch, stream=stream)
    outputs, inputs = [O, lse, K, V], rows
    used = {x.data_ptr() for x in outputs + inputs}
    like = [(x.shape, x.dtype) for x in outputs + inputs]
    del O, lse, K, V, rows, outputs, inputs
    assert not side.query()                                  # still asleep
    fresh = [torch.empty(s, dtype=d, device="cuda") for s, d in like]
    assert not used & {x.data_ptr() for x in fresh}
    side.synchronize()
    assert p.cache.check_errors() == al.LORA_OK
