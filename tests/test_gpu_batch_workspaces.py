"""Caches of one device share a workspace per stream and thread."""
import gc
import threading

import pytest

from host_streamed_paged_gb300 import kvs
from test_gpu_chunk import queries
from test_gpu_q4 import Filled

pytestmark = pytest.mark.gpu


def calls(D, seed):
    """A cache with an attend and a chunk of its own, as a function of nothing that runs both."""
    import torch
    f = Filled([900, 70, 3000], 2, D, 64, seed=seed, dt="f16")
    q, cu = queries([60, 1, 130], 8, D, "f16", seed=seed)
    one = torch.randn(3, 1, 8, D, generator=torch.Generator().manual_seed(seed)).half().cuda()
    return f, lambda: (*f.cache.attend(f.table_t, f.lens_t, one), f.cache.attend_chunk(f.table_t, f.lens_t, cu, q))


def test_many_caches_hold_one_workspace_and_give_it_back():
    import torch
    sides = [calls(D, i) for i, D in enumerate((128, 64, 256, 128, 128))]
    need = max(max(kvs.kvs_q4_chunk_workspace(f.cache.pool), kvs.kvs_q4_query_sizes(f.cache.pool, 1, 8, kvs.KVS_F16)[1]) for f, _ in sides)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    gc.collect()
    before = torch.cuda.memory_allocated()

    def held():
        torch.cuda.synchronize()
        gc.collect()
        return torch.cuda.memory_allocated() - before

    for stream, times in ((torch.cuda.current_stream(), 1), (other, 2)):
        with torch.cuda.stream(stream):
            for _, call in sides:
                call()
        assert times * need <= held() <= times * (need + (2 << 20))  # (the allocator rounds up to 2 MB)
    for f, call in sides[1:]:
        f.cache._spaces = None
    assert held() >= 2 * need  # the first still has them
    sides[0][0].cache._spaces = None
    assert held() == 0


def test_caches_in_turn_on_streams_and_threads():
    import torch
    sides = [calls(D, i) for i, D in enumerate((128, 64, 256))]
    want = [call() for _, call in sides]
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        for _ in range(10):
            with torch.cuda.stream(stream):
                got = [call() for _, call in sides]
            stream.synchronize()
            for a, b in zip(got, want):
                wrong.extend(i for i, (x, y) in enumerate(zip(a, b)) if not torch.equal(x, y))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    work()
    for t in threads:
        t.join()
    assert not wrong
