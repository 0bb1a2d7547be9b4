"""Q4Cache's workspaces: each thread has its own, which goes with the thread."""
import gc
import threading

import pytest

from test_gpu_q4 import Filled

pytestmark = pytest.mark.gpu


def test_workspaces_go_with_their_threads():
    import torch
    f = Filled([300, 70], 2, 128, 64, seed=15, dt="f16")
    q = torch.randn(2, 1, 8, 128).half().cuda()
    out, lse = f.cache.attend(f.table_t, f.lens_t, q)
    torch.cuda.synchronize()
    n = 8
    for _ in range(2):
        gc.collect()
        before, at_once, same = torch.cuda.memory_allocated(), threading.Barrier(n), []

        def work():
            at_once.wait(60)
            o, z = f.cache.attend(f.table_t, f.lens_t, q)
            torch.cuda.synchronize()
            same.append(torch.equal(o, out) and torch.equal(z, lse))
            at_once.wait(60)

        threads = [threading.Thread(target=work) for _ in range(n)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        gc.collect()
        assert same == [True] * n
        assert torch.cuda.memory_allocated() == before
