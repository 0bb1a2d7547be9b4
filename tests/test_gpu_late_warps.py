"""Warps that come late (made to by kvs_debug_inject): whatever another warp does in the meantime, outputs are the same
bits."""
import numpy as np
import pytest

import test_gpu_chunk
from host_streamed_paged_gb300 import kvs
from test_gpu_q4 import Filled

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def disarm():
    yield
    kvs.kvs_debug_inject(None, kvs.KVS_FAULT_NONE, 0)


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 3), (128, 8), (256, 5)])
def test_chunks_whose_outputs_are_read_late(D, G, window):
    """Several units a worker, of one query tile and of two, an odd or even number of blocks each, whole and cut: the next
    unit's first P V waits until both warpgroups have read the last one's output."""
    import torch
    rng = np.random.default_rng(D + G)
    lens = rng.integers(1, 300, 250).tolist() + [3000, 2500]
    rows = [int(rng.integers(0, min(n, 90) + 1)) for n in lens]
    f = Filled(lens, 2, D, 32, seed=G, dt="f16")
    out, lse, q, cu = test_gpu_chunk.run(f, rows, 2, G, D, "f16", window=window, sinks=3)
    c = cu.tolist()
    s = slice(c[0], c[-1])
    for _ in range(3):
        kvs.kvs_debug_inject(None, kvs.KVS_FAULT_DEVICE_LATE, 1)
        z = torch.full_like(lse, 7.0)
        got = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q, lse=z, window=window, sinks=3)
        assert torch.equal(got[s], out[s]) and torch.equal(z, lse)
