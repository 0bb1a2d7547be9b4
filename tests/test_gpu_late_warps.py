"""Warps that come late (made to by kvs_debug_inject): whatever another warp does in the meantime, outputs are the same
bits."""
import numpy as np
import pytest

import test_gpu_chunk
from host_streamed_paged_gb300 import kvs
from test_gpu_prompt import make
from test_gpu_q4 import Filled
from test_gpu_window import check_prompt

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


@pytest.mark.parametrize("D,G", [(64, 1), (64, 3), (128, 2), (128, 8), (256, 3)])
def test_prompts_whose_products_are_issued_late(D, G):
    """Tiles of one key block beside tiles of two (a prompt's first rows, and short windows), several units a CTA: such a
    tile gives its queries back at once, and the next unit's may come before it has seen the second block's keys."""
    import torch
    lens = [3000, 100, 70, 128, 129, 64, 1] + [(29 * i) % 131 for i in range(200)]
    q, k, v, cu = make(lens, 4, G, D, "bf16" if D == 64 else "f16", seed=G)
    for window, sinks in ((60, 2), (1, 0), (100, 0)):
        want = kvs.prompt_attend(q, k, v, cu, window=window, sinks=sinks)
        check_prompt(*want, q, k, v, cu, "bf16" if D == 64 else "f16", D ** -0.5, window, sinks)
        for _ in range(2):
            kvs.kvs_debug_inject(None, kvs.KVS_FAULT_DEVICE_LATE, 1)
            for a, b in zip(kvs.prompt_attend(q, k, v, cu, window=window, sinks=sinks), want):
                assert torch.equal(a, b)
