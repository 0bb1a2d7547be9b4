"""Around the windowed calls: what their lse is not for, pages that rows see and that are not there, precision."""
import math

import numpy as np
import pytest

import batch_ref as ref
from host_streamed_paged_gb300 import kvs
from test_gpu_prompt import make
from test_gpu_q4 import Filled

pytestmark = pytest.mark.gpu


def test_weights_count_every_key_whatever_the_lse():
    """As the header states them: exp(scale q k - lse) for all keys up to the row's, so beside a windowed lse they add up
    to more than the rows' number.  Tolerance: scores off by 2e-4 (their fp32 sums), a sum's relative error below that."""
    import torch
    q, k, v, cu = make([500], 1, 2, 64, "f16", seed=3)
    full, windowed = (kvs.prompt_attend(q, k, v, cu, window=w, sinks=4)[1] for w in (0, 64))
    w = kvs.prompt_weights(q, k, windowed, cu, 500)[0].double().cpu().numpy()
    q64, k64 = q.double().cpu().numpy(), k.double().cpu().numpy()
    want = ref.prompt_weights(q64, k64, windowed.double().cpu().numpy(), 64 ** -0.5)
    assert np.allclose(w, want, rtol=5e-4, atol=0) and w.sum() > 1.5 * 1000
    assert abs(kvs.prompt_weights(q, k, full, cu, 500).double().sum().item() - 1000) < 0.5
    f = Filled([600], 1, 64, 64, seed=2, dt="f16")
    x = torch.randn(1, 1, 4, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    lse = [f.cache.attend(f.table_t, f.lens_t, x, window=w, sinks=4)[1] for w in (0, 100)]
    w = [f.cache.weights(f.table_t, f.lens_t, x, z, width=600)[0].double().cpu().numpy() for z in lse]
    assert np.allclose(w[1], ref.cache_weights(x[0].double().cpu().numpy(), f.seq(0)[0], lse[1][0].double().cpu().numpy(), 0.125), rtol=1e-3, atol=0)
    assert abs(w[0].sum() - 4) < 4e-3 and w[1].sum() > 6
