"""Batches whose prefix sums bring a kernel's shared memory near 48 KB, the limit without an opt-in: every size up to
4096 sequences runs, whichever call of a process comes first (so each runs in a process of its own)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
CHILD = """
import sys
sys.path[:0] = [{here!r}, {root!r}]
import math
import numpy as np
import torch
import batch_ref as ref
from test_gpu_q4 import S_ERR, Filled, _t, check_attend

call, D, G, dt, n = {case!r}
rng = np.random.default_rng(n)
f = Filled([int(x) for x in rng.integers(0, 40, n)], 1, D, 32, seed=9, dt=dt)
q = torch.randn(n, 1, G, D, generator=torch.Generator().manual_seed(8)).to(_t(dt)).cuda()
scale = 1 / math.sqrt(D)
if call == "attend":
    out, lse = f.cache.attend(f.table_t, f.lens_t, q)
    check_attend(out, lse, q, f, dt, scale)
else:
    lse = torch.full((n, 1, G), 3.0, device="cuda")
    w = f.cache.weights(f.table_t, f.lens_t, q, lse, width=64).double().cpu().numpy()
    for i, T in enumerate(f.lens):
        want = np.zeros((1, 64))
        want[:, :T] = ref.cache_weights(q[i].double().cpu().numpy(), f.seq(i)[0], np.full((1, G), 3.0), scale)
        assert (np.abs(w[i] - want) <= (S_ERR + 1e-5) * want + 1e-37).all(), i
print("done")
"""


@pytest.mark.parametrize("case", [("attend", 64, 16, "f16", 480), ("attend", 64, 16, "bf16", 511), ("attend", 64, 2, "f16", 1023),
                                  ("attend", 64, 2, "f32", 992), ("weights", 64, 2, "f16", 3808), ("weights", 128, 2, "f16", 2687),
                                  ("attend", 64, 1, "f16", 4096)])
def test_first_call_of_a_process(case):
    code = CHILD.format(here=HERE, root=os.path.dirname(HERE), case=case)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-1500:]
