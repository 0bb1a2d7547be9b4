"""Scales of the 4-bit cache's calls beside the usual positive one: zero, tiny and negative (every finite one is taken).

Bounds as in test_gpu_q4: the scores' error is at most S_ERR for |scale| up to 1 / sqrt(D), and none at scale 0.
"""
import math

import numpy as np
import pytest

import batch_ref as ref
from test_gpu_q4 import DT, LENS, S_ERR, Filled, _t, check_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-44, 1e-30, -0.05])
@pytest.mark.parametrize("D,P,Hk,G,R", [(64, 32, 2, 3, 1), (128, 64, 1, 4, 3), (256, 256, 1, 6, 2)])
def test_attend_and_weights_take_any_finite_scale(D, P, Hk, G, R, scale, dt):
    """At scale 0 every seen token has the same weight: out is the mean of their V, lse the logarithm of their number."""
    import torch
    f = Filled(LENS, Hk, D, P, seed=D + R, dt=dt)
    q = torch.randn(len(LENS), R, Hk * G, D, generator=torch.Generator().manual_seed(5)).to(_t(dt)).cuda()
    out, lse = f.cache.attend(f.table_t, f.lens_t, q, scale=scale)
    check_attend(out, lse, q, f, dt, scale)
    if abs(scale) < 1e-20:
        seen = torch.tensor([[max(0, n - R + 1 + r) for r in range(R)] for n in LENS], dtype=torch.float64)
        want = seen.log().view(len(LENS), R, 1).expand(-1, -1, Hk * G)
        some = want > -math.inf
        assert (lse.double().cpu()[some] - want[some]).abs().max() <= 1e-5 and (lse.cpu()[~some] == -math.inf).all()
    width = f.table.shape[1] * P
    got = f.cache.weights(f.table_t, f.lens_t, q, lse, width=width, scale=scale).double().cpu().numpy()
    qn, zn = q.double().cpu().numpy(), lse.double().cpu().numpy()
    for i, T in enumerate(LENS):
        w = np.zeros((Hk, width))
        w[:, :T] = ref.cache_weights(qn[i], f.seq(i)[0], zn[i], scale)
        assert (np.abs(got[i] - w) <= (S_ERR + 1e-5) * w + 1e-37).all()


@pytest.mark.parametrize("scale", [0.0, 0.1])
def test_queries_of_zeros(scale):
    import torch
    f = Filled([77, 3], 1, 128, 64, seed=2)
    q = torch.zeros(2, 1, 4, 128, device="cuda")
    out, lse = f.cache.attend(f.table_t, f.lens_t, q, scale=scale)
    check_attend(out, lse, q, f, "f32", scale)
    assert math.isclose(float(lse[0, 0, 0]), math.log(77), abs_tol=1e-5)
