"""What the batch operators keep beyond their types' roundings."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def test_weights_of_a_long_prompt_add_up_in_two_levels():
    """80000 equal terms for the first key: a term's error is that of exp (below 8e-7 for an lse below 7), a sum's half a
    step an addition: 16 in a tile of 128 rows, 625 tiles, 8 at the end.  (In one chain of 10000 additions equal terms
    are rounded the same way for long stretches: 1e-4.)"""
    import torch
    from host_streamed_paged_gb300 import kvs
    L, Hk, G, D = 20000, 8, 4, 64
    q = torch.zeros(L, Hk * G, D, dtype=torch.float16, device="cuda")
    k = torch.zeros(L, Hk, D, dtype=torch.float16, device="cuda")
    c = torch.tensor([0.3, 1.0, 2.5, 3.1, 4.0, 5.3, 6.1, 0.7])
    lse = c.repeat_interleave(G).view(1, -1).expand(L, -1).contiguous().cuda()
    w = kvs.prompt_weights(q, k, lse, torch.tensor([0, L], dtype=torch.int32, device="cuda"), L)[0].double().cpu().numpy()
    want = np.exp(-lse[0, ::G].double().cpu().numpy())[:, None] * (G * (L - np.arange(L)))[None]
    tol = (16 + L * G / 128 + 8) * 2.0 ** -24 + 8e-7
    assert (np.abs(w / want - 1) <= tol).all(), np.abs(w / want - 1).max(1)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_small_prompt_weights_reach_the_output(D):
    """One key of weight 1 and value 0, thousands of weight e^-18.5 and value 1.  Weights enter the second product as
    f16 times 2^7: what lies below f16's smallest step is half of 2^-24 2^-7 per key, i 2^-32 for row i in all; the
    output has half a step of its own, 2^-11 of it or 2^-25, and the scores are exact."""
    import torch
    from host_streamed_paged_gb300 import kvs
    L = 6000
    q, k, v = (torch.zeros(L, 1, D, dtype=torch.float16, device="cuda") for _ in range(3))
    q[..., 0] = 1.0
    k[1:, :, 0] = -18.5
    v[1:] = 1.0
    out, lse = kvs.prompt_attend(q, k, v, torch.tensor([0, L], dtype=torch.int32, device="cuda"), scale=1.0)
    i = np.arange(L, dtype=np.float64)[:, None]
    total = 1 + i * math.exp(-18.5)
    want = i * math.exp(-18.5) / total
    got = out[:, 0].double().cpu().numpy()
    # ex2 of an argument of 27 in fp32: 2^-20 ln 2 and 2^-22, below 2^-19 of each weight
    tol = i * 2.0 ** -32 + 2.0 ** -25 + (2.0 ** -11 + 2.0 ** -19) * want
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()
    # lse: the sum is 1 and a little throughout, held in two fp32 numbers with one addition to either for each block of 64
    # keys (128 at D 256); each is off by at most half a step, 2^-24 of a sum that the small weights never double, and all
    # blocks may be off to the same side
    assert np.abs(lse[:, 0].double().cpu().numpy() - np.log(total[:, 0])).max() <= 1e-6 + math.ceil(L / 64) * 2.0 ** -24
