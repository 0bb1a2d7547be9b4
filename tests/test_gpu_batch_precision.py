"""What the batch operators keep beyond their types' roundings."""
import math

import numpy as np
import pytest

import batch_ref as ref
from test_gpu_q4 import Filled

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


@pytest.mark.parametrize("D,Hk,G,R", [(64, 1, 4, 1), (128, 2, 4, 1), (128, 1, 8, 2), (256, 1, 6, 1)])
def test_fp32_attention_keeps_fp32(D, Hk, G, R):
    """Norm-wise.  An output is sum p v over tokens whose errors are independent, so ||err|| / ||out|| is the root mean
    square of the weights' relative errors.  Those of an fp32 call, for unit-normal rows and queries of 1.5:
      scores: a query is f16 hi + lo, cut 2^-22 of the row's largest element (4.5) and, uniform in it, 2^-24 on
        average; over sqrt(D) products of 1 and a scale of 1 / sqrt(D): 3e-7; fp32 block sums of up to 4 sqrt(D)
        (2^-24 of them, 1 / sqrt(D)): 2e-7;
      exponent: half a step of an argument below 16, uniform: 2^-20 / 2 ln 2 / sqrt(3) = 2e-7; ex2: 2^-22 = 2.4e-7;
      weight x scale as hi + lo pairs: 2^-22 / sqrt(3) = 1.4e-7; sums of O cut at 2^-23 of it a step, over the tens of
        tiles of a worker: 5e-7.
    Together below 1e-6 (root of the squares; 1.6e-6 added up): 2e-6.  (Codes of 0 .. 15 as f16 subnormals, the form of
    16-bit calls, leave 17 bits of a sum: 7e-6.)  lse: three roundings at up to 16 (2^-21 each) and the scores': 3e-6."""
    import torch
    f = Filled([4096, 1031, 70], Hk, D, 64, seed=D + R)
    q = (1.5 * torch.randn(3, R, Hk * G, D, generator=torch.Generator().manual_seed(6))).cuda()
    out, lse = f.cache.attend(f.table_t, f.lens_t, q)
    o, z, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for i in range(3):
        k, v, _ = f.seq(i)
        ro, rz, _ = ref.attend(qn[i], k, v, 1 / math.sqrt(D))
        rel = np.linalg.norm(o[i] - ro) / np.linalg.norm(ro)
        assert rel <= 2e-6, (i, rel)
        assert np.abs(z[i] - rz).max() <= 3e-6, (i, np.abs(z[i] - rz).max())
