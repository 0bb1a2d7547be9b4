"""What the batch operators keep beyond their types' roundings."""
import pytest

pytestmark = pytest.mark.gpu


def test_weights_of_a_long_prompt_add_up_in_two_levels():
    """80000 equal terms for the first key: a term's error is that of exp (below 8e-7 for an lse below 7), a sum's half a
    step an addition: 16 in a tile of 128 rows, 625 tiles, 8 at the end.  (In one chain of 10000 additions equal terms
    are rounded the same way for long stretches: 1e-4.)"""
    import numpy as np
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
