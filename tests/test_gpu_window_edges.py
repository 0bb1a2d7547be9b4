"""Around the windowed calls: what their lse is not for, and pages that rows see and that are not there."""
import numpy as np
import pytest

import batch_ref as ref
from host_streamed_paged_gb300 import kvs
from test_gpu_chunk import queries
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


@pytest.mark.parametrize("R", [1, 3])
@pytest.mark.parametrize("P", [32, 64, 256])
@pytest.mark.parametrize("which", ["last", "first", "window"])
def test_a_page_that_steps_see_and_that_is_outside_the_pool(which, P, R):
    """The last token's, the first tokens' or the one where the window begins: that sequence's outputs are NaN."""
    import torch
    lens, window, sinks = [1500, 5000, 90], 200, 4
    f = Filled(lens, 2, 128, P, seed=4, dt="f16")
    q = torch.randn(3, R, 8, 128, generator=torch.Generator().manual_seed(5)).half().cuda()
    want = f.cache.attend(f.table_t, f.lens_t, q, window=window, sinks=sinks)
    token = {"last": 4999, "first": 3, "window": 5000 - R - window + 1}[which]
    for number in (-1, f.cache.n_pages, 1 << 30):
        table = f.table_t.clone()
        table[1, token // P] = number
        out, lse = f.cache.attend(table, f.lens_t, q, window=window, sinks=sinks)
        assert out[1].isnan().all() and lse[1].isnan().all()
        for i in (0, 2):
            assert torch.equal(out[i], want[0][i]) and torch.equal(lse[i], want[1][i])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [32, 256])
def test_a_page_that_chunks_see_and_that_is_outside_the_pool(P, D):
    """Under a window: every row that sees one of its tokens is NaN, other sequences are as they were."""
    import torch
    import window_ref
    lens, rows, window, sinks = [700, 3000, 90], [70, 300, 5], 200, 4
    f = Filled(lens, 1, D, P, seed=4, dt="f16")
    q, cu = queries(rows, 4, D, "f16")
    want, c = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q, window=window, sinks=sinks), cu.tolist()
    see = window_ref.sees(2700 + np.arange(300), 3000, window, sinks)
    for token in (2999, 3, 2700, 2600):
        table, page = f.table_t.clone(), token // P
        table[1, page] = f.cache.n_pages
        lse = torch.zeros(q.shape[:2], device="cuda")
        got = f.cache.attend_chunk(table, f.lens_t, cu, q, lse=lse, window=window, sinks=sinks)
        hit = torch.from_numpy(see[:, page * P:(page + 1) * P].any(1)).cuda()
        assert hit.any() and got[c[1]:c[2]][hit].isnan().all() and lse[c[1]:c[2]][hit].isnan().all()
        for i in (0, 2):
            assert torch.equal(got[c[i]:c[i + 1]], want[c[i]:c[i + 1]])


@pytest.mark.parametrize("n", [1, 20, 33, 70])
@pytest.mark.parametrize("D,P", [(64, 32), (128, 32), (128, 256), (256, 64)])
def test_rows_that_see_nothing_but_nan(D, P, n):
    """Short sequences of a page outside the pool, or of NaN keys alone: no other key gives their rows a reference."""
    import torch
    f = Filled([n, n, 50], 1, D, P, seed=4, dt="f16")
    q, cu = queries([n, 1, 5], 4, D, "f16")
    want, c = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q), cu.tolist()
    pages = f.table_t.clone()
    pages[:2, :-(-n // P)] = -1
    k = f.k.clone()
    k[:2 * n] = float("nan")
    for what in ("pages", "keys"):
        if what == "keys":
            f.cache.append(torch.from_numpy(f.slots).cuda(), k.cuda(), f.v.cuda())
        lse = torch.zeros(q.shape[:2], device="cuda")
        got = f.cache.attend_chunk(pages if what == "pages" else f.table_t, f.lens_t, cu, q, lse=lse)
        assert got[:c[2]].isnan().all() and lse[:c[2]].isnan().all(), what
        assert torch.equal(got[c[2]:], want[c[2]:])
