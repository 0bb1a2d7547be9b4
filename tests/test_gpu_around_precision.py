"""The calls around the cache norm-wise: ||err|| / ||out||, which one token left out of thousands moves by 1% and more.

Rows and cached values are unit normal, so errors of single keys are independent: of an output sum p v they add up as
squares, each relative error r of the weights or values giving r ||out||.  One rounding to f16 is off by 2^-11 / sqrt(3) of
the value at most, uniform in its half step: 2.8e-4 (bf16: 2.26e-3).
- Chunks round to f16: K (a score, of D products of 1 under a scale of 1 / sqrt(D), is off by 2.8e-4, and its weight by as
  much of it), V, the weights and, for f16 calls, the output: 2 x 2.8e-4 = 5.6e-4.
- Prompts and steps round the weights (steps: times V's scale) and the output: sqrt(2) x 2.8e-4 = 4e-4, bf16 prompts
  3.2e-3; their scores and sums are off by 1e-5 and below.  fp32 steps: 2e-6, as without a window.
A quarter more is left for what the norms of a sample stray: 7e-4, 5e-4, 4e-3.
"""
import numpy as np
import pytest

import window_ref
from host_streamed_paged_gb300 import kvs
from test_gpu_chunk import queries
from test_gpu_prompt import make
from test_gpu_q4 import Filled, _t

pytestmark = pytest.mark.gpu


def off(got, want):
    return np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1000, 4)])
@pytest.mark.parametrize("rows", [[2, 1], [70, 33], [300, 129]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunks(D, rows, window, sinks):
    """Histories that many workers share (few rows), and ones that a worker goes through: pieces of units, joined."""
    f = Filled([9000, 4000], 2, D, 64, seed=D, dt="f16")
    q, cu = queries(rows, 8, D, "f16", seed=len(rows))
    out, c = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q, window=window, sinks=sinks), cu.tolist()
    for i, n in enumerate(rows):
        s, T = slice(c[i], c[i + 1]), f.lens[i]
        k, v, _ = f.seq(i)
        want = window_ref.rows(q[s].double().cpu().numpy(), k, v, T - n + np.arange(n), D ** -0.5, window, sinks)[0]
        assert off(out[s], want) <= 7e-4, (i, off(out[s], want))


@pytest.mark.parametrize("dt,most", [("f16", 5e-4), ("bf16", 4e-3)])
@pytest.mark.parametrize("window,sinks", [(1, 3), (70, 4), (700, 0)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_windowed_prompts(D, window, sinks, dt, most):
    lens = [2100, 333, 65]
    q, k, v, cu = make(lens, 2, 4, D, dt, seed=D)
    out, c = kvs.prompt_attend(q, k, v, cu, window=window, sinks=sinks)[0], cu.tolist()
    for i, n in enumerate(lens):
        s = slice(c[i], c[i + 1])
        want = window_ref.rows(*(x[s].double().cpu().numpy() for x in (q, k, v)), np.arange(n), D ** -0.5, window, sinks)[0]
        assert off(out[s], want) <= most, (i, off(out[s], want))


@pytest.mark.parametrize("dt,most", [("f32", 2e-6), ("f16", 5e-4)])
@pytest.mark.parametrize("window,sinks", [(70, 4), (700, 0), (3000, 40)])
@pytest.mark.parametrize("D,R", [(64, 1), (128, 2), (256, 1)])
def test_windowed_steps(D, R, window, sinks, dt, most):
    import torch
    f = Filled([4096, 1031, 65], 2, D, 64, seed=D + R)
    q = (1.5 * torch.randn(3, R, 8, D, generator=torch.Generator().manual_seed(6))).to(_t(dt)).cuda()
    out = f.cache.attend(f.table_t, f.lens_t, q, window=window, sinks=sinks)[0]
    for i, T in enumerate(f.lens):
        k, v, _ = f.seq(i)
        want = window_ref.rows(q[i].double().cpu().numpy(), k, v, T - R + np.arange(R), D ** -0.5, window, sinks)[0]
        assert off(out[i], want) <= most, (i, off(out[i], want))
