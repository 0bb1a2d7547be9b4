"""Windows with first tokens that stay visible, on packed prompts and on the 4-bit cache's decode and span rows, against a
plain 64-bit form.  Tolerances as in test_gpu_prompt and test_gpu_q4: the arithmetic is theirs, over fewer keys."""
import math

import numpy as np
import pytest

import window_ref
from test_gpu_chunk import queries
from test_gpu_prompt import CASES as PROMPTS
from test_gpu_prompt import S_ERR as PROMPT_ERR
from test_gpu_prompt import make
from test_gpu_q4 import A_ERR, DT, S_ERR, Filled, _t, half_step

pytestmark = pytest.mark.gpu
WINDOWS = [(1, 0), (1, 3), (64, 4), (33, 40), (100, 0), (130, 129)]


def check_prompt(out, lse, q, k, v, cu, dt, scale, window, sinks):
    u = half_step(dt)
    o, z, qn, kn, vn = (x.double().cpu().numpy() for x in (out, lse, q, k, v))
    c = cu.tolist()
    for i in range(len(c) - 1):
        s, n = slice(c[i], c[i + 1]), c[i + 1] - c[i]
        if n == 0:
            continue
        ro, rz, A, _ = window_ref.rows(qn[s], kn[s], vn[s], np.arange(n), scale, window, sinks)
        sub = n * 2.0 ** -25 * np.abs(vn[s]).max() if dt == "f16" else 0.0
        err = np.abs(o[s] - ro)
        tol = u * np.abs(ro) + (u + PROMPT_ERR) * A + sub
        assert (err <= tol).all(), (i, np.argwhere(~(err <= tol))[:4], np.nanmax(err / tol))
        assert np.abs(z[s] - rz).max() <= PROMPT_ERR


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("D,Hk,G,lens", PROMPTS)
def test_prompts(D, Hk, G, lens, window, sinks):
    import torch
    from host_streamed_paged_gb300 import kvs
    dt = "bf16" if (window + D + G) % 2 else "f16"
    q, k, v, cu = make(lens, Hk, G, D, dt, seed=D + G, lead=3, tail=5)
    wide = torch.full((q.shape[0], Hk * G + 1, D), 7.0, dtype=_t(dt), device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out, _ = kvs.prompt_attend(q, k, v, cu, out=wide[:, :Hk * G], lse=lse, window=window, sinks=sinks)
    check_prompt(out, lse, q, k, v, cu, dt, 1 / math.sqrt(D), window, sinks)
    for x in (out, lse):
        assert (x[:3] == 7).all() and (x[-5:] == 7).all()
    assert (wide[:, Hk * G:] == 7).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_prompts_and_long_ones(D):
    from host_streamed_paged_gb300 import kvs
    lens = [(37 * i) % 90 for i in range(300)] + [1500]
    q, k, v, cu = make(lens, 1, 3, D, "bf16", seed=D)
    out, lse = kvs.prompt_attend(q, k, v, cu, window=50, sinks=2)
    check_prompt(out, lse, q, k, v, cu, "bf16", 1 / math.sqrt(D), 50, 2)


def test_a_window_past_the_prompts_is_none():
    import torch
    from host_streamed_paged_gb300 import kvs
    q, k, v, cu = make([300, 70], 1, 4, 128, "f16")
    want = kvs.prompt_attend(q, k, v, cu)
    for window, sinks in ((0, 9), (370, 0), (1 << 40, 1 << 40)):
        for a, b in zip(kvs.prompt_attend(q, k, v, cu, window=window, sinks=sinks), want):
            assert torch.equal(a, b)
    # one that only the longest prompt reaches past: the kernel with a window, the same weights
    out, lse = kvs.prompt_attend(q, k, v, cu, window=300, sinks=1)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def check_step(out, lse, q, f, dt, scale, window, sinks):
    out, lse, q = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    u = half_step(dt)
    for i, T in enumerate(f.lens):
        k, v, vs = f.seq(i)
        pos = T - q.shape[1] + np.arange(q.shape[1])
        o, z, A, _ = window_ref.rows(q[i], k, v, pos, scale, window, sinks)
        A8 = window_ref.rows(q[i], k, 8 * vs, pos, scale, window, sinks)[2]
        tol = u * np.abs(o) + ((2.0 ** -22 if dt == "f32" else 2.0 ** -11) + S_ERR) * A + A_ERR * A8
        bad = ~(np.abs(out[i] - o) <= tol)
        assert not bad.any(), (i, T, np.argwhere(bad)[:4])
        none = z == -np.inf
        assert np.array_equal(none, lse[i] == -np.inf) and (out[i][none] == 0).all()
        assert np.abs(lse[i][~none] - z[~none]).max(initial=0) <= S_ERR + 1e-5


LENS = [1, 0, 2, 31, 32, 33, 64, 99, 100, 101, 131, 700, 1024, 5000]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("D,P,Hk,G,R", [(64, 32, 2, 3, 1), (64, 256, 1, 8, 5), (128, 64, 1, 4, 3), (128, 128, 2, 7, 2), (256, 256, 1, 6, 2), (256, 32, 2, 2, 1)])
def test_steps(D, P, Hk, G, R, window, sinks, dt):
    import torch
    f = Filled(LENS, Hk, D, P, seed=D + R, dt=dt)
    q = torch.randn(len(LENS), R, Hk * G, D, generator=torch.Generator().manual_seed(5)).to(_t(dt)).cuda()
    out, lse = f.cache.attend(f.table_t, f.lens_t, q, window=window, sinks=sinks)
    check_step(out, lse, q, f, dt, 1 / math.sqrt(D), window, sinks)


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_steps_take_any_finite_scale(scale):
    import torch
    f = Filled([300, 33, 0, 70], 2, 128, 64, seed=2, dt="f16")
    q = torch.randn(4, 2, 6, 128, generator=torch.Generator().manual_seed(5)).half().cuda()
    out, lse = f.cache.attend(f.table_t, f.lens_t, q, scale=scale, window=50, sinks=4)
    check_step(out, lse, q, f, "f16", scale, 50, 4)


def test_a_window_past_the_table_is_none():
    import torch
    f = Filled([300, 33, 0], 2, 64, 64, seed=2)
    q = torch.randn(3, 1, 4, 64, generator=torch.Generator().manual_seed(5)).cuda()
    want = f.cache.attend(f.table_t, f.lens_t, q)
    for window, sinks in ((0, 9), (320, 0), (1 << 40, 1 << 40), (300, 5)):
        for a, b in zip(f.cache.attend(f.table_t, f.lens_t, q, window=window, sinks=sinks), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("P", [32, 64, 256])
def test_pages_behind_the_window_may_be_gone(P):
    import torch
    lens, R, window, sinks = [1500, 5000, 90], 3, 200, 4
    f = Filled(lens, 1, 128, P, seed=4, dt="f16")
    q = torch.randn(3, R, 4, 128, generator=torch.Generator().manual_seed(5)).half().cuda()
    want = f.cache.attend(f.table_t, f.lens_t, q, window=window, sinks=sinks)
    table = f.table.copy()
    for i, T in enumerate(lens):
        for page in range(table.shape[1]):
            if page * P >= sinks and (page + 1) * P <= T - R - window + 1:
                table[i, page] = -1 if page % 2 else 1 << 30
    assert (table != f.table).any()
    for a, b in zip(f.cache.attend(torch.from_numpy(table).cuda(), f.lens_t, q, window=window, sinks=sinks), want):
        assert torch.equal(a, b)
    table[1, -1 if P == 32 else 5000 // P] = -1  # the last token's
    out, _ = f.cache.attend(torch.from_numpy(table).cuda(), f.lens_t, q, window=window, sinks=sinks)
    if (5000 - 1) // P == 5000 // P or P == 32:
        assert torch.equal(out[0], want[0][0]) and torch.equal(out[2], want[0][2])


def test_waits_that_give_up_under_a_window():
    import torch
    from host_streamed_paged_gb300 import kvs
    f = Filled([0, 1, 33, 3000], 2, 128, 64, seed=3, dt="f16")
    q = torch.randn(4, 1, 8, 128, generator=torch.Generator().manual_seed(5)).half().cuda()
    want = f.cache.attend(f.table_t, f.lens_t, q, window=500, sinks=4)
    pq, cu = queries([700, 3], 4, 128, "f16")
    kv = torch.randn(703, 2, 128, generator=torch.Generator().manual_seed(6)).half().cuda()
    prompts = kvs.prompt_attend(pq, kv[:, :1], kv[:, 1:], cu, window=100)
    try:
        for _ in range(3):
            kvs.kvs_debug_inject(None, kvs.KVS_FAULT_DEVICE_WAIT, 1)
            out, z = f.cache.attend(f.table_t, f.lens_t, q, window=500, sinks=4)
            assert out[1:].isnan().all() and z[1:].isnan().all() and not out[0].any()
            out, z = f.cache.attend(f.table_t, f.lens_t, q, window=500, sinks=4)
            assert torch.equal(out, want[0]) and torch.equal(z, want[1])
            kvs.kvs_debug_inject(None, kvs.KVS_FAULT_DEVICE_WAIT, 1)
            assert kvs.prompt_attend(pq, kv[:, :1], kv[:, 1:], cu, window=100)[0].isnan().all()
            for a, b in zip(kvs.prompt_attend(pq, kv[:, :1], kv[:, 1:], cu, window=100), prompts):
                assert torch.equal(a, b)
    finally:
        kvs.kvs_debug_inject(None, kvs.KVS_FAULT_NONE, 0)


def test_a_graph_of_a_windowed_step():
    import torch
    f = Filled([5000, 70], 2, 128, 64, seed=14, dt="f16")
    q = torch.randn(2, 1, 8, 128, generator=torch.Generator().manual_seed(1)).half().cuda()
    want = f.cache.attend(f.table_t, f.lens_t, q, window=300, sinks=4)
    out, lse = torch.empty_like(q), torch.empty(2, 1, 8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f.cache.attend(f.table_t, f.lens_t, q, out=out, lse=lse, window=300, sinks=4)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    f.lens_t.copy_(torch.tensor([900, 3], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    want = f.cache.attend(f.table_t, f.lens_t, q, window=300, sinks=4)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


MANY = [  # lens, kv heads, group: several units of every CTA
    ([3000, 1, 2000, 500, 35, 36, 37], 4, 7),
    ([2500] + [(53 * i) % 150 for i in range(60)], 2, 16),
    ([(29 * i) % 60 for i in range(400)] + [700], 2, 5),
]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,Hk,G", MANY)
def test_prompts_of_many_units(lens, Hk, G, D):
    import torch
    from host_streamed_paged_gb300 import kvs
    dt = "f16" if D == 128 else "bf16"
    q, k, v, cu = make(lens, Hk, G, D, dt, seed=D + Hk)
    out, lse = kvs.prompt_attend(q, k, v, cu, window=90, sinks=3)
    check_prompt(out, lse, q, k, v, cu, dt, 1 / math.sqrt(D), 90, 3)
    # a prompt's rows do not depend on what else is in the batch, or on which CTA has them
    c = cu.tolist()
    for i in (0, len(lens) - 1):
        s = slice(c[i], c[i + 1])
        one = torch.tensor([0, lens[i]], dtype=torch.int32, device="cuda")
        for a, b in zip(kvs.prompt_attend(q[s], k[s], v[s], one, window=90, sinks=3), (out, lse)):
            assert torch.equal(a, b[s])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_windowed_prompts_beside_rows_that_are_not_finite(D):
    import torch
    from host_streamed_paged_gb300 import kvs
    lens = [1100, 70, 901, 33, 64, 1]
    q, k, v, cu = make(lens, 3, 8, D, "f16", seed=D)
    want = kvs.prompt_attend(q, k, v, cu, window=100, sinks=2)
    c = cu.tolist()
    for i in (1, 3, 5):
        k[c[i]:c[i + 1]] = math.nan
        v[c[i]:c[i + 1]] = math.inf
    got = kvs.prompt_attend(q, k, v, cu, window=100, sinks=2)
    for i in (0, 2, 4):
        for a, b in zip(got, want):
            assert torch.equal(a[c[i]:c[i + 1]], b[c[i]:c[i + 1]])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_units_after_a_wait_that_gave_up(D):
    import torch
    from host_streamed_paged_gb300 import kvs
    q, k, v, cu = make([4000, 300, 2], 4, 4, D, "bf16", seed=D)
    want = kvs.prompt_attend(q, k, v, cu, window=200, sinks=1)
    try:
        for _ in range(2):
            kvs.kvs_debug_inject(None, kvs.KVS_FAULT_DEVICE_WAIT, 1)
            out, lse = kvs.prompt_attend(q, k, v, cu, window=200, sinks=1)
            assert out.isnan().all() and lse.isnan().all()
            for a, b in zip(kvs.prompt_attend(q, k, v, cu, window=200, sinks=1), want):
                assert torch.equal(a, b)
    finally:
        kvs.kvs_debug_inject(None, kvs.KVS_FAULT_NONE, 0)


def test_a_graph_of_windowed_prompts_beside_an_eager_one():
    import torch
    from host_streamed_paged_gb300 import kvs
    q, k, v, cu = make([2000, 77, 900], 4, 4, 128, "bf16", seed=2)
    want = kvs.prompt_attend(q, k, v, cu, window=150, sinks=4)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvs.prompt_attend(q, k, v, cu, out=out, lse=lse, window=150, sinks=4)
    other = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        other.wait_stream(torch.cuda.current_stream())
        g.replay()
        with torch.cuda.stream(other):
            beside = kvs.prompt_attend(q, k, v, cu, window=150, sinks=4)
        torch.cuda.synchronize()
        for a, b, c in zip((out, lse), beside, want):
            assert torch.equal(a, c) and torch.equal(b, c)
