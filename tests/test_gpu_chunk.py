"""Chunks of new rows over the 4-bit cache (kvs_q4_attend_chunk) against a plain 64-bit form.

Tolerances, from the arithmetic the kernel states; A = sum p |v|, u the half step of the output type, n the tokens seen:
- K is rounded to f16 once (2^-11 of each value) and a score's products are summed in fp32 by the tensor core, 16 at a
  time, each sum cut off below 2^-23 of it: a score is off by at most E = (2^-11 + 16 2^-22) max scale sum |q k|, its
  weight by a factor e^E, in numerator and denominator: expm1(2 E) A of the output, E of lse;
- V and the weights are rounded to f16 once: 2 2^-11 A; weights below f16's 2^-14 lose up to 2^-25 each, where a row's
  largest weight is at least 2^2 (times its tile's power of two) and V's values, brought to their tile's power of two, at
  most 2^-2: n 2^-27 of those units; the largest weight's tile holds a value of 2^-3 of them or more, so that is at most
  n 2^-27 2^3 2^-2 = n 2^-26 max|v| of the output; values below 2^-14 of their units, 2^-12 of the tile's largest, are off by
  2^-25, 2^-23 of the largest, which 2^-11 of it in A's place covers where weights are as large, and n 2^-26 max|v| else;
- outputs are summed in fp32, 16 tokens at a time, and rescaled: (n / 16 + 32) 2^-22 A;
- out is rounded: u |out|; lse adds the exponentials' and the logarithm's 1e-5.
"""
import math

import numpy as np
import pytest

import window_ref
from test_gpu_q4 import Filled, _t

pytestmark = pytest.mark.gpu


def queries(rows, Hq, D, dt, seed=1, lead=0, tail=0, wide=1):
    """q [lead + sum + tail][Hq][D], strided, with NaN rows outside the sequences, and cu."""
    import torch
    n = lead + sum(rows) + tail
    x = torch.randn(n, Hq + wide, D, generator=torch.Generator().manual_seed(seed)).to(_t(dt))
    x[:lead] = math.nan
    x[n - tail:] = math.nan
    cu = torch.tensor(np.concatenate([[lead], lead + np.cumsum(rows)]), dtype=torch.int32).cuda()
    return x.cuda()[:, :Hq], cu


def check(out, lse, q, cu, filled, dt, scale, window=0, sinks=0, skip=()):
    import torch
    u = torch.finfo(_t(dt)).eps / 2
    o, qn = out.double().cpu().numpy(), q.double().cpu().numpy()
    z = lse.double().cpu().numpy()
    c = cu.tolist()
    for i in range(len(c) - 1):
        n, T = c[i + 1] - c[i], filled.lens[i]
        if i in skip or n == 0:
            continue
        s = slice(c[i], c[i + 1])
        k, v, _ = filled.seq(i)
        ro, rz, A, most = window_ref.rows(qn[s], k, v, T - n + np.arange(n), scale, window, sinks)
        E = (2.0 ** -11 + 2.0 ** -18) * most
        top = np.abs(v).max(initial=0)
        tol = u * np.abs(ro) + (np.expm1(2 * E)[..., None] + 2.0 ** -10 + (T / 16 + 32) * 2.0 ** -22) * A + T * 2.0 ** -26 * top
        bad = ~(np.abs(o[s] - ro) <= tol)
        assert not bad.any(), (i, n, T, np.argwhere(bad)[:4], np.nanmax(np.abs(o[s] - ro) / np.maximum(tol, 1e-300)))
        none = rz == -np.inf
        assert np.array_equal(none, z[s] == -np.inf) and (o[s][none] == 0).all()
        assert (np.abs(z[s][~none] - rz[~none]) <= E[~none] + 1e-5).all()


def run(f, rows, Hk, G, D, dt, scale=None, lead=3, tail=5, seed=1, **kw):
    """The call with strided q and out, and that rows of no sequence are left."""
    import torch
    q, cu = queries(rows, Hk * G, D, dt, seed, lead, tail)
    room = torch.full((q.shape[0], Hk * G + 2, D), 7.0, dtype=_t(dt), device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q, scale=scale, out=room[:, :Hk * G], lse=lse, **kw)
    assert out.data_ptr() == room.data_ptr() and (room[:, Hk * G:] == 7).all()
    end = lead + sum(rows)
    for x in (out, lse):
        assert (x[:lead] == 7).all() and (x[end:] == 7).all()
    check(out, lse, q, cu, f, dt, D ** -0.5 if scale is None else scale, **kw)
    return out, lse, q, cu


CASES = [  # D, P, Hk, G, rows, lens
    (64, 32, 2, 4, [1, 0, 31, 129, 300, 2], [1, 40, 64, 129, 700, 0]),
    (64, 256, 1, 64, [5, 70], [5, 333]),
    (64, 64, 3, 1, [128, 1, 257], [1000, 63, 257]),
    (128, 64, 2, 4, [1, 63, 64, 65, 200], [64, 63, 65, 1025, 200]),
    (128, 32, 1, 6, [21, 22, 1, 43, 150], [33, 96, 97, 43, 640]),
    (128, 128, 1, 3, [600], [777]),
    (128, 256, 2, 8, [1, 1, 1, 1, 40], [5000, 1, 31, 256, 2000]),
    (256, 32, 1, 6, [1, 37, 64, 65], [32, 37, 700, 127]),
    (256, 256, 2, 1, [127, 129, 3], [127, 1400, 3]),
    (256, 64, 2, 5, [19, 20, 77, 1], [19, 64, 300, 4000]),
    (256, 128, 1, 50, [7, 30], [7, 500]),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D,P,Hk,G,rows,lens", CASES)
def test_attend_chunk(D, P, Hk, G, rows, lens, dt):
    run(Filled(lens, Hk, D, P, seed=D + G, dt=dt, extra=1), rows, Hk, G, D, dt)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (33, 40), (100, 0), (130, 65), (300, 1000)])
@pytest.mark.parametrize("D,P,Hk,G,rows,lens", [CASES[0], CASES[4], CASES[6], CASES[7], CASES[9]])
def test_under_a_window(D, P, Hk, G, rows, lens, window, sinks):
    run(Filled(lens, Hk, D, P, seed=D + G, dt="f16"), rows, Hk, G, D, "f16", window=window, sinks=sinks)


@pytest.mark.parametrize("D,P", [(64, 32), (128, 32), (128, 64), (256, 256)])
def test_pages_behind_the_window_may_be_gone(D, P):
    """Their numbers are taken out of the table, their bytes are never read: the result is the same."""
    import torch
    lens, rows, window, sinks = [1500, 400], [70, 1], 200, 4
    f = Filled(lens, 1, D, P, seed=4, dt="f16")
    out, lse, q, cu = run(f, rows, 1, 4, D, "f16", window=window, sinks=sinks)
    table = f.table.copy()
    for i, (T, n) in enumerate(zip(lens, rows)):
        for page in range(table.shape[1]):
            if page * P >= sinks and (page + 1) * P <= T - n - window + 1:
                table[i, page] = -1 if page % 2 else 1 << 30
    assert (table != f.table).sum() >= 2
    z = torch.full_like(lse, 7.0)
    got = f.cache.attend_chunk(torch.from_numpy(table).cuda(), f.lens_t, cu, q, window=window, sinks=sinks, lse=z)
    s = slice(int(cu[0]), int(cu[-1]))
    assert torch.equal(got[s], out[s]) and torch.equal(z, lse)


@pytest.mark.parametrize("scale", [0.0, 1e-30, -0.05])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_any_finite_scale(D, scale):
    run(Filled([300, 33, 0], 2, D, 64, seed=D, dt="bf16"), [40, 1, 2], 2, 3, D, "bf16", scale=scale)


@pytest.mark.parametrize("v_scale", [1e-4, 1.0, 3e4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_cached_values_of_any_size(D, v_scale):
    """Scales from f16's subnormals to its largest (f16 takes values up to 8 times as large from them)."""
    run(Filled([500, 70], 1, D, 64, seed=D, dt="f32", v_scale=v_scale), [65, 3], 1, 4, D, "bf16")


@pytest.mark.parametrize("k_scale", [1e-4, 100.0])
def test_keys_and_queries_of_any_size(k_scale):
    """Keys and queries at far ends, their products as usual; tokens of other sizes beside each other."""
    import torch
    f = Filled([500, 70], 1, 128, 64, seed=3, dt="f32")
    from batch_ref import q4_encode, q4_values
    size = torch.where(torch.arange(570) % 3 == 0, k_scale, 1.0).view(-1, 1, 1)
    f.k *= size
    f.cache.append(torch.from_numpy(f.slots).cuda(), f.k.cuda(), f.v.cuda())
    f.kv[0] = q4_values(*q4_encode(f.k.numpy()))
    run(f, [65, 3], 1, 4, 128, "f16", scale=0.088 / max(k_scale, 1.0))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_histories_are_shared_by_many_workers(D):
    """Few rows over many keys: the units are cut and joined, and a second run gives the same bits."""
    import torch
    f = Filled([9000, 4000], 2, D, 256, seed=D, dt="f16")
    out, lse, q, cu = run(f, [2, 1], 2, 4, D, "f16")
    again = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q)
    assert torch.equal(again[3:6], out[3:6])


def test_many_sequences():
    """More than there are workers, most of them of one row, some of none."""
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 90, 700).tolist()
    rows = [int(min(n, r)) for n, r in zip(lens, rng.integers(0, 4, 700))]
    run(Filled(lens, 2, 64, 32, seed=1, dt="bf16"), rows, 2, 3, 64, "bf16")


@pytest.mark.parametrize("D,G", [(64, 4), (128, 3), (256, 5)])
def test_many_short_units(D, G):
    """Units of one to a few blocks, of one query tile and of two, one after another in every worker: the stages' and
    buffers' phases go on from unit to unit."""
    rng = np.random.default_rng(D)
    lens = rng.integers(1, 200, 300).tolist()
    rows = [int(rng.integers(0, min(n, 90) + 1)) for n in lens]
    f = Filled(lens, 2, D, 32, seed=1, dt="bf16")
    run(f, rows, 2, G, D, "bf16")
    run(f, rows, 2, G, D, "bf16", window=40, sinks=3)


def test_the_most_sequences():
    lens = [(7 * i) % 40 for i in range(4096)]
    rows = [min(n, 1 + i % 2) for i, n in enumerate(lens)]
    run(Filled(lens, 1, 64, 32, seed=2, dt="f16"), rows, 1, 2, 64, "f16")


def test_a_page_outside_the_pool_makes_its_sequence_nan():
    import torch
    f = Filled([200, 200, 100], 1, 128, 64, seed=6, dt="f16")
    want, lse, q, cu = run(f, [70, 70, 5], 1, 4, 128, "f16")
    table = f.table_t.clone()
    table[1, 1] = f.cache.n_pages
    got = f.cache.attend_chunk(table, f.lens_t, cu, q)
    a, b = int(cu[1]), int(cu[2])
    assert got[a:b].isnan().all()
    for s in (slice(int(cu[0]), a), slice(b, int(cu[3]))):
        assert torch.equal(got[s], want[s])


@pytest.mark.parametrize("bad", [math.nan, math.inf, 1e30])
def test_cached_rows_that_are_not_finite_stay_with_their_sequence_and_head(bad):
    import torch
    f = Filled([40, 100, 300], 2, 64, 64, seed=8)
    want, _, q, cu = run(f, [20, 50, 66], 2, 2, 64, "f16")
    k, v = f.k.clone(), f.v.clone()
    k[60:70, 1] = bad
    v[90:95, 1, 3] = bad
    f.cache.append(torch.from_numpy(f.slots).cuda(), k.cuda(), v.cuda())
    got = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q)
    c = cu.tolist()
    for i in (0, 2):
        assert torch.equal(got[c[i]:c[i + 1]], want[c[i]:c[i + 1]])
    assert torch.equal(got[c[1]:c[2], :2], want[c[1]:c[2], :2])


def test_queries_that_are_not_finite_stay_alone():
    import torch
    f = Filled([300], 1, 128, 64, seed=9, dt="f16")
    q, cu = queries([40], 4, 128, "f16")
    want = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q)
    q = q.clone()
    q[7, 2, 5], q[9, 0] = math.nan, math.inf
    got = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q)
    rest = torch.ones(40, 4, dtype=torch.bool)
    rest[7, 2] = rest[9, 0] = False
    assert torch.equal(got[rest.cuda()], want[rest.cuda()]) and got[7, 2].isnan().all() and got[9, 0].isnan().all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_out_may_be_the_query(D):
    import torch
    f = Filled([3000, 33, 0, 64], 2, D, 64, seed=5, dt="bf16")
    rows = [90, 33, 1, 1]
    q, cu = queries(rows, 8, D, "bf16", wide=0)
    want = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q)
    x = q.clone()
    assert f.cache.attend_chunk(f.table_t, f.lens_t, cu, x, out=x) is x and torch.equal(x, want)


def test_offsets_and_lengths_are_clamped():
    """Offsets outside the rows, lengths past the table or below zero: what they address stays inside the arrays."""
    import torch
    f = Filled([100, 60, 50], 1, 64, 32, seed=3, dt="f16")
    q, _ = queries([90], 2, 64, "f16")
    cu = torch.tensor([-5, 40, 30, 4000], dtype=torch.int32, device="cuda")  # 40 rows, none (60 > 30), rows 30 .. 89
    lens = torch.tensor([1 << 30, 60, -7], dtype=torch.int32, device="cuda")
    out = f.cache.attend_chunk(f.table_t, lens, cu, q)
    # the first: as long as the table holds, of which the last tokens were never written; the third: nothing cached
    assert not out[40:].any()
    torch.cuda.synchronize()


def test_pages_past_four_gigabytes():
    import torch
    from host_streamed_paged_gb300 import kvs
    P, Hk, D, G = 256, 8, 256, 2
    cache = kvs.Q4Cache(page_tokens=P, n_kv_head=Hk, head_dim=D, n_pages=8200)  # 4.8e9 bytes
    small = Filled([600, 33], Hk, D, P, seed=3, dt="f16")
    table = (cache.n_pages - 1 - torch.arange(6, dtype=torch.int32).view(2, 3)).cuda()
    slots = torch.cat([table[i].long().cpu()[torch.arange(n) // P] * P + torch.arange(n) % P for i, n in enumerate(small.lens)]).cuda()
    cache.append(slots, small.k.cuda(), small.v.cuda())
    q, cu = queries([70, 33], Hk * G, D, "f16")
    assert torch.equal(cache.attend_chunk(table, small.lens_t, cu, q), small.cache.attend_chunk(small.table_t, small.lens_t, cu, q))


def test_rows_past_four_gigabytes():
    import torch
    f = Filled([900, 90], 1, 64, 64, seed=3, dt="f16")
    rows, stride = [610, 90], 4 << 20
    store = torch.empty(700 * stride, dtype=torch.float16, device="cuda")  # 5.9e9 bytes
    x = store.as_strided((700, 4, 64), (stride, 64, 1))
    q, cu = queries(rows, 2, 64, "f16")
    x[:, :2].copy_(q)
    got = f.cache.attend_chunk(f.table_t, f.lens_t, cu, x[:, :2], out=x[:, 2:])
    assert torch.equal(got, f.cache.attend_chunk(f.table_t, f.lens_t, cu, q))


def test_graphs_side_by_side_and_replays_read_what_the_device_holds():
    """Each captured call has a workspace of its own; a replay takes the offsets, lengths and tables found then."""
    import torch
    f = Filled([9000, 700], 2, 128, 64, seed=14, dt="f16")
    rows = [[60, 130], [3, 1]]
    qs = [queries(r, 8, 128, "f16", seed=i) for i, r in enumerate(rows)]
    want = [f.cache.attend_chunk(f.table_t, f.lens_t, cu, q) for q, cu in qs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q, cu in qs:
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                f.cache.attend_chunk(f.table_t, f.lens_t, cu, q, out=out)
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            eager = f.cache.attend_chunk(f.table_t, f.lens_t, qs[0][1], qs[0][0])
        torch.cuda.synchronize()
        assert torch.equal(eager, want[0])
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    q, cu = qs[0]
    cu.copy_(torch.tensor([0, 190, 190], dtype=torch.int32))
    f.lens_t.copy_(torch.tensor([333, 0], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], f.cache.attend_chunk(f.table_t, f.lens_t, cu, q)) and not torch.equal(outs[0], want[0])


def test_two_streams():
    import torch
    f = Filled([5000, 700], 2, 128, 64, seed=15, dt="f16")
    qs = [queries([60 + i, 130], 8, 128, "f16", seed=i) for i in range(2)]
    want = [f.cache.attend_chunk(f.table_t, f.lens_t, cu, q) for q, cu in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (q, cu) in enumerate(qs):
            with torch.cuda.stream(streams[i]):
                got[i].append(f.cache.attend_chunk(f.table_t, f.lens_t, cu, q))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, w) for x in g)


@pytest.mark.parametrize("D,G", [(64, 4), (128, 3), (256, 6)])
def test_a_wait_that_gives_up_makes_its_outputs_nan(D, G):
    import torch
    from host_streamed_paged_gb300 import kvs
    lens, rows = [1, 700, 64, 3000, 0, 2], [1, 33, 0, 200, 1, 4]
    f = Filled(lens, 2, D, 64, seed=D, dt="f16")
    out, lse, q, cu = run(f, rows, 2, G, D, "f16")
    c = cu.tolist()
    try:
        for _ in range(3):
            kvs.kvs_debug_inject(None, kvs.KVS_FAULT_DEVICE_WAIT, 1)
            z = torch.full_like(lse, 7.0)
            got = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q, lse=z)
            for i, T in enumerate(lens):
                for r in range(c[i], c[i + 1]):
                    if T - (c[i + 1] - r) < 0:
                        continue  # it sees nothing: zeros, or NaN beside rows that do
                    assert got[r].isnan().all() and z[r].isnan().all()
            again = f.cache.attend_chunk(f.table_t, f.lens_t, cu, q, lse=z)
            assert torch.equal(again[c[0]:c[-1]], out[c[0]:c[-1]]) and torch.equal(z, lse)
    finally:
        kvs.kvs_debug_inject(None, kvs.KVS_FAULT_NONE, 0)
