"""Calls of the batch operators at the edges of what include/kvs.h allows: byte offsets past 32 bits, graphs replayed side
by side, rows of neighbours that are not finite, accumulation that goes on after an eviction.  Bounds as in the files that
the helpers come from."""
import math

import numpy as np
import pytest

import batch_ref as ref
from test_gpu_prompt import check
from test_gpu_q4 import S_ERR, Filled, check_attend

pytestmark = pytest.mark.gpu


def test_pages_past_four_gigabytes():
    import torch
    from host_streamed_paged_gb300 import kvs
    P, Hk, D, G = 256, 8, 256, 2
    cache = kvs.Q4Cache(page_tokens=P, n_kv_head=Hk, head_dim=D, n_pages=8200)  # 4.8e9 bytes
    small = Filled([600, 33], Hk, D, P, seed=3, dt="f16")
    top = cache.n_pages - 1 - torch.arange(6, dtype=torch.int32).view(2, 3)
    table = top.cuda()
    assert int(top.min()) * cache.page_bytes > 1 << 32
    slots = torch.cat([top[i].long()[torch.arange(n) // P] * P + torch.arange(n) % P for i, n in enumerate(small.lens)]).cuda()
    cache.append(slots, small.k.cuda(), small.v.cuda())
    q = torch.randn(2, 1, Hk * G, D, generator=torch.Generator().manual_seed(4)).half().cuda()
    for a, b in zip(cache.read(slots), small.cache.read(torch.from_numpy(small.slots).cuda())):
        assert torch.equal(a, b)
    got, want = cache.attend(table, small.lens_t, q), small.cache.attend(small.table_t, small.lens_t, q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    w = cache.weights(table, small.lens_t, q, got[1], width=768)
    assert torch.equal(w, small.cache.weights(small.table_t, small.lens_t, q, got[1], width=768))
    dst = (cache.n_pages - 10 - torch.arange(4, dtype=torch.int32).view(2, 2)).cuda()
    kept, lens, _ = cache.evict(table, dst, small.lens_t, w, 300, sinks=4, recent=16)
    assert lens.tolist() == [300, 33]
    at = torch.arange(300)
    k, v = cache.read((dst[0].long().cpu()[at // P] * P + at % P).cuda())
    ks, vs, _ = small.seq(0)
    for h in range(Hk):
        i = kept[0, h].cpu().numpy()
        assert np.array_equal(k[:, h].double().cpu().numpy() + 0.0, ks[i, h] + 0.0)
        assert np.array_equal(v[:, h].double().cpu().numpy() + 0.0, vs[i, h] + 0.0)


def test_prompt_rows_past_four_gigabytes():
    import torch
    from host_streamed_paged_gb300 import kvs
    n, stride, D = 700, 4 << 20, 64  # 5.9e9 bytes
    store = torch.empty(n * stride, dtype=torch.float16, device="cuda")
    x = store.as_strided((n, 6, D), (stride, D, 1))
    x.copy_(torch.randn(n, 6, D, generator=torch.Generator().manual_seed(2)).half())
    q, k, v, room = x[:, :2], x[:, 2:3], x[:, 3:4], x[:, 4:6]
    cu = torch.tensor([0, 90, 700], dtype=torch.int32, device="cuda")
    o, lse = kvs.prompt_attend(q, k, v, cu, out=room)
    check(o, lse, q, k, v, cu, "f16", 1 / 8)
    w = kvs.prompt_weights(q, k, lse, cu, 610)
    assert torch.equal(w, kvs.prompt_weights(q.contiguous(), k.contiguous(), lse, cu, 610))


def test_weights_past_two_giga_entries():
    import torch
    f = Filled([70, 0, 45], 2, 64, 64, seed=6, dt="f16")
    q = torch.randn(3, 1, 4, 64, generator=torch.Generator().manual_seed(4)).half().cuda()
    lse = f.cache.attend(f.table_t, f.lens_t, q)[1]
    width = 1 << 29  # 6 rows of 2^29 entries
    w = torch.zeros(3, 2, width, device="cuda")
    f.cache.weights(f.table_t, f.lens_t, q, lse, prev=w, out=w)
    small = f.cache.weights(f.table_t, f.lens_t, q, lse, width=128)
    assert torch.equal(w[..., :128], small) and not w[..., 128:].any()
    fresh = f.cache.weights(f.table_t, f.lens_t, q, lse, width=width, out=w.fill_(7))
    assert torch.equal(fresh[..., :128], small) and not fresh[..., 128:].any()


def test_two_graphs_of_one_stream_replayed_side_by_side():
    """Each captured attend has a workspace of its own."""
    import torch
    f = Filled([9000, 70], 2, 128, 64, seed=14, dt="f16")
    qs = [torch.randn(2, 1, 8, 128, generator=torch.Generator().manual_seed(i)).half().cuda() for i in range(2)]
    want = [f.cache.attend(f.table_t, f.lens_t, q) for q in qs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q in qs:
        out, lse = torch.empty_like(q), torch.empty(2, 1, 8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                f.cache.attend(f.table_t, f.lens_t, q, out=out, lse=lse)
        graphs.append(g)
        outs.append((out, lse))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for o, z in outs:
            o.zero_()
            z.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            eager = f.cache.attend(f.table_t, f.lens_t, qs[0])
        torch.cuda.synchronize()
        assert torch.equal(eager[0], want[0][0])
        for (o, z), (wo, wz) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(z, wz)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D,G", [(64, 3), (128, 4), (256, 6)])
def test_rows_that_are_not_finite_stay_with_their_prompt(D, G, bad):
    import torch
    from host_streamed_paged_gb300 import kvs
    lens = [50, 129, 1, 70]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), G + 2, D, generator=torch.Generator().manual_seed(7)).half().cuda()
    y = x.clone()
    for i in (1, 2):
        y[cu[i]:cu[i + 1]] = bad
    want, lse = kvs.prompt_attend(x[:, :G], x[:, G:G + 1], x[:, G + 1:], cu)
    got, z = kvs.prompt_attend(y[:, :G], y[:, G:G + 1], y[:, G + 1:], cu)
    w, u = kvs.prompt_weights(x[:, :G], x[:, G:G + 1], lse, cu, 130), kvs.prompt_weights(y[:, :G], y[:, G:G + 1], z, cu, 130)
    for i in (0, 3):
        s = slice(int(cu[i]), int(cu[i + 1]))
        assert torch.equal(got[s], want[s]) and torch.equal(z[s], lse[s]) and torch.equal(u[i], w[i])


@pytest.mark.parametrize("bad", [math.nan, math.inf, 1e30])
def test_cached_rows_that_are_not_finite_stay_with_their_sequence_and_head(bad):
    """1e30 is finite, but its block's scale is not an fp16 number."""
    import torch
    lens = [40, 100, 300]
    f = Filled(lens, 2, 64, 64, seed=8)
    q = torch.randn(3, 1, 4, 64, generator=torch.Generator().manual_seed(4)).cuda()
    want, lse = f.cache.attend(f.table_t, f.lens_t, q)
    w = f.cache.weights(f.table_t, f.lens_t, q, lse)
    k, v = f.k.clone(), f.v.clone()
    k[60:70, 1] = bad
    v[90:95, 1, 3] = bad
    f.cache.append(torch.from_numpy(f.slots).cuda(), k.cuda(), v.cuda())
    got, z = f.cache.attend(f.table_t, f.lens_t, q)
    u = f.cache.weights(f.table_t, f.lens_t, q, z)
    for i in (0, 2):
        assert torch.equal(got[i], want[i]) and torch.equal(z[i], lse[i]) and torch.equal(u[i], w[i])
    assert torch.equal(got[1, :, :2], want[1, :, :2]) and torch.equal(z[1, :, :2], lse[1, :, :2]) and torch.equal(u[1, 0], w[1, 0])


def test_a_replayed_graph_of_append_evict_and_read():
    import torch
    lens, keep, P = [300, 90], 100, 64
    f = Filled(lens, 2, 64, P, seed=9, dt="f16", spare=6)
    dst = torch.from_numpy(f.free[:4].reshape(2, 2).astype(np.int32).copy()).cuda()
    w = torch.rand(2, 2, 320, generator=torch.Generator().manual_seed(1)).cuda()
    slots = torch.from_numpy(f.slots).cuda()
    k, v = f.k.cuda(), f.v.cuda()
    cur = f.lens_t.clone()
    at = torch.arange(keep, device="cuda")
    there = (dst.long()[:, at // P] * P + at % P).flatten()

    def step():
        f.cache.append(slots, k, v)
        kept, new, kw = f.cache.evict(f.table_t, dst, cur, w, keep, sinks=2, recent=5)
        return [kept, new, kw, *f.cache.read(there)]

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed, new in ((2, [300, 90]), (3, [100, 101]), (4, [0, 77])):
        gen = torch.Generator().manual_seed(seed)
        w.copy_(torch.rand(2, 2, 320, generator=gen))
        k.copy_(torch.randn(k.shape, generator=gen))
        cur.copy_(torch.tensor(new, dtype=torch.int32))
        f.cache.pages.zero_()
        g.replay()
        got = [x.clone() for x in out]
        f.cache.pages.zero_()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        for i in range(2):
            for h in range(2):
                want = ref.evict(w[i, h, :new[i]].cpu().numpy(), keep, 2, 5)
                assert got[0][i, h].tolist() == want.tolist() + [-1] * (keep - len(want))


def test_the_most_prompts():
    import torch
    from host_streamed_paged_gb300 import kvs
    lens = np.random.default_rng(5).integers(0, 4, 4096)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    x = torch.randn(int(lens.sum()), 4, 64, generator=torch.Generator().manual_seed(7)).half().cuda()
    q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
    out, lse = kvs.prompt_attend(q, k, v, cu)
    check(out, lse, q, k, v, cu, "f16", 1 / 8)
    w = kvs.prompt_weights(q, k, lse, cu, 4).double().cpu().numpy()
    qn, kn, zn, c = q.double().cpu().numpy(), k.double().cpu().numpy(), lse.double().cpu().numpy(), cu.tolist()
    for i, n in enumerate(lens):
        want = np.zeros((1, 4))
        if n:
            s = slice(c[i], c[i + 1])
            want[:, :n] = ref.prompt_weights(qn[s], kn[s], zn[s], 1 / 8)
        assert (np.abs(w[i] - want) <= 5e-5 * want + 1e-37).all(), i


@pytest.mark.parametrize("D,G", [(64, 64), (128, 64), (256, 64), (256, 33)])
def test_the_widest_groups(D, G):
    import torch
    from host_streamed_paged_gb300 import kvs
    lens = [90, 1, 131]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), G + 2, D, generator=torch.Generator().manual_seed(D + G)).bfloat16().cuda()
    q, k, v = x[:, :G], x[:, G:G + 1], x[:, G + 1:]
    out, lse = kvs.prompt_attend(q, k, v, cu)
    check(out, lse, q, k, v, cu, "bf16", 1 / math.sqrt(D))
    for window in (0, 5):
        w = kvs.prompt_weights(q, k, lse, cu, 131, window=window).double().cpu().numpy()
        qn, kn, zn, c = q.double().cpu().numpy(), k.double().cpu().numpy(), lse.double().cpu().numpy(), cu.tolist()
        for i, n in enumerate(lens):
            s = slice(c[i], c[i + 1])
            want = ref.prompt_weights(qn[s], kn[s], zn[s], 1 / math.sqrt(D), window)
            assert (np.abs(w[i, :, :n] - want) <= (5e-5 + n * G / 4 * 2.0 ** -24) * want + 1e-37).all(), i
    for dt in ("f32", "f16"):
        f = Filled([0, 1, 70, 900], 1, D, 32, seed=4, dt=dt)
        q = torch.randn(4, 1, G, D, generator=torch.Generator().manual_seed(6)).to(f.k.dtype).cuda()
        out, lse = f.cache.attend(f.table_t, f.lens_t, q)
        check_attend(out, lse, q, f, dt, 1 / math.sqrt(D))


def test_accumulation_goes_on_after_an_eviction():
    """The kept tokens' weights, in the first columns of a row as wide as the new pages hold, are prev from then on."""
    import torch
    lens, keep, P, Hk, G, D = [700, 90], 200, 64, 2, 4, 128
    f = Filled(lens, Hk, D, P, seed=21, dt="f16", spare=8)
    gen = torch.Generator().manual_seed(3)
    q = torch.randn(2, 1, Hk * G, D, generator=gen).half().cuda()
    lse = f.cache.attend(f.table_t, f.lens_t, q)[1]
    w = f.cache.weights(f.table_t, f.lens_t, q, lse)
    dst = torch.from_numpy(f.free[:8].reshape(2, 4).astype(np.int32).copy()).cuda()
    kept, cur, kw = f.cache.evict(f.table_t, dst, f.lens_t, w, keep, sinks=4, recent=16)
    acc = torch.zeros(2, Hk, dst.shape[1] * P, device="cuda")
    acc[..., :keep] = kw
    values = []
    for i, n in enumerate(lens):
        k, v, _ = f.seq(i)
        idx = [kept[i, h, :min(n, keep)].cpu().numpy() for h in range(Hk)]
        values.append([np.stack([a[idx[h], h] for h in range(Hk)], 1) for a in (k, v)])
    want = acc.double().cpu().numpy()
    for _ in range(3):
        kn, vn = (torch.randn(2, Hk, D, generator=gen).half().cuda() for _ in range(2))
        q = torch.randn(2, 1, Hk * G, D, generator=gen).half().cuda()
        slot = dst.long().gather(1, (cur.long() // P).view(-1, 1)).view(-1) * P + cur.long() % P
        f.cache.append(slot, kn, vn)
        cur += 1
        _, lse = f.cache.attend(dst, cur, q)
        assert f.cache.weights(dst, cur, q, lse, prev=acc, out=acc) is acc
        for i in range(2):
            for c, a in ((0, kn), (1, vn)):
                values[i][c] = np.concatenate([values[i][c], ref.q4_values(*ref.q4_encode(a[i].float().cpu().numpy()))[None]])
            T = len(values[i][0])
            want[i, :, :T] += ref.cache_weights(q[i].double().cpu().numpy(), values[i][0], lse[i].double().cpu().numpy(), 1 / math.sqrt(D))
    got = acc.double().cpu().numpy()
    assert (np.abs(got - want) <= (S_ERR + 1e-5) * want + 3 * 2.0 ** -22 * want).all()
    assert cur.tolist() == [203, 93] and not acc[0, :, 203:].any()


def test_out_may_be_the_query():
    import torch
    for dt, D, G, R in (("f16", 128, 4, 3), ("f32", 64, 8, 2), ("bf16", 256, 20, 2)):
        f = Filled([5000, 33, 0, 64], 2, D, 64, seed=5, dt=dt)
        q = torch.randn(4, R, 2 * G, D, generator=torch.Generator().manual_seed(6)).to(f.k.dtype).cuda()
        out, lse = f.cache.attend(f.table_t, f.lens_t, q)
        check_attend(out, lse, q, f, dt, 1 / math.sqrt(D))
        x = q.clone()
        same, z = f.cache.attend(f.table_t, f.lens_t, x, out=x)
        assert same is x and torch.equal(x, out) and torch.equal(z, lse)
