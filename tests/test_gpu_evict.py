"""kvs_q4_evict on the GPU: the kept tokens, their weights and their encoded rows are exact."""
import math

import numpy as np
import pytest

import batch_ref as ref
from test_gpu_q4 import Filled

pytestmark = pytest.mark.gpu


def run(lens, Hk, D, P, keep, sinks, recent, weights, seed=0):
    import torch
    f = Filled(lens, Hk, D, P, seed=seed, spare=2 + len(lens) * -(-keep // P))
    w = torch.from_numpy(weights).cuda()
    dst = torch.from_numpy(f.free[:len(lens) * -(-keep // P)].reshape(len(lens), -1).astype(np.int32).copy()).cuda()
    kept, new_lens, kw = f.cache.evict(f.table_t, dst, f.lens_t, w, keep, sinks=sinks, recent=recent)
    dn = dst.cpu().numpy().astype(np.int64)
    assert new_lens.tolist() == [min(n, keep) for n in lens]
    for i, n in enumerate(lens):
        m = min(n, keep)
        pos = np.arange(m)
        k, v = f.cache.read(torch.from_numpy(dn[i, pos // P] * P + pos % P).cuda())
        ks, vs, _ = f.seq(i)
        for h in range(Hk):
            want = ref.evict(weights[i, h, :n], keep, sinks, recent)
            got = kept[i, h].cpu().numpy()
            assert np.array_equal(got[:m], want), (i, h)
            assert (got[m:] == -1).all()
            assert np.array_equal(kw[i, h, :m].cpu().numpy(), weights[i, h, :n][want], equal_nan=True) and not kw[i, h, m:].any()
            assert np.array_equal(k[:, h].double().cpu().numpy() + 0.0, ks[want, h] + 0.0)
            assert np.array_equal(v[:, h].double().cpu().numpy() + 0.0, vs[want, h] + 0.0)
    return f


@pytest.mark.parametrize("D,P,Hk,keep,sinks,recent", [(64, 32, 2, 100, 4, 32), (128, 64, 3, 33, 0, 0), (256, 256, 1, 64, 1, 63),
                                                      (128, 128, 2, 1, 0, 0), (64, 64, 1, 257, 10, 0), (64, 32, 1, 40, 0, 40)])
def test_ragged_batch(D, P, Hk, keep, sinks, recent):
    lens = [0, 1, keep - 1, keep, keep + 1, 700, 99]
    rng = np.random.default_rng(keep)
    w = np.exp(2 * rng.standard_normal((len(lens), Hk, 800))).astype(np.float32)
    run(lens, Hk, D, P, keep, sinks, recent, w)


def test_ties_go_to_the_lowest_index_and_odd_values_have_an_order():
    lens = [500, 500, 500, 500]
    w = np.zeros((4, 1, 512), np.float32)          # row 0: all equal
    rng = np.random.default_rng(2)
    w[1] = rng.integers(0, 3, 512)                 # few distinct values
    w[2] = rng.choice([0.0, -0.0, 1.0, -1.0, np.inf, -np.inf, np.nan, 1e-40], 512)
    w[3] = np.nan
    run(lens, 1, 64, 64, 130, 3, 17, w)


@pytest.mark.parametrize("T", [9000, 40000, 140001, 300007, 400001])
def test_long_sequences_shared_by_a_cluster(T):
    lens = [T, 8191, 60]
    rng = np.random.default_rng(T)
    w = np.exp(3 * rng.standard_normal((3, 2, T + 3))).astype(np.float32)
    w[0, 1] = np.round(w[0, 1])                    # long runs of ties across the shares
    run(lens, 2, 64, 256, 1500, 4, 100, w)


def test_a_sequence_below_the_budget_may_keep_its_pages():
    import torch
    f = Filled([90, 30], 2, 128, 64, seed=4)
    before = f.cache.read(torch.from_numpy(f.slots).cuda())
    w = torch.rand(2, 2, 128).cuda()
    kept, lens, _ = f.cache.evict(f.table_t, f.table_t, f.lens_t, w, 100)
    after = f.cache.read(torch.from_numpy(f.slots).cuda())
    assert lens.tolist() == [90, 30] and all(torch.equal(a, b) for a, b in zip(before, after))
    assert torch.equal(kept[0, 0, :90].cpu(), torch.arange(90, dtype=torch.int32))


def test_pages_outside_the_pool():
    import torch
    f = Filled([200, 200], 1, 64, 64, seed=5, spare=6)
    w = torch.rand(2, 1, 256).cuda()
    dst = torch.from_numpy(f.free[:4].reshape(2, 2).astype(np.int32).copy()).cuda()
    dst[0, 1] = 1 << 22
    f.table_t[1, 0] = -7                           # the second sequence's first page
    before = f.cache.pages.clone()
    kept, _, _ = f.cache.evict(f.table_t, dst, f.lens_t, w, 128, sinks=8)
    page = f.cache.page_bytes
    changed = {i for i in range(f.cache.n_pages) if not torch.equal(before[i * page:(i + 1) * page], f.cache.pages[i * page:(i + 1) * page])}
    assert changed <= {int(dst[0, 0]), int(dst[1, 0]), int(dst[1, 1])}
    k, _ = f.cache.read(int(dst[1, 0]) * 64 + torch.arange(8, device="cuda"))
    assert not k.any()                             # the sinks came from the bad page
    assert kept[1, 0, :8].tolist() == list(range(8))


def test_prompt_to_cache_to_eviction_to_decode():
    """The operators together: packed prompts are attended, cached and weighed, decode steps add their weight, the
    cache is cut back, and decode goes on over what stayed."""
    import torch
    from host_streamed_paged_gb300 import kvs
    lens, Hk, G, D, P, keep = [333, 40, 150], 2, 4, 128, 32, 96
    gen = torch.Generator().manual_seed(1)
    total, n = sum(lens), len(lens)
    q, k, v = (torch.randn(total, h, D, generator=gen).half().cuda() for h in (Hk * G, Hk, Hk))
    cu = torch.tensor([0, 333, 373, 523], dtype=torch.int32).cuda()
    out, lse = kvs.prompt_attend(q, k, v, cu)
    pages_per = -(-(max(lens) + 8) // P)
    cache = kvs.Q4Cache(page_tokens=P, n_kv_head=Hk, head_dim=D, n_pages=2 * n * pages_per)
    table = torch.arange(n * pages_per, dtype=torch.int32).view(n, pages_per).cuda()
    dst = table + n * pages_per
    slots = torch.cat([table[i].long().cpu()[torch.arange(m) // P] * P + torch.arange(m) % P for i, m in enumerate(lens)]).cuda()
    cache.append(slots, k, v)
    width = pages_per * P
    w = kvs.prompt_weights(q, k, lse, cu, width, window=32)
    cur = torch.tensor(lens, dtype=torch.int32).cuda()
    rows = {i: [x[int(cu[i]):int(cu[i + 1])] for x in (k, v)] for i in range(n)}

    def step(table, cur, w):
        kn, vn = torch.randn(n, Hk, D, generator=gen).half().cuda(), torch.randn(n, Hk, D, generator=gen).half().cuda()
        qn = torch.randn(n, 1, Hk * G, D, generator=gen).half().cuda()
        at = table.long().gather(1, (cur.long() // P).view(-1, 1)).view(-1) * P + cur.long() % P
        cache.append(at, kn, vn)
        cur += 1
        o, z = cache.attend(table, cur, qn)
        if w is not None:
            cache.weights(table, cur, qn, z, prev=w, out=w)
        return qn, kn, vn, o, z

    values = {}
    for i in range(n):
        values[i] = [ref.q4_values(*ref.q4_encode(x.float().cpu().numpy())) for x in rows[i]]
    ws = {i: ref.prompt_weights(q[int(cu[i]):int(cu[i + 1])].double().cpu().numpy(), rows[i][0].double().cpu().numpy(),
                                lse[int(cu[i]):int(cu[i + 1])].double().cpu().numpy(), 1 / math.sqrt(D), 32) for i in range(n)}

    def follow(qn, kn, vn, o, z, w):
        for i in range(n):
            for c, x in ((0, kn), (1, vn)):
                row = ref.q4_values(*ref.q4_encode(x[i].float().cpu().numpy()))[None]
                values[i][c] = np.concatenate([values[i][c], row])
            qq = qn[i].double().cpu().numpy()
            ro, rz, mag = ref.attend(qq, *values[i], 1 / math.sqrt(D))
            # f16 weights and output (2^-11 each), the scores' error as in test_gpu_q4
            assert (np.abs(o[i].double().cpu().numpy() - ro) <= 2.0 ** -11 * np.abs(ro) + (2.0 ** -11 + 3e-4) * mag).all()
            assert np.abs(z[i].double().cpu().numpy() - rz).max() <= 2e-4
            if w is not None:
                T = len(values[i][0])
                ws[i] = np.concatenate([ws[i], np.zeros((Hk, 1))], 1) + ref.cache_weights(qq, values[i][0], rz, 1 / math.sqrt(D))
                assert np.abs(w[i, :, :T].double().cpu().numpy() - ws[i]).max() <= 4e-4 * ws[i].max()

    for _ in range(3):
        follow(*step(table, cur, w), w)
    kept, cur2, w2 = cache.evict(table, dst, cur, w, keep, sinks=4, recent=16)
    for i in range(n):
        T = int(cur[i])
        m = min(T, keep)
        assert int(cur2[i]) == m
        wi = w[i].cpu().numpy()
        idx = [ref.evict(wi[h, :T], keep, 4, 16) for h in range(Hk)]
        for h in range(Hk):
            assert np.array_equal(kept[i, h, :m].cpu().numpy(), idx[h])
        values[i] = [np.stack([x[idx[h], h] for h in range(Hk)], 1) for x in values[i]]
    for _ in range(2):
        follow(*step(dst, cur2, None), None)
