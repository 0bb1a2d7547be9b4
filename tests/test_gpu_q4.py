"""The 4-bit page cache on the GPU (kvs_q4_append, read, attend, weights) against plain 64-bit forms.

Tolerances, from the arithmetic the kernels state.  With A = sum p |v| per
output element, u the half step of the output type, w11 = 2^-11 the half step
of f16 (softmax weight x V scale of 16-bit calls):
  out: |err| <= u |out| + w11 A + s A + a A8, where s bounds the scores' error
       (it moves numerator and denominator) and a the fp32 sums of 0..15 codes
       whose offset is taken back (A8 = sum p 8 |scale| >= what cancels).
A score is a sum of D products of codes up to 15: with at most D/8 fp32
additions in a row and the sums bounded by 15 sum |q| scale_k, its error is
at most D/8 2^-24 15 scale sum |q| d_k, below 1.5e-4 for the inputs here (unit
normal rows, D <= 256: sum |q| <= 260, d_k <= 0.6, scale 1/16); a is D/8 2^-24
15/8 rounded up to 4e-6.
"""
import math

import numpy as np
import pytest

import batch_ref as ref

pytestmark = pytest.mark.gpu

S_ERR = 1.5e-4
A_ERR = 4e-6
DT = ["f32", "f16", "bf16"]


def _t(dt):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dt]


def half_step(dt):
    import torch
    return torch.finfo(_t(dt)).eps / 2


class Filled:
    """A cache of sequences of the given lengths on shuffled pages, appended through the library, and its values."""

    def __init__(self, lens, Hk, D, P, seed=0, dt="f32", spare=2, extra=0, v_scale=1.0):
        import torch
        from host_streamed_paged_gb300 import kvs
        rng = np.random.default_rng(seed)
        self.lens, self.P = lens, P
        width = max(1, max(-(-n // P) for n in lens)) + extra
        n_pages = sum(-(-n // P) for n in lens) + spare
        order = rng.permutation(n_pages)
        self.table = np.full((len(lens), width), -1, np.int32)
        at, slots = 0, []
        for i, n in enumerate(lens):
            m = -(-n // P)
            self.table[i, :m] = order[at:at + m]
            at += m
            pos = np.arange(n)
            slots.append(self.table[i, pos // P].astype(np.int64) * P + pos % P)
        self.free = order[at:]
        self.cache = kvs.Q4Cache(page_tokens=P, n_kv_head=Hk, head_dim=D, n_pages=n_pages)
        self.cache.pages.fill_(0xff)  # never-written tokens hold NaN scales
        self.k = torch.from_numpy(rng.standard_normal((sum(lens), Hk, D), np.float32)).to(_t(dt))
        self.v = (v_scale * torch.from_numpy(rng.standard_normal((sum(lens), Hk, D), np.float32))).to(_t(dt))
        self.slots = np.concatenate(slots) if slots else np.zeros(0, np.int64)
        self.cache.append(torch.from_numpy(self.slots).cuda(), self.k.cuda(), self.v.cuda())
        self.kv = [ref.q4_values(*ref.q4_encode(x.float().numpy())) for x in (self.k, self.v)]
        self.vs = np.abs(ref.q4_encode(self.v.float().numpy())[1].astype(np.float64)).repeat(32, -1)
        self.table_t = torch.from_numpy(self.table).cuda()
        self.lens_t = torch.tensor(lens, dtype=torch.int32).cuda()

    def seq(self, i):
        a = sum(self.lens[:i])
        return [x[a:a + self.lens[i]] for x in (*self.kv, self.vs)]


def check_attend(out, lse, q, filled, dt, scale, skip=()):
    out, lse, q = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    u = half_step(dt)
    for i in range(len(filled.lens)):
        if i in skip:
            continue
        k, v, vs = filled.seq(i)
        o, z, A = ref.attend(q[i], k, v, scale)
        _, _, A8 = ref.attend(q[i], k, 8 * vs, scale)
        tol = u * np.abs(o) + ((2.0 ** -22 if dt == "f32" else 2.0 ** -11) + S_ERR) * A + A_ERR * A8
        bad = np.abs(out[i] - o) > tol
        assert not bad.any(), (i, filled.lens[i], np.abs(out[i] - o).max(), np.argwhere(bad)[:4])
        fin, none = np.isfinite(z), z == -np.inf
        assert np.array_equal(fin, np.isfinite(lse[i])) and np.array_equal(none, lse[i] == -np.inf)
        assert np.abs(lse[i][fin] - z[fin]).max(initial=0) <= S_ERR + 1e-5
        assert (out[i][none] == 0).all()
        nan = np.isnan(z)  # a row whose query holds an infinity
        assert np.isnan(out[i][nan]).all() and np.isnan(lse[i][nan]).all()


# ------------------------------------------------------------------ append and read

@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("D,P,Hk", [(64, 32, 3), (128, 64, 2), (256, 256, 1), (128, 256, 8)])
def test_append_stores_the_stated_bytes_and_read_returns_them(D, P, Hk, dt):
    import torch
    from host_streamed_paged_gb300 import kvs
    rng = np.random.default_rng(D + P)
    n_pages, n = 3, 70
    cache = kvs.Q4Cache(page_tokens=P, n_kv_head=Hk, head_dim=D, n_pages=n_pages)
    cache.pages.fill_(7)
    slots = rng.permutation(n_pages * P)[:n].astype(np.int64)
    n = len(slots)
    fused = rng.standard_normal((n, 2 * Hk, D)).astype(np.float32) * np.exp(rng.standard_normal((n, 2 * Hk, 1))).astype(np.float32)
    fused[0] = 0                                   # zero blocks
    fused[1, :, :32] = np.where(np.arange(32) % 2, 3.0, -3.0)  # ties of the largest magnitude: the first decides
    fused[2, :, 0:32] = 1e-30                      # a scale that fp16 flushes to zero
    fused[3, :, 5] = 60000.0
    x = torch.from_numpy(fused).to(_t(dt))
    xs = x.cuda()
    cache.append(torch.from_numpy(slots).cuda(), xs[:, :Hk], xs[:, Hk:])  # strided rows
    enc = [ref.q4_encode(x[:, a:a + Hk].float().numpy()) for a in (0, Hk)]
    want = np.full((n_pages, Hk, P // 32, 36 * D), 7, np.uint8)
    full = [np.zeros((n_pages * P, Hk, D // 32, 32), np.uint8), np.zeros((n_pages * P, Hk, D // 32), np.float16)] * 2
    full = [a.copy() for a in full]
    for c in range(2):
        full[2 * c][slots], full[2 * c + 1][slots] = enc[c]
    written = np.zeros(n_pages * P, bool)
    written[slots] = True
    mark = [np.ones((32, D // 32, 32), np.uint8), np.ones((32, D // 32), np.float16)]
    for pg in range(n_pages):
        for h in range(Hk):
            for ti in range(P // 32):
                s = slice(pg * P + ti * 32, pg * P + ti * 32 + 32)
                tile = ref.q4_tile(full[0][s, h], full[1][s, h], full[2][s, h], full[3][s, h])
                on = written[s]
                mk = ref.q4_tile(mark[0] * on[:, None, None], mark[1] * on[:, None], mark[0] * on[:, None, None], mark[1] * on[:, None])
                # bytes of a written token: its codes carry the mark 0x11, its scales fp16 1.0 (0x3c00)
                place = mk != 0
                hv = place.view(np.uint16) != 0
                place[16 * D:18 * D] = np.repeat(hv[8 * D:9 * D], 2)
                place[34 * D:] = np.repeat(hv[17 * D:], 2)
                want[pg, h, ti][place] = tile[place]
    got = cache.pages.cpu().numpy().reshape(want.shape)
    assert np.array_equal(got, want)
    for rt in DT:
        k, v = cache.read(torch.from_numpy(slots).cuda(), _t(rt))
        for c, y in enumerate((k, v)):
            val = torch.from_numpy(ref.q4_values(*enc[c])).to(_t(rt))
            assert torch.equal(y.cpu() + 0.0, val + 0.0)


def test_slots_outside_the_pool_are_skipped_and_read_as_zero():
    import torch
    from host_streamed_paged_gb300 import kvs
    cache = kvs.Q4Cache(page_tokens=32, n_kv_head=2, head_dim=64, n_pages=2)
    before = cache.pages.clone()
    slots = torch.tensor([-1, 64, -(1 << 40), 1 << 40, 65], dtype=torch.int64).cuda()
    k = torch.randn(5, 2, 64).cuda()
    cache.append(slots, k, k)
    assert torch.equal(before, cache.pages)
    k, v = cache.read(slots)
    assert not k.any() and not v.any()
    cache.append(slots[:0], k[:0], v[:0])
    assert cache.read(slots[:0])[0].shape == (0, 2, 64)


# ------------------------------------------------------------------ attention

LENS = [0, 1, 2, 31, 32, 33, 64, 65, 200, 257, 1000]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("D,P,Hk,G,R", [(64, 32, 2, 1, 1), (64, 64, 1, 5, 3), (128, 64, 2, 4, 1), (128, 128, 1, 8, 8),
                                        (128, 256, 3, 3, 4), (256, 256, 2, 6, 1), (256, 64, 1, 6, 6), (64, 128, 1, 64, 1)])
def test_attend_ragged_batch(D, P, Hk, G, R, dt):
    import torch
    f = Filled(LENS, Hk, D, P, seed=D + R, dt=dt)
    fused = torch.randn(len(LENS), R, Hk * G + 3, D, generator=torch.Generator().manual_seed(5)).to(_t(dt)).cuda()
    q = fused[:, :, :Hk * G]  # strided rows
    out, lse = f.cache.attend(f.table_t, f.lens_t, q)
    check_attend(out, lse, q, f, dt, 1 / math.sqrt(D))


@pytest.mark.parametrize("dt,D,G,R", [("bf16", 128, 4, 1), ("f32", 64, 2, 3), ("f16", 256, 6, 1), ("f16", 128, 8, 2)])
def test_attend_one_long_sequence_is_split_and_joined(dt, D, G, R):
    import torch
    f = Filled([20001], 1, D, 64, seed=3, dt=dt)
    q = (3 * torch.randn(1, R, G, D, generator=torch.Generator().manual_seed(6))).to(_t(dt)).cuda()
    out, lse = f.cache.attend(f.table_t, f.lens_t, q, scale=0.5 / math.sqrt(D))
    check_attend(out, lse, q, f, dt, 0.5 / math.sqrt(D))
    again = f.cache.attend(f.table_t, f.lens_t, q, scale=0.5 / math.sqrt(D))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("scale", [1e-5, 1.0, 3000.0])
def test_attend_values_of_any_size(scale):
    """V scales from f16 subnormals to large: the running reference keeps the weights' precision (bounds as above:
    relative to the values; a subnormal f16 scale is exact as it stands)."""
    import torch
    f = Filled([700, 45], 2, 128, 64, seed=8, v_scale=scale)
    q = torch.randn(2, 1, 8, 128, generator=torch.Generator().manual_seed(7)).cuda()
    for dt in DT:
        qq = q.to(_t(dt))
        if dt == "f16" and scale < 1e-2:
            continue  # the output type itself has no such values
        out, lse = f.cache.attend(f.table_t, f.lens_t, qq)
        check_attend(out, lse, qq, f, dt, 1 / math.sqrt(128))


def test_attend_many_sequences():
    import torch
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 150, 700)]
    f = Filled(lens, 1, 64, 32, seed=9, dt="f16")
    q = torch.randn(700, 1, 2, 64, generator=torch.Generator().manual_seed(8)).half().cuda()
    out, lse = f.cache.attend(f.table_t, f.lens_t, q)
    check_attend(out, lse, q, f, "f16", 1 / 8)


def test_attend_large_and_tiny_queries():
    import torch
    f = Filled([300], 1, 64, 64, seed=10)
    for mag, dt in ((1e-4, "bf16"), (30000.0, "f16"), (8000.0, "f16"), (1e-3, "f32"), (1e6, "f32")):
        q = (mag * torch.randn(1, 1, 4, 64, generator=torch.Generator().manual_seed(9))).to(_t(dt)).cuda()
        out, lse = f.cache.attend(f.table_t, f.lens_t, q, scale=0.125 / mag)
        check_attend(out, lse / 1.0, q, f, dt, 0.125 / mag)


def test_bad_pages_make_their_sequence_nan_and_no_other():
    import torch
    lens = [300, 100, 500]
    for bad in (-1, 1 << 20):
        f = Filled(lens, 2, 128, 64, seed=11)
        f.table_t[1, 1] = bad
        q = torch.randn(3, 1, 4, 128).cuda()
        out, lse = f.cache.attend(f.table_t, f.lens_t, q)
        assert out[1].isnan().all() and lse[1].isnan().all()
        check_attend(out, lse, q, f, "f32", 1 / math.sqrt(128), skip=(1,))
        w = f.cache.weights(f.table_t, f.lens_t, q, torch.nan_to_num(lse))
        assert w[1, :, 64:96].isnan().all() and not w[1, :, :64].isnan().any() and not w[0].isnan().any()


def test_lengths_are_clamped_to_the_table():
    import torch
    f = Filled([128, 64], 1, 64, 64, seed=12)
    long = torch.tensor([1 << 30, 64], dtype=torch.int32).cuda()
    q = torch.randn(2, 1, 2, 64).cuda()
    a, b = f.cache.attend(f.table_t, long, q), f.cache.attend(f.table_t, f.lens_t, q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    neg = torch.tensor([-5, 64], dtype=torch.int32).cuda()
    out, lse = f.cache.attend(f.table_t, neg, q)
    assert not out[0].any() and (lse[0] == -math.inf).all() and torch.equal(out[1], b[0][1])


def test_attend_and_weights_in_a_replayed_graph_follow_the_lengths():
    import torch
    f = Filled([500, 90], 2, 128, 64, seed=13, dt="bf16")
    q = torch.randn(2, 1, 8, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    out, lse = torch.empty_like(q), torch.empty(2, 1, 8, device="cuda")
    w = torch.zeros(2, 2, 512, device="cuda")
    lens = f.lens_t.clone()

    def step():
        f.cache.attend(f.table_t, lens, q, out=out, lse=lse)
        f.cache.weights(f.table_t, lens, q, lse, prev=w, out=w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in ([500, 90], [33, 0], [1, 64]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        w.zero_()
        graph.replay()
        want = f.cache.attend(f.table_t, lens, q)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(w, f.cache.weights(f.table_t, lens, q, lse, width=512))


def test_two_streams_at_once():
    import torch
    f = Filled([9000, 70], 2, 128, 64, seed=14, dt="f16")
    qs = [torch.randn(2, 1, 8, 128, generator=torch.Generator().manual_seed(i)).half().cuda() for i in range(2)]
    want = [f.cache.attend(f.table_t, f.lens_t, q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(f.cache.attend(f.table_t, f.lens_t, qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(z, want[i][1]) for o, z in got[i])


def test_two_threads_on_one_stream():
    """A call is two launches; another thread's may come between them."""
    import threading
    import torch
    f = Filled([9000, 70], 2, 128, 64, seed=15, dt="f16")
    qs = [torch.randn(2, 1, 8, 128, generator=torch.Generator().manual_seed(i)).half().cuda() for i in range(2)]
    want = [f.cache.attend(f.table_t, f.lens_t, q) for q in qs]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        for _ in range(300):
            got[i].append(f.cache.attend(f.table_t, f.lens_t, qs[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 300 and all(torch.equal(o, want[i][0]) and torch.equal(z, want[i][1]) for o, z in got[i])


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("D,P,Hk,G,R", [(64, 32, 2, 1, 1), (128, 64, 2, 4, 1), (128, 128, 1, 8, 5), (256, 256, 2, 6, 3), (64, 64, 1, 9, 7),
                                         (64, 32, 2, 12, 2), (128, 64, 2, 6, 4), (128, 32, 1, 10, 4), (256, 128, 1, 20, 2)])
def test_weights_are_added_to_prev(D, P, Hk, G, R, dt):
    """exp(s - lse) with the scores' error S_ERR (relative), the lse as given, fp32 sums of R G terms."""
    import torch
    f = Filled(LENS, Hk, D, P, seed=D + R, dt=dt)
    gen = torch.Generator().manual_seed(5)
    q = torch.randn(len(LENS), R, Hk * G, D, generator=gen).to(_t(dt)).cuda()
    scale = 1 / math.sqrt(D)
    lse = f.cache.attend(f.table_t, f.lens_t, q)[1]
    width = f.table.shape[1] * P + 5
    prev = torch.rand(len(LENS), Hk, width, generator=gen).cuda()
    got = f.cache.weights(f.table_t, f.lens_t, q, lse, prev=prev)
    plain = f.cache.weights(f.table_t, f.lens_t, q, lse, width=width)
    narrow = f.cache.weights(f.table_t, f.lens_t, q, lse, width=40)
    same = prev.clone()
    assert f.cache.weights(f.table_t, f.lens_t, q, lse, prev=same, out=same) is same
    assert torch.equal(same, got) and torch.equal(narrow, plain[..., :40])
    qn, zn, pn = q.double().cpu().numpy(), lse.double().cpu().numpy(), prev.double().cpu().numpy()
    for i, T in enumerate(LENS):
        w = np.zeros((Hk, width))
        w[:, :T] = ref.cache_weights(qn[i], f.seq(i)[0], zn[i], scale)
        tol = (S_ERR + 1e-5) * w
        assert (np.abs(plain[i].double().cpu().numpy() - w) <= tol + 1e-37).all()
        assert (np.abs(got[i].double().cpu().numpy() - (w + pn[i])) <= tol + 2.0 ** -22 * (w + pn[i])).all()
