"""Attention over packed prompts and the weights of their keys (kvs_prompt_*) against plain 64-bit forms.

Tolerances: with A = sum p |v|, u the half step of the type and n keys: the
weights are rounded to the type (u A; f16 weights below 2^-14 lose up to
2^-25 each, n 2^-25 max|v| in all), the output is (u |out|), and the scores'
fp32 sums (at most D/16 + 4 additions in a row over sum |q k| scale <= 16 for
the unit-normal rows here) move a weight by at most 20 2^-23 16 = 4e-5, in
numerator and denominator: S = 8e-5 A.
"""
import math

import numpy as np
import pytest

import batch_ref as ref

pytestmark = pytest.mark.gpu

S_ERR = 8e-5


def _t(dt):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[dt]


def make(lens, Hk, G, D, dt, seed=0, lead=0, tail=0):
    """Fused rows [lead + sum + tail][Hq + 2 Hk][D] with NaN outside the prompts, as strided q, k, v, and cu."""
    import torch
    n = lead + sum(lens) + tail
    x = torch.randn(n, Hk * G + 2 * Hk, D, generator=torch.Generator().manual_seed(seed)).to(_t(dt))
    x[:lead] = math.nan
    x[n - tail:] = math.nan
    x = x.cuda()
    cu = torch.tensor(np.concatenate([[lead], lead + np.cumsum(lens)]), dtype=torch.int32).cuda()
    return x[:, :Hk * G], x[:, Hk * G:Hk * G + Hk], x[:, Hk * G + Hk:], cu


def check(out, lse, q, k, v, cu, dt, scale):
    import torch
    u = torch.finfo(_t(dt)).eps / 2
    o, z, qn, kn, vn = (x.double().cpu().numpy() for x in (out, lse, q, k, v))
    c = cu.tolist()
    for i in range(len(c) - 1):
        s = slice(c[i], c[i + 1])
        if c[i] == c[i + 1]:
            continue
        ro, rz, A = ref.prompt(qn[s], kn[s], vn[s], scale)
        sub = (c[i + 1] - c[i]) * 2.0 ** -25 * np.abs(vn[s]).max() if dt == "f16" else 0.0
        tol = u * np.abs(ro) + (u + S_ERR) * A + sub
        err = np.abs(o[s] - ro)
        assert (err <= tol).all(), (i, np.argwhere(~(err <= tol))[:4], np.nanmax(err / tol))
        assert np.abs(z[s] - rz).max() <= S_ERR


CASES = [  # D, Hk, G, lens
    (64, 2, 1, [1]),
    (64, 2, 4, [1, 2, 31, 129, 0, 300]),
    (64, 1, 64, [5, 70]),
    (128, 1, 1, [128, 1, 256, 257, 700]),
    (128, 2, 4, [1, 63, 64, 65, 500]),
    (128, 1, 6, [21, 22, 42, 43, 640]),
    (128, 1, 3, [1000]),
    (256, 1, 6, [1, 37, 64, 65, 300]),
    (256, 2, 1, [127, 129, 400]),
    (256, 1, 7, [90, 33, 18]),
    (256, 1, 50, [7, 30]),
    (256, 2, 5, [19, 20, 39, 200]),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D,Hk,G,lens", CASES)
def test_attend(D, Hk, G, lens, dt):
    import torch
    from host_streamed_paged_gb300 import kvs
    q, k, v, cu = make(lens, Hk, G, D, dt, seed=D + G, lead=3, tail=5)
    wide = torch.full((q.shape[0], Hk * G + 1, D), 7.0, dtype=_t(dt), device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out, _ = kvs.prompt_attend(q, k, v, cu, out=wide[:, :Hk * G], lse=lse)
    check(out, lse, q, k, v, cu, dt, 1 / math.sqrt(D))
    # rows of no prompt, and what lies between the rows, are left as they were
    assert (wide[:3] == 7).all() and (wide[-5:] == 7).all() and (wide[:, Hk * G:] == 7).all()
    assert (lse[:3] == 7).all() and (lse[-5:] == 7).all()


@pytest.mark.parametrize("n", [33, 256, 300])
def test_many_prompts(n):
    """More prompts than a warp has lanes, up to and past those that are ordered by work; the keys' weights as well."""
    import torch
    from host_streamed_paged_gb300 import kvs
    lens = np.random.default_rng(n).integers(0, 60, n).tolist()
    lens[n // 2] = 400
    q, k, v, cu = make(lens, 2, 3, 64, "f16", seed=n)
    out, lse = kvs.prompt_attend(q, k, v, cu)
    check(out, lse, q, k, v, cu, "f16", 1 / 8)
    got = kvs.prompt_weights(q, k, lse, cu, 400).double().cpu().numpy()
    qn, kn, zn = (x.double().cpu().numpy() for x in (q, k, lse))
    c = cu.tolist()
    for i, L in enumerate(lens):
        w = np.zeros((2, 400))
        if L:
            s = slice(c[i], c[i + 1])
            w[:, :L] = ref.prompt_weights(qn[s], kn[s], zn[s], 1 / 8, 0)
        assert (np.abs(got[i] - w) <= (5e-5 + L * 3 / 4 * 2.0 ** -24) * w + 1e-37).all(), i


def test_large_scores_move_the_maximum_late():
    """Keys whose scores grow along the prompt: O is rescaled again and again."""
    import torch
    from host_streamed_paged_gb300 import kvs
    for D, dt in ((64, "f16"), (128, "bf16"), (256, "f16")):
        q, k, v, cu = make([600], 1, 2, D, dt, seed=2)
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        q[..., 0] = 8.0
        k[..., 0] = (torch.arange(600, device="cuda") / 20).to(_t(dt))[:, None]
        out, lse = kvs.prompt_attend(q, k, v, cu, scale=0.5)
        u = torch.finfo(_t(dt)).eps / 2
        o, z, A = ref.prompt(*(x.double().cpu().numpy() for x in (q, k, v)), 0.5)
        # scores reach 8 * 30 * 0.5 + ...: sum |q k| scale <= 250, so S is 20 2^-23 250 twice = 1.2e-3
        assert (np.abs(out.double().cpu().numpy() - o) <= u * np.abs(o) + (u + 1.2e-3) * A + 1e-5).all()
        assert np.abs(lse.double().cpu().numpy() - z).max() <= 1.2e-3


def test_offsets_outside_the_rows_are_clamped():
    import torch
    from host_streamed_paged_gb300 import kvs
    q, k, v, cu = make([200], 1, 2, 64, "f16", seed=4)
    want, lse = kvs.prompt_attend(q, k, v, cu)
    got, _ = kvs.prompt_attend(q, k, v, torch.tensor([0, 1 << 30], dtype=torch.int32).cuda())
    assert torch.equal(want, got)
    mark = torch.full_like(want, 3.0)
    for odd in ([200, 100], [-5, -2], [300, 400]):
        kvs.prompt_attend(q, k, v, torch.tensor(odd, dtype=torch.int32).cuda(), out=mark)
    assert (mark == 3).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("window", [0, 1, 50])
@pytest.mark.parametrize("D,Hk,G,lens", CASES)
def test_weights(D, Hk, G, lens, window, dt):
    """exp(s - lse): the scores' error 4e-5 and ex2 (2^-22), fp32 sums of L G terms in chains of L G / 4."""
    import torch
    from host_streamed_paged_gb300 import kvs
    q, k, v, cu = make(lens, Hk, G, D, dt, seed=D + G, lead=3, tail=5)
    _, lse = kvs.prompt_attend(q, k, v, cu)
    width = max(lens) + 9
    prev = torch.rand(len(lens), Hk, width, generator=torch.Generator().manual_seed(1)).cuda()
    plain = kvs.prompt_weights(q, k, lse, cu, width, window=window)
    summed = kvs.prompt_weights(q, k, lse, cu, width, window=window, prev=prev)
    same = prev.clone()
    kvs.prompt_weights(q, k, lse, cu, width, window=window, prev=same, out=same)
    narrow = kvs.prompt_weights(q, k, lse, cu, 20, window=window)
    both = min(20, width)
    assert torch.equal(same, summed) and torch.equal(narrow[..., :both], plain[..., :both]) and not narrow[..., both:].any()
    qn, kn, zn, pn = (x.double().cpu().numpy() for x in (q, k, lse, prev))
    c = cu.tolist()
    for i, L in enumerate(lens):
        w = np.zeros((Hk, width))
        if L:
            s = slice(c[i], c[i + 1])
            w[:, :L] = ref.prompt_weights(qn[s], kn[s], zn[s], 1 / math.sqrt(D), window)
        tol = (5e-5 + L * G / 4 * 2.0 ** -24) * w + 1e-37
        assert (np.abs(plain[i].double().cpu().numpy() - w) <= tol).all(), i
        assert (np.abs(summed[i].double().cpu().numpy() - w - pn[i]) <= tol + 2.0 ** -22 * (w + pn[i])).all(), i


def test_weights_of_empty_prompts_are_what_was_there():
    import torch
    from host_streamed_paged_gb300 import kvs
    prev = torch.rand(3, 2, 5000, generator=torch.Generator().manual_seed(2)).cuda()
    for rows in (0, 4):  # no rows at all; rows of no prompt
        q, k = (torch.zeros(rows, h, 64, dtype=torch.float16, device="cuda") for h in (4, 2))
        cu = torch.zeros(4, dtype=torch.int32, device="cuda")
        lse = torch.zeros(rows, 4, device="cuda")
        assert torch.equal(kvs.prompt_weights(q, k, lse, cu, 5000, prev=prev), prev)
        assert not kvs.prompt_weights(q, k, lse, cu, 5000).any()
        assert kvs.prompt_attend(q, k, k, cu)[0].shape == q.shape


def test_batches_of_nothing():
    import torch
    from host_streamed_paged_gb300 import kvs
    cache = kvs.Q4Cache(page_tokens=32, n_kv_head=2, head_dim=64, n_pages=2)
    i32 = dict(dtype=torch.int32, device="cuda")
    none, table = torch.zeros(0, **i32), torch.zeros(0, 4, **i32)
    q = torch.zeros(0, 1, 4, 64, device="cuda")
    out, lse = cache.attend(table, none, q)
    assert out.shape == q.shape and lse.shape == q.shape[:3]
    w = cache.weights(table, none, q, lse)
    assert w.shape == (0, 2, 128)
    kept, lens, kw = cache.evict(table, table, none, w, 64)
    assert kept.shape == kw.shape == (0, 2, 64) and lens.shape == (0,)
    slots, rows = torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, 2, 64, device="cuda")
    cache.append(slots, rows, rows)
    assert cache.read(slots)[0].shape == rows.shape
    p, c = torch.zeros(0, 4, 64, dtype=torch.float16, device="cuda"), torch.zeros(1, **i32)
    o, z = kvs.prompt_attend(p, p[:, :2], p[:, :2], c)
    assert kvs.prompt_weights(p, p[:, :2], z, c, 9).shape == (0, 2, 9)
    torch.cuda.synchronize()


def test_replayed_graph_follows_the_offsets():
    import torch
    from host_streamed_paged_gb300 import kvs
    q, k, v, cu = make([300, 100, 57], 2, 2, 128, "bf16", seed=6)
    out, lse = torch.zeros(q.shape, dtype=q.dtype, device="cuda"), torch.zeros(q.shape[:2], device="cuda")
    w = torch.zeros(3, 2, 457, device="cuda")

    def step():
        kvs.prompt_attend(q, k, v, cu, out=out, lse=lse)
        kvs.prompt_weights(q, k, lse, cu, 457, out=w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in ([0, 300, 400, 457], [0, 1, 2, 457], [0, 0, 457, 457]):
        cu.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        o, z = kvs.prompt_attend(q, k, v, cu)
        assert torch.equal(o, out) and torch.equal(z, lse)
        assert torch.equal(w, kvs.prompt_weights(q, k, z, cu, 457))
