"""Rotary positions and the norm before them (kvs_rotate, kvs_norm_rotate) against a plain 64-bit form.

Tolerances.  An angle reaches sincospif as a fp32 number of half turns, off by 2^-25 and what the 64-bit product cuts off
(2^-31): 1e-7 radians; sine and cosine come within 2 units of 2^-24 (1.2e-7).  With |u| + |v| of a pair and fp32 products
and sums (3 2^-24), an output is off by at most magnitude (|u| + |v|) 5e-7 before its rounding (half a step of its type).
A norm's sum of squares has at most 20 additions in a row, its root half of that error, the products 2 more roundings:
1.5e-6 of the value.
"""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from test_gpu_q4 import DT, _t, half_step
from test_rotary_plan import PI

pytestmark = pytest.mark.gpu


def angles(pos, freqs):
    """[n][pairs] radians in -pi .. pi: each product in rational numbers, reduced by turns, then a double."""
    turns = [Fraction(f) / (2 * PI) for f in freqs]
    out = np.zeros((len(pos), len(freqs)))
    for i, p in enumerate(pos):
        for j, t in enumerate(turns):
            x = int(p) * t
            x -= math.floor(x + Fraction(1, 2))
            out[i, j] = float(x * 2 * PI)
    return out


def reference(x, pos, r, weight=None, eps=None):
    """float64 rows [n][H][D] turned; and |u| + |v| of each element's pair, times magnitude."""
    x = x.double().cpu().numpy()
    if eps is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * weight.double().cpu().numpy()
    a = angles(pos, r.freqs)[:, None]
    n = r.rot_dim
    u, v = (slice(0, n, 2), slice(1, n, 2)) if r.interleaved else (slice(0, n // 2), slice(n // 2, n))
    y, size = x.copy(), np.abs(x)
    y[..., u] = r.magnitude * (x[..., u] * np.cos(a) - x[..., v] * np.sin(a))
    y[..., v] = r.magnitude * (x[..., v] * np.cos(a) + x[..., u] * np.sin(a))
    size[..., u] = size[..., v] = abs(r.magnitude) * (np.abs(x[..., u]) + np.abs(x[..., v]))
    return y, size


def check(got, x, pos, r, dt, weight=None, eps=None):
    y, size = reference(x, pos, r, weight, eps)
    err = np.abs(got.double().cpu().numpy() - y)
    tiny = {"f32": 1.5e-45, "f16": 3e-8, "bf16": 1e-40}[dt]  # half of the type's smallest number
    tol = half_step(dt) * np.abs(y) + (5e-7 if eps is None else 2e-6) * size + tiny
    assert (err <= tol).all(), (np.argwhere(~(err <= tol))[:4], np.nanmax(err / tol))
    if eps is None:  # the other dims are copied
        assert np.array_equal(got[..., r.rot_dim:].cpu().float().numpy(), x[..., r.rot_dim:].cpu().float().numpy())


def rows(n, Hq, Hk, D, dt, seed=0):
    import torch
    x = torch.randn(n, Hq + Hk + 1, D, generator=torch.Generator().manual_seed(seed)).to(_t(dt)).cuda()
    return x[:, :Hq], x[:, Hq:Hq + Hk]


SHAPES = [  # D, rot, Hq, Hk, n
    (64, 64, 4, 2, 5), (64, 16, 1, 1, 1), (64, 48, 9, 3, 77), (128, 128, 32, 8, 33), (128, 32, 6, 1, 300), (128, 112, 5, 5, 7), (128, 0, 3, 1, 4),
    (256, 256, 24, 4, 19), (256, 64, 7, 1, 64), (256, 176, 2, 2, 9),
]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,Hq,Hk,n", SHAPES)
def test_rotate_and_norm_rotate(D, rot, Hq, Hk, n, interleaved, dt):
    import torch
    from host_streamed_paged_gb300 import kvs
    r = kvs.Rotary(D, rot_dim=rot, base=10000.0, interleaved=interleaved, scaling="yarn" if rot and n % 2 else None, factor=8, context=512)
    q, k = rows(n, Hq, Hk, D, dt, seed=n)
    pos = torch.randint(0, 200000, (n,), generator=torch.Generator().manual_seed(1))
    p = pos.to(torch.int32 if n % 2 else torch.int64).cuda()
    for got, x in zip(r.rotate(p, q, k), (q, k)):
        check(got, x, pos.tolist(), r, dt)
    g = torch.Generator().manual_seed(2)
    for wt in (dt, "f32", "bf16"):
        wq, wk = (torch.randn(D, generator=g).to(_t(wt)).cuda() for _ in range(2))
        for got, x, w in zip(r.norm_rotate(p, q, k, wq, wk, eps=1e-5), (q, k), (wq, wk)):
            check(got, x, pos.tolist(), r, dt, w, 1e-5)
    got, none = r.norm_rotate(p, q, q_weight=wq)
    assert none is None
    check(got, q, pos.tolist(), r, dt, wq, 1e-6)
    for got, x, w in zip(r.norm_rotate(p, q, k, None, wk), (q, k), (None, wk)):
        check(got, x, pos.tolist(), r, dt, w, 1e-6)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    """The angle is exact at any int64 position: to the double that a frequency is, times the position."""
    import torch
    from host_streamed_paged_gb300 import kvs
    r = kvs.Rotary(128, freqs=[2.0 ** -i for i in range(32)], interleaved=interleaved)  # exact frequencies
    pos = [0, 1, -1, 1 << 20, (1 << 24) + 1, -(1 << 30), (1 << 31) - 1, 1 << 31, (1 << 34) + 12345]
    q, k = rows(len(pos), 4, 2, 128, "f32")
    p = torch.tensor(pos).cuda()
    # turns are doubles of 53 bits, cut at 2^-64: position * 2^-53 of a turn and the angle is off by 2 pi times that
    y, size = reference(q, pos, r)
    off = np.abs(np.array(pos, dtype=np.float64))[:, None, None] * 2.0 ** -53 * 2 * math.pi
    err = np.abs(r.rotate(p, q)[0].double().cpu().numpy() - y)
    assert (err <= 2.0 ** -24 * np.abs(y) + (5e-7 + off) * size).all()
    back = r.rotate(-p, r.rotate(p, q)[0])[0]  # a turn back
    assert (back - q).abs().max() <= 4e-6


@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_angles_of_very_far_positions(base):
    """Turns are off by half of their last bit, 2^-65 of a turn, position times (2^-13 of a turn at 2^52)."""
    import torch
    from host_streamed_paged_gb300 import kvs
    r = kvs.Rotary(128, base=base)
    pos = [1 << 36, -(1 << 40) - 7, (1 << 44) + 12345, (1 << 48) - 1, -(1 << 52) + 3]
    q, k = rows(len(pos), 3, 2, 128, "f32")
    y, size = reference(q, pos, r)
    off = np.abs(np.array(pos, dtype=np.float64))[:, None, None] * 2.0 ** -65 * 2 * math.pi
    err = np.abs(r.rotate(torch.tensor(pos).cuda(), q)[0].double().cpu().numpy() - y)
    assert (err <= 2.0 ** -24 * np.abs(y) + (5e-7 + off) * size).all()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_row_may_be_its_own_output(D, dt):
    import torch
    from host_streamed_paged_gb300 import kvs
    for interleaved in (False, True):
        r = kvs.Rotary(D, rot_dim=D // 2, interleaved=interleaved)
        q, k = rows(40, 5, 2, D, dt)
        pos = torch.arange(40, device="cuda") * 1001
        want, wn = r.rotate(pos, q, k), r.norm_rotate(pos, q, k)
        store = torch.full((40, 9, D), 7.0, dtype=_t(dt), device="cuda")
        for call, w in ((r.rotate, want), (r.norm_rotate, wn)):
            store[:, 1:6], store[:, 6:8] = q, k
            a, b = store[:, 1:6], store[:, 6:8]
            got = call(pos, a, b, out=(a, b))
            assert got[0] is a and torch.equal(a, w[0]) and torch.equal(b, w[1]) and (store[:, 0] == 7).all() and (store[:, 8] == 7).all()


def test_rows_of_spans():
    """[sequences][rows][heads][D] with positions [sequences][rows], as Q4Cache.attend takes its queries."""
    import torch
    from host_streamed_paged_gb300 import kvs
    r = kvs.Rotary(128)
    q, _ = rows(12, 8, 1, 128, "bf16")
    pos = torch.arange(12, device="cuda").view(4, 3) * 77
    got, _ = r.rotate(pos, q.unflatten(0, (4, 3)))
    assert got.shape == (4, 3, 8, 128) and torch.equal(got.flatten(0, 1), r.rotate(pos.flatten(), q)[0])
    assert r.rotate(pos[:0], q[:0].unflatten(0, (0, 3)))[0].shape == (0, 3, 8, 128)


@pytest.mark.parametrize("n", [1, 31, 2433, 20000])
def test_row_counts_around_the_jobs_of_a_launch(n):
    import torch
    from host_streamed_paged_gb300 import kvs
    r = kvs.Rotary(64, interleaved=True)
    q, k = rows(n, 9, 2, 64, "f16")
    pos = torch.arange(n, device="cuda") * 3
    got, want = r.rotate(pos, q, k), r.rotate(pos.int(), q.contiguous(), k.contiguous())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for i in (0, n // 2, n - 1):
        one = r.rotate(pos[i:i + 1], q[i:i + 1], k[i:i + 1])
        assert torch.equal(one[0][0], got[0][i]) and torch.equal(one[1][0], got[1][i])


@pytest.mark.parametrize("dt,size,eps", [("f32", 1e-30, 0.0), ("f32", 1e-25, 0.0), ("f32", 1e25, 1e-6), ("f32", 3e37, 0.0), ("bf16", 1e30, 1e-6), ("bf16", 1e-30, 0.0),
                                         ("f16", 6e4, 1e-6), ("f16", 1e-6, 0.0), ("f32", 1e-12, 1e-6), ("bf16", 1e-20, 1e-30)])
def test_norms_of_any_size(dt, size, eps):
    import torch
    from host_streamed_paged_gb300 import kvs
    r = kvs.Rotary(128, rot_dim=64)
    x = torch.randn(6, 4, 128, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    x[2, 1] = 0
    if eps == 0:
        x[2, 1, 5] = 1
    q = (x / x.abs().max() * size).to(_t(dt)).cuda()
    pos = torch.arange(6)
    check(r.norm_rotate(pos.cuda(), q, eps=eps)[0], q, pos.tolist(), r, dt, None, eps)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("size,eps", [(3e-39, 0.0), (1e-40, 0.0), (1e-42, 0.0), (1e-44, 0.0), (1e-42, 1e-45), (1e-40, 1e-45), (3e38, 0.0)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_norms_of_subnormal_rows(D, size, eps, dt):
    """Their roots' reciprocals pass fp32, the values do not; and a row with one large element beside small ones."""
    import torch
    from host_streamed_paged_gb300 import kvs
    r = kvs.Rotary(D, rot_dim=32)
    x = torch.randn(6, 3, D, generator=torch.Generator().manual_seed(D), dtype=torch.float64)
    x = x / x.abs().max() * size
    x[1, 1] = 0
    x[1, 1, 7] = -size
    x[4, 2] = size * 2.0 ** -20
    x[4, 2, D - 1] = size
    q = x.to(_t(dt))
    keep = (q != 0).any(-1)  # (a head of zeros has no norm where eps is 0)
    q[~keep] = 1.0
    q = q.cuda()
    pos = torch.arange(6)
    w = (1 + 0.1 * torch.randn(D, generator=torch.Generator().manual_seed(2))).cuda()
    for weight in (None, w):
        got = r.norm_rotate(pos.cuda(), q, q_weight=weight, eps=eps)[0]
        check(got, q, pos.tolist(), r, dt, weight, ctypes.c_float(eps).value)


@pytest.mark.parametrize("size,eps", [(1e-36, 1e-32), (1e-37, 7e-31), (1e-30, 1e-38), (1e-38, 1e-45), (1e-36, 1e38)])
def test_an_eps_of_any_size_beside_the_rows(size, eps):
    import torch
    from host_streamed_paged_gb300 import kvs
    r = kvs.Rotary(128, rot_dim=64)
    x = torch.randn(5, 3, 128, generator=torch.Generator().manual_seed(4), dtype=torch.float64)
    q = (x / x.abs().max() * size).float().cuda()
    pos = torch.arange(5)
    check(r.norm_rotate(pos.cuda(), q, eps=eps)[0], q, pos.tolist(), r, "f32", None, ctypes.c_float(eps).value)


def test_values_that_are_not_finite_stay_with_their_head():
    import torch
    from host_streamed_paged_gb300 import kvs
    for interleaved in (False, True):
        r = kvs.Rotary(128, rot_dim=64, interleaved=interleaved)
        q, k = rows(9, 4, 2, 128, "f16")
        pos = torch.arange(9, device="cuda")
        want, wn = r.rotate(pos, q, k), r.norm_rotate(pos, q, k)
        y = q.clone()
        y[3, 1, 100], y[4, 2, 7], y[5, 0, 127] = math.inf, math.nan, -math.inf
        got, gn = r.rotate(pos, y, k), r.norm_rotate(pos, y, k)
        assert got[0][3, 1, 100] == math.inf and got[0][5, 0, 127] == -math.inf  # copied dims
        partner = 6 if interleaved else 39
        assert got[0][4, 2, 7].isnan() and got[0][4, 2, partner].isnan() and got[0][4, 2].isnan().sum() == 2
        rest = torch.ones(9, 4, dtype=torch.bool, device="cuda")
        rest[3, 1] = rest[4, 2] = rest[5, 0] = False
        assert torch.equal(got[0][rest], want[0][rest]) and torch.equal(gn[0][rest], wn[0][rest]) and gn[0][4, 2].isnan().all()
        assert torch.equal(got[1], want[1]) and torch.equal(gn[1], wn[1])


def test_rows_past_four_gigabytes():
    import torch
    from host_streamed_paged_gb300 import kvs
    r = kvs.Rotary(64)
    n, stride = 700, 4 << 20  # 5.9e9 bytes
    store = torch.empty(n * stride, dtype=torch.float16, device="cuda")
    x = store.as_strided((n, 6, 64), (stride, 64, 1))
    q, k = rows(n, 4, 2, 64, "f16")
    x[:, :4], x[:, 4:] = q, k
    pos = torch.arange(n, device="cuda")
    want = r.norm_rotate(pos, q, k)
    r.norm_rotate(pos, x[:, :4], x[:, 4:], out=(x[:, :4], x[:, 4:]))
    assert torch.equal(x[:, :4], want[0]) and torch.equal(x[:, 4:], want[1])


def test_captured_and_replayed_on_other_streams():
    import torch
    from host_streamed_paged_gb300 import kvs
    r = kvs.Rotary(128)
    q, k = (x.contiguous() for x in rows(64, 8, 2, 128, "bf16"))
    pos = torch.arange(64, device="cuda")
    outs = torch.empty_like(q), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = r.rotate(pos, q, k)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.rotate(pos, q, k, out=outs)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    pos += 1000
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], r.rotate(pos, q, k)[0]) and not torch.equal(outs[0], want[0])


@pytest.mark.parametrize("D,window,sinks", [(128, 0, 0), (128, 150, 4), (64, 33, 0), (256, 100, 2)])
def test_a_layers_step(D, window, sinks):
    """Two sequences come in chunks, then decode: norm and rotation, append, chunk attention, decode attention, each step
    against the formulas over what the cache holds."""
    import torch
    import window_ref
    from host_streamed_paged_gb300 import kvs
    from test_gpu_chunk import check as check_chunk
    Hq, Hk, P, dt = 8, 2, 64, "bf16"
    r = kvs.Rotary(D, base=10000.0)
    cache = kvs.Q4Cache(page_tokens=P, n_kv_head=Hk, head_dim=D, n_pages=20)
    table = torch.randperm(20, generator=torch.Generator().manual_seed(1))[:16].int().view(2, 8).cuda()
    g = torch.Generator().manual_seed(D)
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g)).cuda(), (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    lens = [0, 0]

    class Held:  # what check() asks of a filled cache: lengths, and the values that are held
        @staticmethod
        def seq(i):
            t = torch.arange(lens[i])
            slots = table[i].long().cpu()[t // P] * P + t % P
            k, v = cache.read(slots.cuda())
            return [x.double().cpu().numpy() for x in (k, v, v)]

    for rows_ in ([130, 37], [1, 200], [90, 1], [1, 1]):
        n = sum(rows_)
        qkv = torch.randn(n, Hq + 2 * Hk, D, generator=g).to(_t(dt)).cuda()
        pos = torch.cat([lens[i] + torch.arange(rows_[i]) for i in range(2)])
        slots = torch.cat([table[i].long().cpu()[(lens[i] + torch.arange(rows_[i])) // P] * P + (lens[i] + torch.arange(rows_[i])) % P for i in range(2)])
        q, k = r.norm_rotate(pos.cuda(), qkv[:, :Hq], qkv[:, Hq:Hq + Hk], wq, wk)
        check(q, qkv[:, :Hq], pos.tolist(), r, dt, wq, 1e-6)
        cache.append(slots.cuda(), k, qkv[:, Hq + Hk:])
        lens = [lens[i] + rows_[i] for i in range(2)]
        lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
        cu = torch.tensor([0, rows_[0], n], dtype=torch.int32).cuda()
        lse = torch.empty(n, Hq, device="cuda")
        out = cache.attend_chunk(table, lens_t, cu, q, lse=lse, window=window, sinks=sinks)
        Held.lens = lens
        check_chunk(out, lse, q, cu, Held, dt, D ** -0.5, window, sinks)
        if rows_ == [1, 1]:  # a decode step through the other call: the same attention but for K's rounding
            step, z = cache.attend(table, lens_t, q.view(2, 1, Hq, D), window=window, sinks=sinks)
            for i in range(2):
                k64, v64, _ = Held.seq(i)
                most = window_ref.rows(q[i:i + 1].double().cpu().numpy(), k64, v64, [lens[i] - 1], D ** -0.5, window, sinks)[3]
                assert (np.abs((z[i, 0] - lse[i]).cpu().numpy()) <= (2.0 ** -11 + 2.0 ** -18) * most[0] + 2e-5).all()
            assert (step.view(2, Hq, D) - out).float().norm() <= 2.0 ** -6 * out.float().norm()
