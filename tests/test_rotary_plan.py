"""Rotary's plan (frequencies, their scalings, fractions of a turn) and the refusals of the calls around it, on the CPU."""
import ctypes
import math
from fractions import Fraction

import pytest

from host_streamed_paged_gb300 import kvs
from test_batch_refusals import FAKE, pool, prompt, status

PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


def plan(*a, **kw):
    return kvs.Rotary(*a, device="cpu", **kw)


@pytest.mark.parametrize("D,rot", [(64, None), (128, 32), (128, 48), (256, 256)])
def test_frequencies_and_turns(D, rot):
    r = plan(D, rot_dim=rot, base=10000.0)
    n = rot or D
    assert len(r.freqs) == n // 2 and r.magnitude == 1.0 and r.freqs[0] == 1.0
    for i, (f, t) in enumerate(zip(r.freqs, r.turns.tolist())):
        assert math.isclose(f, math.exp(-2 * i / n * math.log(10000.0)), rel_tol=1e-14)
        # the fraction of a turn, to the rounding of the double f / 2 pi and the last of 64 bits
        exact = Fraction(f) / (2 * PI)
        assert abs(Fraction(t % 2 ** 64, 2 ** 64) - exact) <= exact * Fraction(1, 2 ** 51) + Fraction(1, 2 ** 64)


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
def test_turns_are_rounded_once(base):
    """Half of the last of 64 bits, whatever the frequency: it counts position times."""
    r = plan(256, base=base)
    odd = plan(64, freqs=[-f for f in r.freqs[:26]] + [1e30, -3.7e25, 5e-324, 2.0 ** -70, 0.0, 2 * math.pi])
    for p in (r, odd):
        for f, t in zip(p.freqs, p.turns.tolist()):
            off = Fraction(t, 2 ** 64) - Fraction(f) / (2 * PI)
            off -= math.floor(off + Fraction(1, 2))
            assert abs(off) <= Fraction(1, 2 ** 65) * Fraction(1000001, 1000000)


def test_frequencies_of_more_than_a_turn_and_below_zero():
    r = plan(64, freqs=[7.0, -0.25, 0.0, 1.0] * 2)
    assert r.rot_dim == 16
    t = [x % 2 ** 64 / 2 ** 64 for x in r.turns.tolist()]
    assert math.isclose(t[0], 7 / (2 * math.pi) - 1, rel_tol=1e-12) and math.isclose(t[1], 1 - 0.25 / (2 * math.pi)) and t[2] == 0


def test_scalings():
    n, base, factor, context = 64, 500000.0, 8.0, 4096
    f = plan(64, base=base).freqs
    assert plan(64, base=base, scaling="linear", factor=factor).freqs == [x / 8 for x in f]
    ntk = plan(64, base=base, scaling="ntk", factor=factor).freqs
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], f[-1] / factor, rel_tol=1e-12)
    for scaling, fast, slow in (("yarn", 32, 1), ("bands", 4, 1)):
        r = plan(64, base=base, scaling=scaling, factor=factor, context=context)
        turns = [context * x / (2 * math.pi) for x in f]
        for x, y, t in zip(f, r.freqs, turns):
            assert x / factor <= y * (1 + 1e-12) and y <= x * (1 + 1e-12)
            if t > 2 * fast:
                assert math.isclose(y, x)
            if t < slow / 2:
                assert math.isclose(y, x / factor)
        assert any(x / factor * 1.01 < y < x * 0.99 for x, y in zip(f, r.freqs))
    assert math.isclose(plan(64, scaling="yarn", factor=16, context=4096).magnitude, 0.1 * math.log(16) + 1)
    assert plan(64, scaling="yarn", factor=16, context=4096, magnitude=2.0).magnitude == 2.0
    # at factor 1, x r + x (1 - r): 1 - r, two products and a sum rounded, 4 2^-53 in all
    assert all(math.isclose(x, y, rel_tol=4 * 2.0 ** -53) for x, y in zip(plan(64, scaling="yarn", factor=1.0, context=4096).freqs, plan(64).freqs))


@pytest.mark.parametrize("kw", [dict(head_dim=96), dict(rot_dim=24), dict(rot_dim=80), dict(rot_dim=-16), dict(scaling="other"), dict(scaling="yarn"),
                                dict(scaling="bands", context=0), dict(scaling="bands", context=100, fast=1, slow=2), dict(base=0.0),
                                dict(factor=0.0), dict(freqs=[1.0] * 8, scaling="ntk"), dict(freqs=[1.0] * 7), dict(freqs=[math.nan] * 8),
                                dict(magnitude=math.inf), dict(freqs=[1.0] * 8, rot_dim=32), dict(scaling="yarn", base=1.0, context=9)])
def test_plans_that_are_refused(kw):
    with pytest.raises(ValueError):
        plan(**{**dict(head_dim=64), **kw})


def test_rows_that_are_refused(monkeypatch):
    import torch
    r = plan(64)
    q, k, pos = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64), torch.zeros(5, dtype=torch.int64)
    seen = []
    monkeypatch.setattr(kvs, "_run", lambda dev, fn, *a: seen.append(a))
    for a, kw in [((pos.float(), q), {}), ((pos[:4], q), {}), ((pos, q[..., :32]), {}), ((pos, q, k.half()), {}), ((pos, q, k[:4]), {}),
                  ((torch.zeros(5, 2, dtype=torch.int64)[:, 0], q), {}), ((pos, q.double()), {}), ((pos, q, None), dict(out=(q, q))),
                  ((pos, q, k), dict(out=(q, None))), ((pos, q, k), dict(out=(q, q))), ((pos, q.transpose(0, 1)), {}),
                  ((pos, q), dict(out=q)), ((torch.zeros(1, 1, 5, dtype=torch.int64), q), {})]:
        with pytest.raises(ValueError):
            r.rotate(*a, **kw)
    w = torch.ones(64)
    for qw, kw in ((w[:32], None), (w, w.half()), (torch.ones(128)[::2], None), (w.double(), w.double())):
        with pytest.raises(ValueError):
            r.norm_rotate(pos, q, k, qw, kw)
    assert not seen
    out = r.rotate(pos, q, k)
    assert out[0].shape == q.shape and out[1].shape == k.shape and seen[0][1:4] == (pos.data_ptr(), 8, 5)
    assert r.rotate(pos.int().view(5), q)[1] is None and seen[1][2] == 4
    same = r.norm_rotate(pos.view(5, 1), q.view(5, 1, 4, 64), k.view(5, 1, 2, 64), w, w, out=(q.view(5, 1, 4, 64), k.view(5, 1, 2, 64)))
    assert same[0].data_ptr() == q.data_ptr() and seen[2][3] == 5


def rotary(**kw):
    a = dict(turns=FAKE, head_dim=128, rot_dim=128, interleaved=0, magnitude=1.0)
    a.update(kw)
    return kvs.kvs_rotary(*a.values())


def heads(**kw):
    a = dict(x=FAKE, y=FAKE, x_stride=1024, y_stride=1024, n_head=8, weight=None)
    a.update(kw)
    return kvs.kvs_head_rows(*a.values())


ROTARY_BAD = [(dict(head_dim=96), kvs.KVS_ERR_UNSUPPORTED), (dict(rot_dim=136), kvs.KVS_ERR_UNSUPPORTED), (dict(rot_dim=24), kvs.KVS_ERR_UNSUPPORTED),
              (dict(turns=0), kvs.KVS_ERR_INVALID), (dict(turns=FAKE + 4), kvs.KVS_ERR_INVALID), (dict(magnitude=math.nan), kvs.KVS_ERR_INVALID)]
HEADS_BAD = [dict(x=0), dict(y=0), dict(x=FAKE + 8), dict(y=FAKE + 2), dict(x_stride=1020), dict(x_stride=1028), dict(y_stride=512), dict(n_head=0),
             dict(n_head=65536, x_stride=1 << 24, y_stride=1 << 24), dict(x_stride=(1 << 31) + 8)]


def both(want, r, pos=FAKE, size=8, n=3, dtype=kvs.KVS_F16, q=None, k=None):
    q, k = q or heads(), k or heads()
    assert status(kvs.kvs_rotate, r, pos, size, n, dtype, q, k) == want
    assert status(kvs.kvs_norm_rotate, r, pos, size, n, dtype, q, k, kvs.KVS_F32, 1e-6) == want


def test_the_library_refuses():
    bad = kvs.KVS_ERR_INVALID
    for kw, want in ROTARY_BAD:
        both(want, rotary(**kw))
    for kw in HEADS_BAD:
        both(bad, rotary(), q=heads(**kw))
        both(bad, rotary(), k=heads(**kw))
    both(bad, None)
    both(bad, rotary(), pos=0)
    both(bad, rotary(), pos=FAKE + 4)
    both(bad, rotary(), size=2)
    both(bad, rotary(), dtype=5)
    both(bad, rotary(), n=1 << 31)
    assert status(kvs.kvs_rotate, rotary(), FAKE, 8, 3, kvs.KVS_F16, None, heads()) == bad
    for w, eps in ((7, 1e-6), (0, -1.0), (0, math.nan), (0, math.inf)):
        assert status(kvs.kvs_norm_rotate, rotary(), FAKE, 8, 3, kvs.KVS_F16, heads(), None, w, eps) == bad
    assert status(kvs.kvs_norm_rotate, rotary(), FAKE, 8, 3, kvs.KVS_F16, heads(weight=FAKE + 4), None, 0, 1e-6) == bad
    assert kvs.kvs_rotate(rotary(), 0, 8, 0, kvs.KVS_F16, heads(x=0, y=0), None) == kvs.KVS_OK
    assert ctypes.sizeof(kvs.kvs_rotary) == 24 and ctypes.sizeof(kvs.kvs_head_rows) == 48


def chunk(p, **kw):
    a = dict(table=FAKE, table_width=4, lens=FAKE, cu=FAKE, n_seq=3, total_rows=100, n_q_head=8, q=FAKE, dtype=kvs.KVS_F16, q_stride=1024, scale=0.1,
             window=0, sinks=0, out=FAKE, out_stride=1024, lse=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(kw)
    return kvs.kvs_q4_attend_chunk(p, *a.values())


CHUNK_BAD = [
    (dict(table=0), kvs.KVS_ERR_INVALID), (dict(table_width=0), kvs.KVS_ERR_INVALID), (dict(table_width=1 << 26), kvs.KVS_ERR_INVALID),
    (dict(lens=0), kvs.KVS_ERR_INVALID), (dict(cu=0), kvs.KVS_ERR_INVALID), (dict(n_seq=4097), kvs.KVS_ERR_UNSUPPORTED),
    (dict(n_q_head=9), kvs.KVS_ERR_INVALID), (dict(n_q_head=0), kvs.KVS_ERR_INVALID), (dict(n_q_head=130, q_stride=1 << 15), kvs.KVS_ERR_UNSUPPORTED),
    (dict(q=0), kvs.KVS_ERR_INVALID), (dict(out=0), kvs.KVS_ERR_INVALID), (dict(q=FAKE + 8), kvs.KVS_ERR_INVALID), (dict(out=FAKE + 2), kvs.KVS_ERR_INVALID),
    (dict(dtype=kvs.KVS_F32), kvs.KVS_ERR_UNSUPPORTED), (dict(dtype=4), kvs.KVS_ERR_INVALID), (dict(q_stride=1020), kvs.KVS_ERR_INVALID),
    (dict(out_stride=1028), kvs.KVS_ERR_INVALID), (dict(q_stride=1 << 32), kvs.KVS_ERR_INVALID), (dict(scale=math.inf), kvs.KVS_ERR_INVALID),
    (dict(total_rows=0x7fffffff), kvs.KVS_ERR_INVALID), (dict(window=1 << 31), kvs.KVS_ERR_INVALID), (dict(sinks=0x7fffffff), kvs.KVS_ERR_INVALID),
    (dict(workspace=0), kvs.KVS_ERR_INVALID), (dict(workspace=FAKE + 16), kvs.KVS_ERR_INVALID), (dict(workspace_bytes=1000), kvs.KVS_ERR_CAPACITY),
]


@pytest.mark.parametrize("kw,want", CHUNK_BAD)
def test_chunks_refuse(kw, want):
    assert status(chunk, pool(), **kw) == want


def test_chunks_refuse_a_bad_pool_and_take_empty_batches():
    for kw in (dict(page_tokens=48), dict(head_dim=32)):
        assert status(chunk, pool(**kw)) == kvs.KVS_ERR_UNSUPPORTED
    for kw in (dict(n_kv_head=0), dict(pages=0), dict(n_pages=0)):
        assert status(chunk, pool(**kw)) == kvs.KVS_ERR_INVALID
    assert chunk(pool(), n_seq=0, table=0, lens=0, cu=0) == kvs.KVS_OK
    assert chunk(pool(), total_rows=0, q=0, out=0, workspace=0) == kvs.KVS_OK
    for D in (64, 128, 256):
        ws = kvs.kvs_q4_chunk_workspace(pool(pages=0, head_dim=D))
        assert ws % 256 == 0 and status(chunk, pool(head_dim=D), q_stride=2048, out_stride=2048, workspace_bytes=ws - 1) == kvs.KVS_ERR_CAPACITY
    assert status(kvs.kvs_q4_chunk_workspace, pool(head_dim=96)) == kvs.KVS_ERR_UNSUPPORTED


def windowed(p, **kw):
    a = dict(table=FAKE, table_width=4, lens=FAKE, n_seq=3, n_rows=1, n_q_head=8, q=FAKE, dtype=kvs.KVS_F32, q_stride=1024, scale=0.1, window=64,
             sinks=4, out=FAKE, lse=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(kw)
    return kvs.kvs_q4_attend_window(p, *a.values())


def test_windows_refuse():
    bad = kvs.KVS_ERR_INVALID
    for kw in (dict(window=1 << 31), dict(sinks=0x7fffffff), dict(table=0), dict(q=FAKE + 4), dict(out=0), dict(scale=math.nan), dict(workspace=0)):
        assert status(windowed, pool(), **kw) == bad
    assert status(windowed, pool(), workspace_bytes=64) == kvs.KVS_ERR_CAPACITY
    assert status(windowed, pool(), n_rows=17) == kvs.KVS_ERR_UNSUPPORTED
    assert windowed(pool(), n_seq=0) == kvs.KVS_OK
    for kw in (dict(window=1 << 31), dict(sinks=0x7fffffff)):
        a = {**dict(window=5, sinks=0), **kw}
        assert status(kvs.kvs_prompt_attend_window, prompt(), a["window"], a["sinks"], FAKE, 1024, FAKE) == bad
    assert status(kvs.kvs_prompt_attend_window, prompt(q=0), 5, 0, FAKE, 1024, FAKE) == bad
    assert status(kvs.kvs_prompt_attend_window, prompt(), 5, 0, FAKE + 2, 1024, FAKE) == bad
    with pytest.raises(kvs.KVSError):
        kvs._check(None, kvs.load().kvs_prompt_attend_window(None, 5, 0, FAKE, 1024, FAKE, None))


@pytest.mark.parametrize("kw", [dict(window=-1), dict(sinks=-1), dict(window=5, sinks=-(1 << 32) + 3)])
def test_negative_windows_are_refused(kw):
    import torch
    c = kvs.Q4Cache(page_tokens=32, n_kv_head=2, head_dim=64, n_pages=2, device="cpu")
    c._workspace = lambda need: torch.empty(need, dtype=torch.uint8)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q, cu = torch.zeros(10, 4, 64).half(), torch.tensor([0, 10], dtype=torch.int32)
    with pytest.raises(ValueError, match="negative"):
        c.attend(table, lens, q[None, :1], **kw)
    with pytest.raises(ValueError, match="negative"):
        c.attend_chunk(table, lens, cu, q, **kw)
    with pytest.raises(ValueError, match="negative"):
        kvs.prompt_attend(q, q[:, :2], q[:, :2], cu, **kw)


def test_chunk_arguments_that_are_refused():
    import torch
    c = kvs.Q4Cache(page_tokens=32, n_kv_head=2, head_dim=64, n_pages=2, device="cpu")
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, cu = torch.zeros(10, 4, 64).half(), torch.tensor([0, 4, 10], dtype=torch.int32)
    good = dict(table=table, lens=lens, cu=cu, q=q)
    for kw in (dict(cu=cu.long()), dict(cu=cu[:0]), dict(cu=cu[:2]), dict(table=table[:1]), dict(table=table.long()), dict(lens=lens[:1]),
               dict(q=q[..., :32]), dict(q=q[None]), dict(out=q[:5]), dict(out=q.float()), dict(lse=torch.zeros(10, 3)), dict(lse=torch.zeros(10, 4).half())):
        with pytest.raises(ValueError):
            c.attend_chunk(**{**good, **kw})
    with pytest.raises(ValueError, match="CUDA"):
        c.attend_chunk(**good)


def test_empty_batches_with_the_strides_of_an_empty_array(monkeypatch):
    """numpy's arrays without elements have strides of 0."""
    import numpy as np
    import torch
    monkeypatch.setattr(kvs, "_run", lambda dev, fn, *a: None)
    q, k = (torch.from_numpy(np.random.default_rng(0).standard_normal((0, n, 64), np.float32)) for n in (4, 2))
    assert k.stride() == (0, 0, 0)
    pos = torch.zeros(0, dtype=torch.int64)
    assert plan(64).rotate(pos, q, k)[0].shape == q.shape and plan(64).norm_rotate(pos, q, k)[1].shape == k.shape
    c = kvs.Q4Cache(page_tokens=32, n_kv_head=2, head_dim=64, n_pages=2, device="cpu")
    c._workspace = lambda need: torch.empty(need, dtype=torch.uint8)
    c.append(pos, k, k)
    none = torch.zeros(0, dtype=torch.int32)
    assert c.attend_chunk(none.view(0, 1), none, torch.zeros(1, dtype=torch.int32), q.half()).shape == q.shape
    with pytest.raises(ValueError, match="contiguous"):
        c.append(pos.new_zeros(2), torch.zeros(2, 64, 2).mT, torch.zeros(2, 2, 64))
