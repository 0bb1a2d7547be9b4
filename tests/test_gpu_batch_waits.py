"""Waits of the batch operators that give up (made to by kvs_debug_inject, at once and with every copy under way): what
they owed is NaN, the copies are waited for, and the next call is right."""
import math

import pytest

from host_streamed_paged_gb300 import kvs
from test_gpu_q4 import DT, Filled, _t

pytestmark = pytest.mark.gpu
LENS = [0, 1, 33, 700, 64, 3000]


@pytest.fixture(autouse=True)
def disarm():
    yield
    kvs.kvs_debug_inject(None, kvs.KVS_FAULT_NONE, 0)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("D,Hk,G,R", [(64, 2, 4, 1), (128, 2, 4, 1), (128, 1, 8, 5), (256, 1, 6, 2)])
def test_cache_waits(D, Hk, G, R, dt):
    import torch
    f = Filled(LENS, Hk, D, 64, seed=D + R, dt=dt)
    q = torch.randn(len(LENS), R, Hk * G, D, generator=torch.Generator().manual_seed(5)).to(_t(dt)).cuda()
    want, lse = f.cache.attend(f.table_t, f.lens_t, q)
    prev = torch.rand(len(LENS), Hk, 3100, device="cuda")
    want_w = f.cache.weights(f.table_t, f.lens_t, q, lse, prev=prev)
    for _ in range(3):
        kvs.kvs_debug_inject(None, kvs.KVS_FAULT_DEVICE_WAIT, 1)
        out, z = f.cache.attend(f.table_t, f.lens_t, q)
        assert out[1:].isnan().all() and z[1:].isnan().all()
        assert not out[0].any() and (z[0] == -math.inf).all()
        kvs.kvs_debug_inject(None, kvs.KVS_FAULT_DEVICE_WAIT, 2)
        again, z = f.cache.attend(f.table_t, f.lens_t, q)
        assert torch.equal(again, want) and torch.equal(z, lse)
        w = f.cache.weights(f.table_t, f.lens_t, q, lse, prev=prev)
        for i, n in enumerate(LENS):
            assert w[i, :, :n].isnan().all() and torch.equal(w[i, :, n:], prev[i, :, n:])
        assert torch.equal(f.cache.weights(f.table_t, f.lens_t, q, lse, prev=prev), want_w)
    assert torch.equal(f.cache.attend(f.table_t, f.lens_t, q)[0], want)


def test_only_waits_can_be_armed_without_a_context():
    with pytest.raises(kvs.KVSError) as e:
        kvs.kvs_debug_inject(None, kvs.KVS_FAULT_SYNC_STALL, 1)
    assert e.value.status == kvs.KVS_ERR_INVALID


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D,Hk,G", [(64, 2, 4), (128, 2, 1), (256, 1, 6)])
def test_prompt_waits(D, Hk, G, dt):
    import torch
    lens = [1, 37, 2000, 0, 300]
    rows = sum(lens) + 4
    x = torch.randn(rows, Hk * G + 2 * Hk, D, generator=torch.Generator().manual_seed(D)).to(_t(dt)).cuda()
    q, k, v = x[:, :Hk * G], x[:, Hk * G:Hk * G + Hk], x[:, Hk * G + Hk:]
    cu = torch.tensor([0, 1, 38, 2038, 2038, 2338], dtype=torch.int32, device="cuda")
    out, lse = torch.full((rows, Hk * G, D), 7.0, dtype=_t(dt), device="cuda"), torch.full((rows, Hk * G), 7.0, device="cuda")
    prev = torch.rand(len(lens), Hk, 2100, device="cuda")

    def attend():
        return kvs.prompt_attend(q, k, v, cu, out=out.clone(), lse=lse.clone())

    def weights(window):
        return kvs.prompt_weights(q, k, want[1], cu, 2100, window=window, prev=prev)

    want = attend()
    want_w = weights(0), weights(64)
    for _ in range(3):
        kvs.kvs_debug_inject(None, kvs.KVS_FAULT_DEVICE_WAIT, 1)
        o, z = attend()
        assert o[:2338].isnan().all() and z[:2338].isnan().all() and (o[2338:] == 7).all() and (z[2338:] == 7).all()
        o, z = attend()
        assert torch.equal(o, want[0]) and torch.equal(z, want[1])
        for w, window in zip(want_w, (0, 64)):
            kvs.kvs_debug_inject(None, kvs.KVS_FAULT_DEVICE_WAIT, 1)
            got = weights(window)
            for i, n in enumerate(lens):
                assert got[i, :, :n].isnan().all() and torch.equal(got[i, :, n:], prev[i, :, n:])
            assert torch.equal(weights(window), w)
