"""Arguments of the batch operators that the host sees, beside those of test_batch_refusals: no GPU work is reached."""
import pytest

from host_streamed_paged_gb300 import kvs
from test_batch_refusals import evict, pool, status


def test_evict_refuses_too_many_tiles_before_any_launch():
    """2^26 tiles of each of 129 (sequence, head) pairs: more CTAs than a launch may have."""
    keep = 0x7fffffc0
    assert status(evict, pool(n_kv_head=1, page_tokens=32), n_seq=129, keep=keep, dst_width=1 << 26) == kvs.KVS_ERR_UNSUPPORTED


def _rows(*shape):
    import torch
    return torch.zeros(*shape, dtype=torch.float16)


@pytest.mark.parametrize("window", [-1, -(1 << 32) + 5])
def test_a_negative_window_is_refused(window):
    """(It would reach the library as its value modulo 2^32: every row, or five of them.)"""
    import torch
    q, k, cu = _rows(10, 4, 64), _rows(10, 2, 64), torch.tensor([0, 10], dtype=torch.int32)
    with pytest.raises(ValueError, match="window"):
        kvs.prompt_weights(q, k, torch.zeros(10, 4), cu, 10, window=window)


def test_a_window_beyond_31_bits_is_every_row(monkeypatch):
    import torch
    q, k, cu = _rows(10, 4, 64), _rows(10, 2, 64), torch.tensor([0, 10], dtype=torch.int32)
    seen = []
    monkeypatch.setattr(kvs, "_run", lambda dev, fn, *a: seen.append(a))
    for window in (7, (1 << 32) + 5):
        kvs.prompt_weights(q, k, torch.zeros(10, 4), cu, 10, window=window)
    assert [a[2] for a in seen] == [7, (1 << 31) - 1]


@pytest.mark.parametrize("kw", [dict(keep=-1), dict(sinks=-1), dict(recent=-1), dict(sinks=(1 << 32) + 2), dict(recent=1 << 32),
                                dict(keep=(1 << 32) + 8)])
def test_evict_counts_out_of_range_are_refused(kw):
    import torch
    c = kvs.Q4Cache(page_tokens=32, n_kv_head=2, head_dim=64, n_pages=2, device="cpu")
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match=next(iter(kw))):
        c.evict(table, table, lens, torch.zeros(1, 2, 32), **dict(dict(keep=16), **kw))


def test_one_row_has_no_stride():
    """A row alone may be cut from rows that lie any number of elements apart."""
    import torch
    wide = torch.zeros(3, 4 * 64 + 3, dtype=torch.float16)
    one = wide[:, :256].unflatten(1, (4, 64))[:1]
    assert one.stride(0) == 259 and kvs._row_stride(one, "x") == 256
    assert kvs._row_stride(one[None], "x") == 256 and kvs._row_stride(one[:, None], "x") == 256
    assert kvs._row_stride(wide[:, :256].unflatten(1, (4, 64)), "x") == 259  # which the library then refuses
    assert kvs._row_stride(torch.zeros(5, 2, 4, 64)[:1], "x") == 256 and kvs._row_stride(torch.zeros(5, 2, 4, 64)[:, :1], "x") == 512
    assert kvs._row_stride(torch.zeros(0, 4, 64), "x") == 256 and kvs._row_stride(torch.zeros(0, 3, 4, 64), "x") == 256


def test_a_capture_is_looked_for_on_the_caches_device(monkeypatch):
    """Whether a call is being captured is asked of the current stream of the device that it runs on."""
    import torch

    class Device:
        type, index = "cuda", 1

    class On:
        def __init__(self, d):
            self.d = d.index

        def __enter__(self):
            self.was, now[0] = now[0], self.d

        def __exit__(self, *a):
            now[0] = self.was

    now, capturing, made = [0], {0: False, 1: True}, []
    c = kvs.Q4Cache(page_tokens=32, n_kv_head=2, head_dim=64, n_pages=2, device="cpu")
    c.device = Device()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[now[0]])
    monkeypatch.setattr(kvs, "_stream_of", lambda index: 7)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: made.append(n) or empty(n, dtype=dtype))
    assert c._workspace(512) is not c._workspace(512) and made == [512, 512]  # captured: one each
    capturing.update({0: True, 1: False})
    assert c._workspace(512) is c._workspace(512) and made == [512, 512, 512]
    now[0] = 1
    assert c._workspace(512) is c._workspace(512) and made == [512, 512, 512]
