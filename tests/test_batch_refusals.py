"""Argument checks of the batch operators (kvs_prompt_*, kvs_q4_*): no GPU work is reached."""
import ctypes

import pytest

from host_streamed_paged_gb300 import kvs

FAKE = 1 << 20  # aligned, never dereferenced


def prompt(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_stride=1024, k_stride=256, v_stride=256, cu=FAKE, n_seq=2, total_rows=100, n_q_head=8,
             n_kv_head=2, head_dim=128, dtype=kvs.KVS_F16, scale=0.1)
    a.update(kw)
    return kvs.kvs_prompt(*[a[n] for n, _ in kvs.kvs_prompt._fields_])


def pool(**kw):
    a = dict(pages=FAKE, n_pages=10, page_tokens=64, n_kv_head=2, head_dim=128)
    a.update(kw)
    return kvs.kvs_q4_pool(*[a[n] for n, _ in kvs.kvs_q4_pool._fields_])


def status(f, *a, **kw):
    with pytest.raises(kvs.KVSError) as e:
        f(*a, **kw)
    assert kvs.kvs_last_error(None)
    return e.value.status


PROMPT_BAD = [
    (dict(head_dim=96), kvs.KVS_ERR_UNSUPPORTED), (dict(dtype=kvs.KVS_F32), kvs.KVS_ERR_UNSUPPORTED), (dict(dtype=9), kvs.KVS_ERR_INVALID),
    (dict(n_q_head=7), kvs.KVS_ERR_INVALID), (dict(n_kv_head=0), kvs.KVS_ERR_INVALID), (dict(n_q_head=0), kvs.KVS_ERR_INVALID),
    (dict(n_q_head=130, n_kv_head=2, q_stride=130 * 128), kvs.KVS_ERR_UNSUPPORTED), (dict(n_seq=5000), kvs.KVS_ERR_UNSUPPORTED),
    (dict(total_rows=0x7fffffff), kvs.KVS_ERR_INVALID), (dict(scale=0.0), kvs.KVS_ERR_INVALID), (dict(scale=-1.0), kvs.KVS_ERR_INVALID),
    (dict(scale=float("nan")), kvs.KVS_ERR_INVALID), (dict(scale=float("inf")), kvs.KVS_ERR_INVALID), (dict(cu=0), kvs.KVS_ERR_INVALID),
    (dict(q=0), kvs.KVS_ERR_INVALID), (dict(k=FAKE + 8), kvs.KVS_ERR_INVALID), (dict(q_stride=1028), kvs.KVS_ERR_INVALID),
    (dict(k_stride=128), kvs.KVS_ERR_INVALID), (dict(q_stride=1 << 39), kvs.KVS_ERR_INVALID),
]


@pytest.mark.parametrize("kw,want", PROMPT_BAD)
def test_prompt_calls_refuse(kw, want):
    assert status(kvs.kvs_prompt_attend, prompt(**kw), FAKE, 1024, FAKE) == want
    assert status(kvs.kvs_prompt_weights, prompt(**kw), FAKE, 0, None, FAKE, 100) == want


def test_prompt_attend_refuses_its_outputs():
    assert status(kvs.kvs_prompt_attend, prompt(), 0, 1024, FAKE) == kvs.KVS_ERR_INVALID
    assert status(kvs.kvs_prompt_attend, prompt(), FAKE + 2, 1024, FAKE) == kvs.KVS_ERR_INVALID
    assert status(kvs.kvs_prompt_attend, prompt(), FAKE, 512, FAKE) == kvs.KVS_ERR_INVALID
    assert status(kvs.kvs_prompt_attend, prompt(v=0), FAKE, 1024, FAKE) == kvs.KVS_ERR_INVALID
    assert status(kvs.kvs_prompt_weights, prompt(), None, 0, None, FAKE, 100) == kvs.KVS_ERR_INVALID
    assert status(kvs.kvs_prompt_weights, prompt(), FAKE, 0, None, None, 100) == kvs.KVS_ERR_INVALID
    assert status(kvs.kvs_prompt_weights, prompt(), FAKE, 0, None, FAKE, 1 << 31) == kvs.KVS_ERR_INVALID
    with pytest.raises(kvs.KVSError):
        kvs._check(None, kvs.load().kvs_prompt_attend(None, FAKE, 1024, FAKE, None))


def test_empty_prompt_calls_do_nothing():
    assert kvs.kvs_prompt_attend(prompt(n_seq=0), FAKE, 1024, FAKE) == kvs.KVS_OK
    assert kvs.kvs_prompt_attend(prompt(total_rows=0, q=0, k=0, v=0), 0, 0, 0) == kvs.KVS_OK
    assert kvs.kvs_prompt_weights(prompt(n_seq=0), FAKE, 0, None, FAKE, 100) == kvs.KVS_OK


POOL_BAD = [
    (dict(page_tokens=48), kvs.KVS_ERR_UNSUPPORTED), (dict(page_tokens=512), kvs.KVS_ERR_UNSUPPORTED), (dict(head_dim=32), kvs.KVS_ERR_UNSUPPORTED),
    (dict(n_kv_head=0), kvs.KVS_ERR_INVALID), (dict(pages=0), kvs.KVS_ERR_INVALID), (dict(pages=FAKE + 8), kvs.KVS_ERR_INVALID),
    (dict(n_pages=0), kvs.KVS_ERR_INVALID), (dict(n_pages=1 << 31), kvs.KVS_ERR_INVALID),
]


def attend(p, **kw):
    a = dict(table=FAKE, table_width=4, lens=FAKE, n_seq=3, n_rows=1, n_q_head=8, q=FAKE, dtype=kvs.KVS_F32, q_stride=1024, scale=0.1,
             out=FAKE, lse=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(kw)
    return kvs.kvs_q4_attend(p, *a.values())


def weights(p, **kw):
    a = dict(table=FAKE, table_width=4, lens=FAKE, n_seq=3, n_rows=1, n_q_head=8, q=FAKE, dtype=kvs.KVS_F32, q_stride=1024, scale=0.1,
             lse=FAKE, prev=None, weights=FAKE, width=256)
    a.update(kw)
    return kvs.kvs_q4_weights(p, *a.values())


def evict(p, **kw):
    a = dict(table=FAKE, table_width=4, dst_table=FAKE, dst_width=2, lens=FAKE, n_seq=3, weights=FAKE, width=256, keep=100, sinks=4,
             recent=20, kept=FAKE, kept_weights=2 * FAKE, new_lens=2 * FAKE)
    a.update(kw)
    return kvs.kvs_q4_evict(p, *a.values())


@pytest.mark.parametrize("kw,want", POOL_BAD)
def test_cache_calls_refuse_a_bad_pool(kw, want):
    p = pool(**kw)
    assert status(attend, p) == want and status(weights, p) == want and status(evict, p) == want
    assert status(kvs.kvs_q4_append, p, FAKE, 3, FAKE, FAKE, kvs.KVS_F32, 256, 256) == want
    assert status(kvs.kvs_q4_read, p, FAKE, 3, FAKE, FAKE, kvs.KVS_F32) == want


ROWS_BAD = [
    (dict(table=0), kvs.KVS_ERR_INVALID), (dict(table_width=0), kvs.KVS_ERR_INVALID), (dict(table_width=1 << 26), kvs.KVS_ERR_INVALID),
    (dict(lens=0), kvs.KVS_ERR_INVALID), (dict(n_seq=4097), kvs.KVS_ERR_UNSUPPORTED), (dict(n_rows=0), kvs.KVS_ERR_INVALID),
    (dict(n_rows=17), kvs.KVS_ERR_UNSUPPORTED), (dict(n_q_head=9), kvs.KVS_ERR_INVALID), (dict(n_q_head=0), kvs.KVS_ERR_INVALID),
    (dict(q=0), kvs.KVS_ERR_INVALID), (dict(q=FAKE + 4), kvs.KVS_ERR_INVALID), (dict(dtype=3), kvs.KVS_ERR_INVALID),
    (dict(q_stride=1000), kvs.KVS_ERR_INVALID), (dict(q_stride=1026), kvs.KVS_ERR_INVALID), (dict(scale=float("inf")), kvs.KVS_ERR_INVALID),
    (dict(lse=0), None), (dict(n_rows=(1 << 32) - 1), kvs.KVS_ERR_UNSUPPORTED),
    (dict(n_seq=4096, table_width=1 << 20), kvs.KVS_ERR_UNSUPPORTED),  # 2^34 tiles: their line counts in 31 bits
]


@pytest.mark.parametrize("kw,want", ROWS_BAD)
def test_attend_and_weights_refuse(kw, want):
    if want is not None:
        assert status(attend, pool(), **kw) == want
    assert status(weights, pool(), **kw) == (want or kvs.KVS_ERR_INVALID)


def test_attend_refuses_its_outputs_and_workspace():
    p = pool()
    need = kvs.kvs_q4_query_sizes(p, 1, 8, kvs.KVS_F32)[1]
    assert status(attend, p, out=0) == kvs.KVS_ERR_INVALID
    assert status(attend, p, workspace=0) == kvs.KVS_ERR_INVALID
    assert status(attend, p, workspace=FAKE + 16) == kvs.KVS_ERR_INVALID
    assert status(attend, p, workspace_bytes=need - 1) == kvs.KVS_ERR_CAPACITY
    assert status(weights, p, weights=0) == kvs.KVS_ERR_INVALID
    assert status(weights, p, width=1 << 31) == kvs.KVS_ERR_INVALID
    assert attend(p, n_seq=0) == kvs.KVS_OK and weights(p, n_seq=0) == kvs.KVS_OK and weights(p, width=0) == kvs.KVS_OK


def test_append_and_read_refuse():
    p = pool()
    for a in ((0, 3, FAKE, FAKE, kvs.KVS_F32, 256, 256), (FAKE + 4, 3, FAKE, FAKE, kvs.KVS_F32, 256, 256), (FAKE, 3, 0, FAKE, kvs.KVS_F32, 256, 256),
              (FAKE, 3, FAKE, FAKE + 4, kvs.KVS_F32, 256, 256), (FAKE, 3, FAKE, FAKE, 5, 256, 256), (FAKE, 3, FAKE, FAKE, kvs.KVS_F32, 255, 256),
              (FAKE, 3, FAKE, FAKE, kvs.KVS_F16, 260, 256), (FAKE, 1 << 62, FAKE, FAKE, kvs.KVS_F16, 256, 256)):
        assert status(kvs.kvs_q4_append, p, *a) == kvs.KVS_ERR_INVALID
    assert status(kvs.kvs_q4_read, p, FAKE, 3, FAKE + 2, FAKE, kvs.KVS_F32) == kvs.KVS_ERR_INVALID
    assert status(kvs.kvs_q4_read, p, FAKE, 3, FAKE, FAKE, 7) == kvs.KVS_ERR_INVALID
    assert kvs.kvs_q4_append(p, 0, 0, 0, 0, kvs.KVS_F32, 0, 0) == kvs.KVS_OK
    assert kvs.kvs_q4_read(p, FAKE, 5, None, None, kvs.KVS_F32) == kvs.KVS_OK


@pytest.mark.parametrize("kw,want", [
    (dict(table=0), kvs.KVS_ERR_INVALID), (dict(dst_table=0), kvs.KVS_ERR_INVALID), (dict(weights=0), kvs.KVS_ERR_INVALID),
    (dict(kept=0), kvs.KVS_ERR_INVALID), (dict(new_lens=0), kvs.KVS_ERR_INVALID), (dict(width=0), kvs.KVS_ERR_INVALID),
    (dict(keep=0), kvs.KVS_ERR_INVALID), (dict(sinks=90), kvs.KVS_ERR_INVALID), (dict(sinks=(1 << 32) - 1, recent=(1 << 32) - 1), kvs.KVS_ERR_INVALID),
    (dict(keep=129), kvs.KVS_ERR_CAPACITY), (dict(n_seq=4097), kvs.KVS_ERR_UNSUPPORTED), (dict(kept_weights=FAKE), kvs.KVS_ERR_INVALID),
    (dict(new_lens=FAKE), kvs.KVS_ERR_INVALID), (dict(table_width=0), kvs.KVS_ERR_INVALID)])
def test_evict_refuses(kw, want):
    assert status(evict, pool(), **kw) == want


def test_sizes():
    for D in (64, 128, 256):
        page, ws = kvs.kvs_q4_query_sizes(pool(pages=0, head_dim=D), 1, 8, kvs.KVS_F16)
        assert page == 2 * 64 * D * 9 // 8 and 0 < ws <= 1 << 26
    assert status(kvs.kvs_q4_query_sizes, pool(), 40, 8, kvs.KVS_F16) == kvs.KVS_ERR_UNSUPPORTED
    assert ctypes.sizeof(kvs.kvs_prompt) == 88 and ctypes.sizeof(kvs.kvs_q4_pool) == 32


def test_torch_entry_points_refuse_before_the_library():
    import torch
    q, k = torch.zeros(10, 4, 64, dtype=torch.float16), torch.zeros(10, 2, 64, dtype=torch.float16)
    cu = torch.tensor([0, 10], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kvs.prompt_attend(q, k, k, cu)
    with pytest.raises(ValueError):
        kvs.prompt_attend(q, k, k, cu.long())
    with pytest.raises(ValueError):
        kvs.prompt_attend(q, k[:5], k, cu)
    with pytest.raises(ValueError):
        kvs.prompt_attend(q, k.float(), k, cu)
    with pytest.raises(ValueError):
        kvs.prompt_attend(q.transpose(0, 1), k, k, cu)
    c = kvs.Q4Cache(page_tokens=32, n_kv_head=2, head_dim=64, n_pages=2, device="cpu")
    with pytest.raises(ValueError):
        c.append(torch.zeros(3, dtype=torch.int32), k[:3], k[:3])
    with pytest.raises(ValueError):
        c.append(torch.zeros(3, dtype=torch.int64), k, k)
    with pytest.raises(ValueError, match="CUDA"):
        c.append(torch.zeros(10, dtype=torch.int64), k, k)
    with pytest.raises(ValueError):
        kvs.Q4Cache(page_tokens=32, n_kv_head=2, head_dim=64, pages=torch.zeros(100, dtype=torch.uint8))
