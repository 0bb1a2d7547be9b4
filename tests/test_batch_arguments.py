"""Arguments of the batch operators that the host sees, beside those of test_batch_refusals: no GPU work is reached."""
import pytest

from host_streamed_paged_gb300 import kvs
from test_batch_refusals import evict, pool, status


def test_evict_refuses_too_many_tiles_before_any_launch():
    """2^26 tiles of each of 129 (sequence, head) pairs: more CTAs than a launch may have."""
    keep = 0x7fffffc0
    assert status(evict, pool(n_kv_head=1, page_tokens=32), n_seq=129, keep=keep, dst_width=1 << 26) == kvs.KVS_ERR_UNSUPPORTED
