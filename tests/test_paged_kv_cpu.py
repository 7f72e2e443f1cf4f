"""PagedKV's own bookkeeping, on the CPU (no kernel runs)."""
import pytest
import torch

from speculative_decoding_05_b200 import build
from speculative_decoding_05_b200.kv import PagedKV


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def make(**kw):
    return PagedKV(**dict(dict(B=3, Hq=4, Hkv=2, head_dim=64, max_pages=4, page_size=16,
                               device="cpu"), **kw))


def test_default_table_names_pages_that_exist():
    for n in (None, 12, 20):
        kv = make(n_pages=n)
        assert int(kv.page_table.max()) < kv.k_cache.shape[0] and kv.page_table.shape == (3, 4)
    for n in (0, 1, 11):
        with pytest.raises(ValueError, match="n_pages"):
            make(n_pages=n)


def test_status_is_clean_before_the_first_call(monkeypatch):
    """flags() of a cache that was only appended to must not read what its
    attention workspace's memory held before."""
    from speculative_decoding_05_b200 import dspark as D
    monkeypatch.setattr(D, "workspace",
                        lambda n, device: torch.full((n,), 0xFF, dtype=torch.uint8, device=device))
    kv = make()
    for ws in (kv.ws, kv.ws_attn):
        assert not bool(ws[:16].any())


def test_a_table_of_ones_own_may_share_fewer_pages():
    table = torch.zeros(3, 4, dtype=torch.int32)
    kv = make(n_pages=5, page_table=table)
    assert kv.page_table is table and kv.k_cache.shape[0] == 5


def test_advance_leaves_idle_slots():
    """What the verify returns for an idle slot (a request without drafts) does
    not move it; the accepted tokens and the emitted one move the others."""
    kv = make()
    kv.cache_len.copy_(torch.tensor([5, 0, 9], dtype=torch.int32))
    rows = (torch.zeros(3, dtype=torch.int64), torch.tensor([2, -1, 0], dtype=torch.int32))
    at = kv.cache_len
    for n in (0, 3, -1):
        kv.advance(torch.tensor([1, n, 0], dtype=torch.int32), rows)
    assert kv.cache_len is at and kv.cache_len.dtype == torch.int32
    assert kv.cache_len.tolist() == [11, 0, 12]
    kv.advance(torch.tensor([1, -1, 0], dtype=torch.int32))
    assert kv.cache_len.tolist() == [13, 0, 13]
