"""Tables, lengths and layers that the speculative calls refuse, without a GPU."""

import pytest
import torch

import top_sparse_decode_topk_b200 as tsd
from top_sparse_decode_topk_b200 import speculative


def kv(lens, table, pages=5, max_len=16):
    mk = lambda: torch.zeros(pages, 1, 4, 128, dtype=torch.bfloat16)
    return tsd.KVCache(mk(), mk(), lens, max_len, page_table=table)


def i32(*shape, **kw):
    return torch.zeros(*shape, dtype=torch.int32, **kw)


def test_lengths_have_to_be_dense():
    state = i32(3, 2)
    for n in (1, 2):
        with pytest.raises(ValueError, match="seq_lens"):
            tsd.LayerCaches([kv(state[:, 0], i32(3, 4)) for _ in range(n)])
    with pytest.raises(ValueError, match="seq_lens"):
        tsd.LayerCaches(kv(state, i32(3, 4)))
    tsd.LayerCaches(kv(state.view(-1)[:3], i32(3, 4)))


def test_tables_have_to_be_dense_with_a_row_for_every_sequence():
    with pytest.raises(ValueError, match="page_table"):
        tsd.LayerCaches(kv(i32(3), i32(2, 4)))
    with pytest.raises(ValueError, match="page_table"):
        tsd.LayerCaches(kv(i32(3), i32(3, 4, device="meta")))
    with pytest.raises(ValueError, match="row for every"):
        c = tsd.KVCache(torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16), i32(3), 4)
        tsd.LayerCaches(c)
    tsd.LayerCaches(kv(i32(3), i32(5, 4)))          # spare rows are left alone
    c = kv(i32(3), i32(3, 4))
    c.page_table = i32(3, 8)[:, :4]
    with pytest.raises(ValueError, match="page_table"):
        tsd.LayerCaches(c)


def test_a_copied_table_is_not_written():
    wide, lens = i32(3, 8), i32(3)
    c = kv(lens, wide[:, :4])
    assert c.page_table.is_contiguous()
    with pytest.raises(ValueError, match="copy"):
        speculative._check_written(c)
    with pytest.raises(ValueError, match="copy"):   # not "must share their page table"
        tsd.LayerCaches([kv(lens, wide[:, :4]), kv(lens, wide[:, :4])])
    c.page_table = i32(3, 4)
    speculative._check_written(c)
    speculative._check_written(kv(lens, wide))
    tsd.LayerCaches([kv(lens, wide), kv(lens, wide)])
