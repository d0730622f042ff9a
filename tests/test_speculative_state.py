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


def test_layers_follow_replaced_tensors():
    lens, table = i32(3), i32(3, 4)
    caches = [kv(lens, table) for _ in range(3)]
    layers = tsd.LayerCaches(caches)
    at = lambda: [(x.k, x.v) for x in layers.c_layers]
    where = lambda: [(c.k.data_ptr(), c.v.data_ptr()) for c in caches]
    assert at() == where()
    caches[1].v = torch.zeros_like(caches[1].v)
    assert at() == where()
    for c in caches:                                   # a pool that has grown
        c.k, c.v = (torch.zeros(9, 1, 4, 128, dtype=torch.bfloat16) for _ in range(2))
    assert at() == where()
    caches[2].k = torch.zeros(7, 1, 4, 128, dtype=torch.bfloat16)
    caches[2].v = torch.zeros_like(caches[2].k)        # one layer smaller than the others
    with pytest.raises(ValueError, match="share"):
        layers.c_layers
    caches[2].k = torch.zeros(9, 1, 4, 128, dtype=torch.bfloat16)
    caches[2].v = torch.zeros(9, 1, 4, 256, dtype=torch.bfloat16)[..., ::2]
    with pytest.raises(ValueError, match="contiguous"):
        layers.c_layers
    caches[2].v = torch.zeros(9, 1, 4, 128)
    with pytest.raises(ValueError, match="bfloat16"):
        layers.c_layers
