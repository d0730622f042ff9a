"""Tables, lengths and layers that the speculative calls refuse, without a GPU."""

import ctypes

import pytest
import torch

import top_sparse_decode_topk_b200 as tsd
from tests.test_abi import FAKE, fake_pointer_call, lib, make_cache, make_queries   # noqa: F401
from top_sparse_decode_topk_b200 import _LayerC, _RopeC, speculative


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
    tsd.LayerCaches(kv(i32(3, 1), i32(3, 4)))


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


@fake_pointer_call
def test_pages_wanted_fit_32_bits(lib):
    """The pages that all sequences may want together are summed in 32 bits: more are refused on the host."""
    def resize(**kw):
        c = make_cache(page_size=1, max_seq_len=100, **kw)
        ls = (_LayerC * 1)(_LayerC(FAKE, FAKE))
        return lib.tsd_cache_resize(ctypes.byref(c), 1, ls, FAKE, FAKE, FAKE, 64, None, None)   # 64 bytes are never enough
    small = tsd.TSD_ERR_WORKSPACE_TOO_SMALL
    assert resize(batch=60000, max_pages=35790) == small                      # 60000 x 35791 = 2^31 - 23648
    assert resize(batch=60000, max_pages=35791) == tsd.TSD_ERR_UNSUPPORTED
    assert resize(batch=1, max_pages=2 ** 31 - 2) == small
    assert resize(batch=1, max_pages=2 ** 31 - 1) == tsd.TSD_ERR_UNSUPPORTED
    assert resize(batch=2, max_pages=2 ** 30) == tsd.TSD_ERR_UNSUPPORTED


@fake_pointer_call
def test_outputs_that_overlap_inputs_are_refused(lib):
    """A row may be rotated onto itself; anything else would be read after it is written."""
    T, hq, hkv = 64, 32, 8
    c = make_cache()
    bytes_q, bytes_k = T * hq * 256, T * hkv * 256

    def append(out, q=FAKE + 0x1000000, q_stride=4096, k=FAKE + 0x2000000, v=FAKE + 0x3000000, tokens=T):
        qs = make_queries(q=q, tokens=tokens, q_indptr=FAKE, max_tokens=16)
        r = _RopeC()
        r.rotary_dim = 128
        return lib.tsd_rope_append(ctypes.byref(c), ctypes.byref(qs), ctypes.byref(r), q_stride, k, 1024, v, 1024, None, None,
                                   out, None, None)
    invalid, q = tsd.TSD_ERR_INVALID_ARGUMENT, FAKE + 0x1000000
    fine = lambda status: status in (tsd.TSD_OK, tsd.TSD_ERR_CUDA)   # no GPU: the launch itself fails
    assert append(q + 256) == invalid and append(q - 256) == invalid
    assert append(q, q_stride=8192) == invalid                       # in place, but rows move
    assert fine(append(q)) and fine(append(q, q_stride=8192, tokens=1))
    assert fine(append(q + bytes_q)) and fine(append(q - bytes_q))
    assert append(FAKE + 0x2000000) == invalid and append(FAKE + 0x3000000 + bytes_k - 16) == invalid
    assert fine(append(FAKE + 0x2000000 + bytes_k))

    def decode(out, dt):
        qs = make_queries(q=q, tokens=T, q_indptr=FAKE, max_tokens=16)
        return lib.tsd_tree_decode(ctypes.byref(c), ctypes.byref(qs), None, out, dt, None, FAKE, 1 << 40, None, None)
    assert decode(q, 0) == invalid and decode(q + bytes_q - 16, 0) == invalid
    assert decode(q - bytes_q, 1) == invalid                         # fp32 outputs are twice as long
    assert fine(decode(q - bytes_q, 0)) and fine(decode(q + bytes_q, 1))


def test_workspace_size_and_call_take_the_same_queries(lib):
    """Without q_indptr there is one token a sequence, whatever max_tokens_per_seq says."""
    c = make_cache()
    size = lambda **kw: lib.tsd_tree_decode_workspace_size(ctypes.byref(c), ctypes.byref(make_queries(**kw)), 0)
    assert size(max_tokens=600) == size(max_tokens=1) > 0
    assert size(tokens=2000, q_indptr=FAKE, max_tokens=513) == 0 < size(tokens=2000, q_indptr=FAKE, max_tokens=512)


@fake_pointer_call
def test_positions_behind_a_sequence_fit_32_bits(lib):
    """A table may name a page many times, so lengths are not bounded by the pool."""
    def decode(length):
        c = make_cache(page_size=256, max_pages=2 ** 23, max_seq_len=length, batch=1, hkv=1)
        q = make_queries(tokens=1, hq=1)
        return lib.tsd_tree_decode(ctypes.byref(c), ctypes.byref(q), None, FAKE, 0, None, FAKE, 1 << 40, None, None)
    assert decode(2 ** 31 - 1) == decode(2 ** 31 - 4096) == tsd.TSD_ERR_UNSUPPORTED
    assert decode(2 ** 31 - 4097) == tsd.TSD_ERR_CUDA   # no GPU: past every check
