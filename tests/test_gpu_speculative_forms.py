"""Forms of the speculative kernels that a rule chooses by size, each at the sizes that choose it."""

import numpy as np
import pytest

import top_sparse_decode_topk_b200 as tsd
from oracle import speculative as S
from tests.test_gpu_speculative import compact_case, i32, rope_case, run_tree, status
from tests.test_gpu_tree_wide import compare, expected, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_flags_left():
    status()
    yield
    assert status() == 0


@pytest.mark.parametrize("page", [0, 2, 16])
@pytest.mark.parametrize("kw", [{}, dict(interleaved=True, rotary_dim=64), dict(rotary_dim=50), dict(interleaved=True, rotary_dim=6)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rope_several_tokens_a_block(dtype, kw, page):
    """One sequence of 41 new tokens among 21 of 0 to 2: a block takes four tokens (22 x 41 > 4 x 62)."""
    counts = [0, 1, 2] * 4 + [41] + [2, 1, 0] * 3
    assert len(counts) * max(counts) > 4 * sum(counts)
    before = [int(x) for x in np.random.default_rng(page).integers(0, 50, len(counts))]
    rope_case(counts, before, 6, 2, page, dtype, kw, at="depth", fused=True, seed=page)
    rope_case(counts, before, 6, 2, page, dtype, kw, in_place=True, seed=page + 1)


@pytest.mark.parametrize("qt,ot", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_tree_contiguous_caches_smaller_than_a_tile(qt, ot):
    run_tree([1], [0], 1, 1, 0, qt, ot, mask="chain")
    run_tree([3], [2], 2, 1, 0, qt, ot)
    run_tree([2, 1], [9, 30], 4, 2, 0, qt, ot, mask="custom")


@pytest.mark.parametrize("page", [0, 8])
def test_compact_more_drafts_than_are_resolved_at_once(page):
    """Lists of more than 256 kept drafts are worked off in parts."""
    compact_case([600, 300], [3, 70], [list(range(1, 600, 2)), list(range(20, 300))], page, hkv=3)
    compact_case([513, 257], [0, 9], [list(range(513)), [0] + list(range(2, 257))], page)


@pytest.mark.parametrize("offset", [0, 1])
def test_resize_over_more_pages_than_a_warp_keeps(offset):
    """More than 8 groups of 128 pages for each of the 224 warps that count; refs at any 4-byte address."""
    import torch
    pool, B, width = 300_001, 300, 64
    rng = np.random.default_rng(offset)
    refs = i32(np.concatenate([np.zeros(offset, int), (rng.random(pool) < 0.97)]))[offset:]
    k = torch.zeros(pool, 1, 1, 128, dtype=torch.bfloat16, device="cuda")
    table, lens = i32(np.full((B, width), -1)), i32(np.zeros(B))
    cache = tsd.KVCache(k, k, lens, width, page_table=table)
    model = S.Pool(table.cpu(), [0] * B, refs.cpu(), 1, width)
    for step in range(5):
        new = rng.integers(0, width + 1, B)
        new = np.where(rng.random(B) < 0.3, model.lens, new)
        tsd.cache_resize(cache, refs, i32(new))
        model.resize(new.tolist())
        assert np.array_equal(table.cpu().numpy(), model.table) and np.array_equal(refs.cpu().numpy(), model.refs)
        assert np.array_equal(lens.cpu().numpy(), model.lens)
        assert status() == sum({"NO_PAGES": tsd.DEV_NO_PAGES}[f] for f in model.flags)
        model.flags.clear()


@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 128])
@pytest.mark.parametrize("qt,ot", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_tree_bad_pages_of_every_size(qt, ot, page):
    """Rows of unreadable pages, among the committed tokens and the drafts, drop out, whatever other pages hold."""
    import torch
    n, length, hkv, hq = 20, 700, 2, 8
    dts = {"bf16": torch.bfloat16, "f32": torch.float32}
    cache, table = filled([length, length - 300], hkv, page, page, spare=9)
    used = np.zeros(cache.k.shape[0], bool)
    used[table[table >= 0]] = True
    bad = sorted({p // page * page for p in (0, 130, 131, 333, length - 15)})
    for x in (cache.k, cache.v):
        x[torch.from_numpy(~used).cuda()] = float("nan")
        for p in bad:                                          # the pages that are named no more
            x[int(table[0, p // page])] = float("nan")
    for i, p in enumerate(bad):
        cache.page_table[0, p // page] = (-1, 10 ** 9, cache.k.shape[0], -2 ** 31)[i % 4]
    gone = np.concatenate([np.arange(p, min(length, p + page)) for p in bad])
    q = torch.randn(n + 3, hq, 128, device="cuda").to(dts[qt])
    st = i32([0])
    out, lse = tsd.tree_decode(cache, tsd.Queries(q, i32([0, n, n + 3]), n), None, out_dtype=dts[ot], status=st)
    assert int(st) == tsd.DEV_BAD_PAGE
    for row, t0, m, end, lost in ((table[0], 0, n, length, gone), (table[1], n, 3, length - 300, ())):
        # the formula's copy of a lost row is any number: it is masked
        k = tsd.KVCache(torch.nan_to_num(cache.k), torch.nan_to_num(cache.v), cache.seq_lens, length, page_table=cache.page_table)
        compare(out[t0:t0 + m], lse[t0:t0 + m], *expected(k, row, page, q, t0, m, end, np.tril(np.ones((m, m), bool)),
                                                          1 / np.sqrt(128), lost), ot == "bf16")
