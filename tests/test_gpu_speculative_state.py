"""What the speculative calls keep and write besides their outputs: workspaces, status words, tables, lengths."""

import numpy as np
import pytest

import top_sparse_decode_topk_b200 as tsd
from tests.test_gpu_speculative import Serving, i32, make_cache, status

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_flags_left():
    status()
    yield
    assert status() == 0


def test_a_workspace_keeps_the_status_of_its_calls():
    """Other calls, other shapes and growth do not lose a bit that nobody has read."""
    import torch
    s = Serving(3, 4, 40, 12)
    ws = tsd.Workspace("cuda")
    s.resize([20, 8, 0])
    tsd.cache_resize(s.layers, s.refs, i32([20, 40, 0]), workspace=ws)      # no pages for sequence 1
    q = torch.randn(3, 2, 128, device="cuda").bfloat16()
    cache, _ = make_cache([300, 200, 9], 2, 16)
    ref = tsd.tree_decode(cache, tsd.Queries(q))
    got = tsd.tree_decode(cache, tsd.Queries(q), workspace=ws)               # more scratch than the call before
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    tsd.dense_decode(cache, tsd.Queries(q), workspace=ws)
    tsd.decode_step(cache, tsd.Queries(q), 32, workspace=ws)
    qs = tsd.Queries(torch.randn(60, 16, 128, device="cuda"), i32([0, 20, 40, 60]), 20)
    tsd.tree_decode(cache, qs, out_dtype=torch.float32, workspace=ws)        # sequence 2 holds 9 tokens, not 20 drafts
    assert tsd.read_device_status(ws) == tsd.DEV_NO_PAGES | tsd.DEV_BAD_SEQ
    assert tsd.read_device_status(ws) == 0
    s.check()


def test_scratch_of_these_calls_leaves_the_other_calls_state_alone():
    """A captured dense step whose workspace is zero at the start of every replay, though tree_decode uses it too."""
    import torch
    cache, _ = make_cache([3000, 200, 9000], 2, 16)
    q = torch.randn(3, 4, 128, device="cuda").bfloat16()
    qs = tsd.Queries(q)
    ws = tsd.Workspace("cuda")
    dense = [x.clone() for x in tsd.dense_decode(cache, qs)]
    tree = [x.clone() for x in tsd.tree_decode(cache, qs, workspace=ws)]
    tsd.dense_decode(cache, qs, workspace=ws)
    torch.cuda.synchronize()
    before = ws.buf.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = tsd.dense_decode(cache, qs, workspace=ws)
        b = tsd.tree_decode(cache, qs, workspace=ws)
    for _ in range(3):
        for x in (*a, *b):
            x.fill_(9)
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip(a, dense)) and all(torch.equal(x, y) for x, y in zip(b, tree))
        tsd.tree_decode(cache, tsd.Queries(torch.randn(3, 32, 128, device="cuda")), out_dtype=torch.float32, workspace=ws)
    tsd.tree_decode(cache, qs, workspace=ws)
    assert ws.buf.numel() == before.numel() and torch.equal(ws.buf[:256], before[:256])
    del g
    assert tsd.read_device_status(ws) == 0


def test_a_status_word_is_not_made_during_a_capture(monkeypatch):
    import torch
    cache, _ = make_cache([30, 20], 2, 16)
    qs = tsd.Queries(torch.randn(2, 4, 128, device="cuda"))
    want = tsd.tree_decode(cache, qs)
    ws, parents = tsd.Workspace("cuda"), i32([-1])   # made here: no copies from the host in a capture
    with pytest.raises(RuntimeError, match="before capturing"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            tsd.tree_decode(cache, qs, workspace=ws)
    monkeypatch.setattr(tsd.speculative, "_STATUS", {})
    with pytest.raises(RuntimeError, match="before capturing"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            tsd.tree_mask(parents)
    assert all(torch.equal(a, b) for a, b in zip(tsd.tree_decode(cache, qs, workspace=ws), want))


def test_a_table_or_lengths_that_cannot_be_updated_in_place_are_refused():
    import torch
    page = lambda: torch.zeros(12, 2, 4, 128, dtype=torch.bfloat16, device="cuda")
    wide, state, refs = i32(np.full((3, 20), -1)), i32(np.zeros((3, 2))), i32(np.zeros(12))
    lens = i32([0, 0, 0])
    sliced = tsd.KVCache(page(), page(), lens, 40, page_table=wide[:, :10])
    strided = tsd.KVCache(page(), page(), state[:, 0], 40, page_table=wide[:, :10].contiguous())
    short = tsd.KVCache(page(), page(), lens, 40, page_table=i32(np.full((2, 10), -1)))
    for cache in (sliced, strided, short):
        with pytest.raises(ValueError):
            tsd.cache_resize(cache, refs, i32([4, 0, 0]))
        with pytest.raises(ValueError):
            tsd.cache_fork(cache, refs, i32([0]), i32([1]))
    x = torch.zeros(3, 4, 128, device="cuda")
    for cache in (strided, short):      # reads that would go astray
        with pytest.raises(ValueError):
            tsd.tree_decode(cache, tsd.Queries(x))
        with pytest.raises(ValueError):
            tsd.rope_append(cache, tsd.RotaryEmbedding(), x, x[:, :2], x[:, :2])
        with pytest.raises(ValueError):
            tsd.cache_compact(cache, i32([[0]] * 3))
    assert (wide == -1).all() and not state.any() and not refs.any() and not lens.any()
    ok = tsd.KVCache(page(), page(), lens, 80, page_table=wide)
    tsd.cache_resize(ok, refs, i32([4, 0, 0]))
    assert wide[0, 0] == 0 and lens.tolist() == [4, 0, 0]


def test_pages_are_copied_in_the_tensors_that_the_caches_hold_now():
    import torch
    s = Serving(3, 8, 64, 20)
    s.resize([21, 0, 0])
    s.fork([0], [1])
    old = s.kv.clone()
    s.kv = s.kv + 1                      # a pool somewhere else
    for i, c in enumerate(s.layers.caches):
        c.k, c.v = s.kv[2 * i], s.kv[2 * i + 1]
    s.model.data = s.data()
    s.resize([21, 23, 0])                # the shared page is copied, in the new pool
    before = s.kv.clone()
    keep = i32([[-1, -1], [1, -1], [-1, -1]])
    out = tsd.cache_compact(s.layers, keep, i32([0, 0, 2, 2]), 2, refs=s.refs)
    assert out.tolist() == [21, 22, 0]
    p = int(s.table[1, 2])
    before[:, p, :, 5] = before[:, p, :, 6]
    assert torch.equal(s.kv, before) and old.shape == before.shape


@pytest.mark.parametrize("ip", [[2, 6, 9], [0, 4, 7], [1000, 1004, 1007], [2 ** 31 - 8, 2 ** 31 - 4, 2 ** 31 - 1]])
def test_compact_takes_any_range_of_tokens(ip):
    """Ranges that do not start at 0, as rope_append and tree_decode take them."""
    import torch
    cache, table = make_cache([14, 23], 2, 4, fill="other")
    k, v = cache.k.clone(), cache.v.clone()
    out = tsd.cache_compact(cache, i32([[1, 3], [0, 2]]), i32(ip), 4)
    assert out.tolist() == [12, 22]
    for b, dst, src in ((0, 10, 11), (0, 11, 13), (1, 21, 22)):
        d, s = (int(table[b, dst // 4]), dst % 4), (int(table[b, src // 4]), src % 4)
        for x in (k, v):
            x[d[0], :, d[1]] = x[s[0], :, s[1]].clone()
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v)
    tsd.cache_compact(cache, i32([[1, 3], [0, 2]]), i32([2, 7, 9]), 4)   # five drafts are above the bound, and draft 2 of two
    assert status() == tsd.DEV_BAD_SEQ | tsd.DEV_BAD_INDEX
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v)


def test_trees_of_different_sizes_from_several_host_threads():
    """Each thread's calls find the shared memory that their size needs."""
    import sys
    import threading
    import torch
    lib = tsd.load_library()
    sizes, wrong = (440, 512), []
    inputs = {n: (i32([0, n, 2 * n]), i32(list(range(-1, n - 1)) * 2), i32([0])) for n in sizes}
    outs = [(i32(np.zeros((2 * sizes[i % 2], 16))), i32(np.zeros(2 * sizes[i % 2])), torch.cuda.Stream()) for i in range(8)]
    torch.cuda.synchronize()

    def work(i):
        n = sizes[i % 2]
        (ip, parents, st), (mask, depth, stream) = inputs[n], outs[i]
        args = (2, ip.data_ptr(), 2 * n, n, parents.data_ptr(), mask.data_ptr(), depth.data_ptr(), st.data_ptr(),
                stream.cuda_stream)
        wrong.extend(x for x in (lib.tsd_tree_mask(*args) for _ in range(4000)) if x)

    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    try:
        for t in threads:
            t.start()
    finally:
        for t in threads:
            t.join()
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    assert not wrong, (len(wrong), set(wrong))
    for i, (_, depth, _) in enumerate(outs):
        n = sizes[i % 2]
        assert depth.tolist() == list(range(n)) * 2 and int(inputs[n][2]) == 0


@pytest.mark.parametrize("shrink,grow", [(128, 128), (700, 700)])
def test_pages_that_refs_has_as_free_are_not_released_from_their_new_holder(shrink, grow):
    """Tables name pages that refs has as free, and the call that ends those sequences hands the pages out: whoever comes
    first, the new holders' counts stand."""
    import torch
    B, per = shrink + grow, 4
    pool = torch.zeros(shrink * per, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    for seed in range(20):
        rng = np.random.default_rng(seed)
        who = rng.permutation(B)
        table, lens, new = np.full((B, per), -1), np.zeros(B, int), np.zeros(B, int)
        table[who[:shrink]] = rng.permutation(shrink * per).reshape(shrink, per)
        lens[who[:shrink]], new[who[shrink:]] = 2 * per, 2 * per
        refs, st = i32(np.zeros(shrink * per)), i32([0])
        cache = tsd.KVCache(pool, pool, i32(lens), 2 * per, page_table=i32(table))
        tsd.cache_resize(cache, refs, i32(new), status=st)
        assert int(st) == tsd.DEV_BAD_PAGE
        assert (refs == 1).all(), int((refs != 1).sum())
        held = cache.page_table.cpu().numpy()
        assert (held[who[:shrink]] == -1).all()
        assert held[np.sort(who[shrink:])].ravel().tolist() == list(range(shrink * per))
        assert cache.seq_lens.tolist() == new.tolist()


def test_counts_do_not_fall_below_zero():
    """Three sequences hold a page that refs counts twice, and all of them grow out of it."""
    import torch
    pool = torch.zeros(8, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    table = i32([[3, -1], [3, -1], [3, -1]])
    refs, st = i32([0, 0, 0, 2, 0, 0, 0, 0]), i32([0])
    cache = tsd.KVCache(pool, pool, i32([2, 2, 2]), 8, page_table=table)
    tsd.cache_resize(cache, refs, i32([3, 3, 3]), status=st)
    assert int(st) == tsd.DEV_BAD_PAGE
    assert refs.tolist() == [1, 1, 1, 0, 0, 0, 0, 0] and table[:, 0].tolist() == [0, 1, 2]


def test_outputs_that_overlap_inputs_are_refused():
    import torch
    cache, _ = make_cache([40, 30], 2, 16, fill="other")
    buf = torch.zeros(2 * 6 * 4 * 128, device="cuda").bfloat16()
    q, ip = buf[:6 * 512].view(6, 4, 128), i32([0, 3, 6])
    shifted = buf[512:7 * 512].view(6, 4, 128)
    x = torch.zeros(6, 2, 128, device="cuda").bfloat16()
    rope = tsd.RotaryEmbedding()
    with pytest.raises(tsd.TsdError):
        tsd.rope_append(cache, rope, q, x, x, ip, 3, out_q=shifted)
    with pytest.raises(tsd.TsdError):
        tsd.rope_append(cache, rope, q, buf[6 * 512:9 * 512].view(6, 2, 128), x, ip, 3, out_q=shifted)
    assert tsd.rope_append(cache, rope, q, x, x, ip, 3, out_q=q) is q
    assert tsd.rope_append(cache, rope, q, x, x, ip, 3, out_q=buf[6 * 512:].view(6, 4, 128)).shape == q.shape
    for out in (q, shifted):
        with pytest.raises(tsd.TsdError):
            tsd.tree_decode(cache, tsd.Queries(q, ip, 3), out=out)
    tsd.tree_decode(cache, tsd.Queries(q, ip, 3), out=buf[6 * 512:].view(6, 4, 128))
