"""rope_append, tree_mask, tree_decode, cache_fork, cache_resize and cache_compact against oracle/speculative.py.

Tolerances count roundings.  Half a step is 2^-8 of the value in bf16 and 2^-24 in fp32.
 * Rotation: the reduced angle is off by at most 2^-24 of half a turn (rounded to fp32; pi 2^-24 < 2e-7
   radians) and sine and cosine by 2 units in the last place (2^-22): with three roundings of the sum, at most
   (2e-7 + 2.4e-7 + 2e-7) (|a| + |b|) < 7e-7 (|a| + |b|).
 * Attention: a score is a sum of 128 products in fp32, off by dz <= 128 2^-24 scale sum |q_d k_d| (bf16
   products are exact), 2^-16 of that more for the fp32 exponent arithmetic; an error dz in every exponent
   changes a weighted mean by at most 2 dz sum p|V|; weights of 2^-8 (bf16 outputs; a bf16 weight) or
   2^-22 (fp32 outputs) each by that times sum p|V|.
"""

import math

import numpy as np
import pytest

import top_sparse_decode_topk_b200 as tsd
from oracle import speculative as S

pytestmark = pytest.mark.gpu


def status():
    return tsd.read_device_status(device="cuda:0")


@pytest.fixture(autouse=True)
def no_flags_left():
    status()
    yield
    assert status() == 0


def i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda").contiguous()


def np64(t):
    return t.detach().double().cpu().numpy()


def make_cache(lens, hkv, page, seed=0, fill="randn", max_len=None, spare=3):
    """A paged (page > 0) or contiguous cache; unused slots hold NaN when filled with random numbers."""
    import torch
    rng = np.random.default_rng(seed)
    B, L = len(lens), max(1, max_len or max(lens))
    if page:
        width = -(-L // page)
        need = [-(-x // page) for x in lens]
        pool = sum(need) + spare
        order, table, at = rng.permutation(pool), np.full((B, width), -1, np.int64), 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        shape = (pool, hkv, page, 128)
    else:
        table, shape = None, (B, hkv, L, 128)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    mk = lambda: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    k, v = mk(), mk()
    if fill == "randn":
        used = np.zeros((shape[0], shape[2]), bool)
        for b, n in enumerate(lens):
            for i in range(n):
                used[(table[b, i // page], i % page) if page else (b, i)] = True
        hole = torch.from_numpy(~used).cuda()[:, None, :, None]
        k.masked_fill_(hole, float("nan"))
        v.masked_fill_(hole, float("nan"))
    cache = tsd.KVCache(k, v, i32(lens), L, page_table=None if table is None else i32(table))
    return cache, table


def rows_of(cache, table, b, n, page, arrays=None):
    """(K, V) of the first n tokens of sequence b as [Hkv, n, 128] float64 (arrays: K and V, where they are
    at hand)."""
    i = np.arange(n)
    k, v = arrays or (np64(cache.k), np64(cache.v))
    if not page:
        return k[b][:, :n], v[b][:, :n]
    p, s = table[b, i // page], i % page
    return k[p, :, s].transpose(1, 0, 2), v[p, :, s].transpose(1, 0, 2)


# ---------------------------------------------------------------------------------------------------------------------
# rope_append
# ---------------------------------------------------------------------------------------------------------------------
def rope_case(counts, before, hq, hkv, page, dtype, kw, at="row", fused=False, seed=0, in_place=False):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    T = sum(counts)
    lens = [a + n for a, n in zip(before, counts)]
    cache, table = make_cache(lens, hkv, page, seed, fill="other")
    k0, v0 = cache.k.clone(), cache.v.clone()
    g = torch.Generator(device="cuda").manual_seed(seed + 7)
    if fused:
        x = torch.randn(T, hq + 2 * hkv, 128, generator=g, device="cuda").to(dt)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = (torch.randn(T, h, 128, generator=g, device="cuda").to(dt) for h in (hq, hkv, hkv))
    rng = np.random.default_rng(seed)
    rope = tsd.RotaryEmbedding(**kw)
    ip = None if counts == [1] * len(counts) else i32(np.concatenate([[0], np.cumsum(counts)]))
    row = np.concatenate([np.arange(a, a + n) for a, n in zip(before, counts)]).astype(int)
    pos, extra = row.copy(), {}
    if at == "positions":
        pos = rng.integers(-5, 2 ** 31 - 1, T)
        extra["positions"] = i32(pos)
    elif at == "depth":
        d = rng.integers(0, 9, T)
        pos = np.concatenate([np.full(n, a) for a, n in zip(before, counts)]).astype(int) + d
        extra["depth"] = i32(d)
    xq, xk, xv = np64(q), np64(k), np64(v)
    if in_place:
        extra["out_q"] = q
    out = tsd.rope_append(cache, rope, q, k, v, q_indptr=ip, max_tokens_per_seq=max(counts), **extra)
    o = dict(kw)
    R, inter = o.pop("rotary_dim", 128), o.pop("interleaved", False)
    freq, ms = S.rope_frequencies(R, o.pop("theta", 10000.0), **o)
    pair = (lambda x: np.abs(x) + np.abs(S_partner(x, R, inter)))
    for got, x, half in ((np64(out), xq, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24),):
        ref = S.rope_rotate(x, pos.astype(np.float64), freq, ms, inter)
        assert (np.abs(got - ref) <= half * np.abs(ref) + 7e-7 * ms * pair(x)).all()
        assert np.array_equal(got[..., R:], x[..., R:])
    kk, vv = np64(cache.k), np64(cache.v)
    bseq = np.repeat(np.arange(len(counts)), counts)
    where = (table[bseq, row // page], row % page) if page else (bseq, row)
    ref = S.rope_rotate(xk, pos.astype(np.float64), freq, ms, inter)
    assert (np.abs(kk[where[0], :, where[1]] - ref) <= 2.0 ** -8 * np.abs(ref) + 7e-7 * ms * pair(xk)).all()
    assert np.array_equal(vv[where[0], :, where[1]], np64(v.to(torch.bfloat16)) if not in_place else
                          np64(torch.from_numpy(xv).to(dt).to(torch.bfloat16)))
    # every other row is as it was
    keep = np.ones((kk.shape[0], kk.shape[2]), bool)
    keep[where] = False
    keep = torch.from_numpy(keep).cuda()[:, None, :, None].expand_as(cache.k)
    assert torch.equal(cache.k[keep], k0[keep]) and torch.equal(cache.v[keep], v0[keep])


def S_partner(x, R, inter):
    y = np.zeros_like(x)
    if inter:
        y[..., 0:R:2], y[..., 1:R:2] = x[..., 1:R:2], x[..., 0:R:2]
    else:
        y[..., :R // 2], y[..., R // 2:R] = x[..., R // 2:R], x[..., :R // 2]
    return y


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("R", [128, 96, 64, 50, 32, 24, 16, 8, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rope_layouts(dtype, R, inter):
    rope_case([3, 0, 1, 5], [10, 0, 0, 31], 6, 2, 8, dtype, dict(rotary_dim=R, interleaved=inter), fused=R % 16 == 0)


@pytest.mark.parametrize("page", [0, 1, 2, 16, 64])
@pytest.mark.parametrize("at", ["row", "positions", "depth"])
def test_rope_positions_and_pages(page, at):
    """Positions up to 2^31 keep fp32 accuracy; counts from 0 to 70."""
    rope_case([70, 1, 0, 33], [5, 100, 3, 0], 8, 4, page, "f32", dict(theta=500000.0), at=at, fused=True, seed=page)


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
    dict(scaling="banded", factor=8.0, original_max_len=64.0), dict(scaling="yarn", factor=4.0, original_max_len=64.0)])
def test_rope_scaling(kw):
    rope_case([40, 7], [300, 2], 5, 5, 16, "f32", kw, at="positions")


def test_rope_one_token_each_and_in_place_and_many():
    rope_case([1, 1, 1], [0, 7, 129], 8, 1, 16, "bf16", {})
    rope_case([1, 1, 1], [0, 7, 129], 8, 1, 16, "f32", dict(rotary_dim=50), in_place=True)
    rope_case([9, 2], [4, 4], 3, 3, 4, "bf16", dict(interleaved=True), in_place=True)
    rope_case([2500, 300], [0, 50], 4, 2, 16, "bf16", {}, fused=True)   # several tokens a block


def test_rope_bad_rows_are_skipped_and_flagged():
    import torch
    cache, table = make_cache([20, 9, 6], 2, 4, fill="other")
    cache.page_table[0, 4] = 99          # tokens 16 .. 19
    cache.page_table[1, 2] = -1          # token 8
    before = cache.k.clone()
    x = torch.ones(8, 2, 128, device="cuda")
    st = i32([0])
    rope = tsd.RotaryEmbedding()
    out = torch.full((8, 2, 128), 5.0, device="cuda")
    tsd.rope_append(cache, rope, x, x, x, q_indptr=i32([0, 5, 7, 8]), max_tokens_per_seq=5, out_q=out, status=st)
    assert int(st) == tsd.DEV_BAD_PAGE
    changed = (cache.k != before).any(-1).any(1).cpu().numpy()
    want = np.zeros_like(changed)
    want[table[0, 3], 3] = want[table[1, 1], 3] = want[table[2, 1], 1] = True
    assert np.array_equal(changed, want)
    assert abs(out).max() < 2    # every token's query is rotated all the same
    # more new tokens than the sequence holds, and a bad q_indptr: the sequence is left alone
    out.fill_(5.0)
    st.zero_()
    cache.seq_lens[0] = 4
    before = cache.k.clone()
    tsd.rope_append(cache, rope, x, x, x, q_indptr=i32([0, 5, 4, 8]), max_tokens_per_seq=5, out_q=out, status=st)
    assert int(st) == tsd.DEV_BAD_SEQ
    # tokens 0 .. 3 belong to the first sequence (refused) alone, tokens 4 .. 7 to the third as well
    assert torch.equal(out[:4], torch.full_like(out[:4], 5.0)) and (out[4:] != 5).any()


def test_rope_refusals():
    import torch
    cache, _ = make_cache([20, 9], 2, 4, fill="other")
    rope = tsd.RotaryEmbedding()
    ok = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)
    run = lambda q=ok(2, 4, 128), k=ok(2, 2, 128), v=ok(2, 2, 128), **kw: tsd.rope_append(cache, rope, q, k, v, **kw)
    run()
    for bad in (dict(q=ok(2, 4, 64)), dict(k=ok(2, 3, 128)), dict(v=ok(3, 2, 128)), dict(k=ok(2, 2, 128).bfloat16()),
                dict(q=ok(2, 128, 4).transpose(1, 2)), dict(positions=ok(2)), dict(depth=i32([1, 2, 3])),
                dict(q_indptr=i32([0, 2])), dict(out_q=ok(2, 4, 128).bfloat16()), dict(k=torch.zeros(2, 2, 128))):
        with pytest.raises((ValueError, TypeError)):
            run(**bad)
    with pytest.raises(TypeError):
        run(q=ok(2, 4, 128).half(), k=ok(2, 2, 128).half(), v=ok(2, 2, 128).half())
    with pytest.raises(tsd.TsdError):
        run(positions=i32([1, 2]), depth=i32([1, 2]))
    with pytest.raises(tsd.TsdError):   # rows that are not 16-byte aligned
        run(q=ok(2 * 4 * 128 + 1)[1:].view(2, 4, 128))


# ---------------------------------------------------------------------------------------------------------------------
# tree_mask
# ---------------------------------------------------------------------------------------------------------------------
def random_parents(rng, n, kind):
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] * n
    return [-1 if j == 0 or rng.random() < 0.2 else int(rng.integers(max(0, j - 5), j)) for j in range(n)]


@pytest.mark.parametrize("kind", ["chain", "star", "random"])
@pytest.mark.parametrize("counts", [[1], [1, 1, 1], [5, 0, 33, 1], [64, 31, 32], [512, 3, 511]])
def test_tree_mask(counts, kind):
    rng = np.random.default_rng(len(counts))
    par = [random_parents(rng, n, kind) for n in counts]
    ip = i32(np.concatenate([[0], np.cumsum(counts)]))
    mask, depth = tsd.tree_mask(i32(sum(par, [])), ip, max(counts))
    W = (max(counts) + 31) // 32
    rows = [S.tree_rows(p) for p in par]
    assert np.array_equal(mask.cpu().numpy().view(np.uint32), np.concatenate([S.pack_rows(r, W) for r in rows if r]))
    assert depth.tolist() == [len(x) - 1 for r in rows for x in r]
    if counts == [1, 1, 1]:
        m2, d2 = tsd.tree_mask(i32(sum(par, [])))
        assert m2.tolist() == [[1]] * 3 and d2.tolist() == [0] * 3


def test_tree_mask_bad_parents():
    st = i32([0])
    mask, depth = tsd.tree_mask(i32([-1, 0, 2, 7, -2, 3]), i32([0, 6]), 6, status=st)
    assert int(st) == tsd.DEV_BAD_TREE
    assert [x[0] for x in mask.tolist()] == [1, 3, 4, 8, 16, 8 + 32] and depth.tolist() == [0, 1, 0, 0, 0, 1]
    st.zero_()
    mask.fill_(77)
    tsd.tree_mask(i32([-1] * 6), i32([0, 4, 3]), 3, mask=mask, status=st)   # too many drafts; a range that runs backwards
    assert int(st) == tsd.DEV_BAD_SEQ and mask.tolist() == [[77]] * 6


# ---------------------------------------------------------------------------------------------------------------------
# tree_decode
# ---------------------------------------------------------------------------------------------------------------------
def check_tree(cache, table, page, q, counts, lens, rows, out, lse, scale):
    hkv, hq = cache.num_kv_heads, q.shape[1]
    G = hq // hkv
    o, l, qq = np64(out), np64(lse), np64(q)
    bf16_out = str(out.dtype) == "torch.bfloat16"
    t, arrays = 0, (np64(cache.k), np64(cache.v))
    for b, n in enumerate(counts):
        K, V = rows_of(cache, table, b, lens[b], page, arrays)
        for g in range(hkv):
            ref, rl, spread = S.tree_attention(qq[t:t + n, g * G:(g + 1) * G], K[g], V[g], lens[b] - n, rows[b], scale)
            got, gl = o[t:t + n, g * G:(g + 1) * G], l[t:t + n, g * G:(g + 1) * G]
            size = scale * (np.abs(qq[t:t + n, g * G:(g + 1) * G]) @ np.abs(K[g]).T).max(-1, initial=0.0)
            dz = size * (128 + 2) * 2.0 ** -24 + 2.0 ** -16 * 2.0 ** -8
            tol = (2 * dz[..., None] + (2.0 ** -8 if bf16_out else 2.0 ** -22)) * spread + \
                (2.0 ** -8 if bf16_out else 2.0 ** -23) * np.abs(ref)
            empty = np.isneginf(rl)
            assert np.array_equal(np.isneginf(gl), empty)
            assert not got[empty].any()
            bad = np.abs(got - ref) > tol
            assert not bad.any(), (b, g, np.argwhere(bad)[:4], np.abs(got - ref).max())
            fine = ~empty
            assert (np.abs(gl - np.where(fine, rl, 0))[fine] <= (dz + 2.0 ** -22 * (4 + np.abs(rl)))[fine]).all()
        t += n


def run_tree(counts, before, hq, hkv, page, qt="bf16", ot="bf16", mask="random", seed=0, scale=None, max_n=None):
    import torch
    dts = {"bf16": torch.bfloat16, "f32": torch.float32}
    lens = [a + n for a, n in zip(before, counts)]
    cache, table = make_cache(lens, hkv, page, seed)
    T, n_max = sum(counts), max_n or max(counts)
    g = torch.Generator(device="cuda").manual_seed(seed + 3)
    q = (2 * torch.randn(T, hq, 128, generator=g, device="cuda")).to(dts[qt])
    rng = np.random.default_rng(seed)
    if mask == "custom":   # any bits, rows that see nothing
        rows = [[{i for i in range(n) if rng.random() < 0.3} if rng.random() < 0.7 else set() for _ in range(n)] for n in counts]
    else:
        rows = [S.tree_rows(random_parents(rng, n, mask)) for n in counts]
    W = (n_max + 31) // 32
    words = np.concatenate([S.pack_rows(r, W) for r in rows if r])
    if mask == "custom":   # bits behind a sequence's drafts mean nothing
        t = 0
        for n in counts:
            for j in range(n):
                for i in range(n, 32 * W):
                    if rng.random() < 0.5:
                        words[t + j, i >> 5] |= np.uint32(1 << (i & 31))
            t += n
    scale = scale or 1 / math.sqrt(128)
    ip = None if counts == [1] * len(counts) else i32(np.concatenate([[0], np.cumsum(counts)]))
    qs = tsd.Queries(q, q_indptr=ip, max_tokens_per_seq=n_max, sm_scale=scale)
    m = None if mask == "chain" else i32(words.view(np.int32))
    out, lse = tsd.tree_decode(cache, qs, m, out_dtype=dts[ot])
    check_tree(cache, table, page, q, counts, lens, rows, out, lse, scale)
    return cache, qs, m, out, lse


@pytest.mark.parametrize("page", [0, 1, 2, 4, 8, 16, 32, 128, 256])
@pytest.mark.parametrize("qt,ot", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_tree_pages_and_types(page, qt, ot):
    run_tree([8, 3, 0, 12], [500, 0, 7, 130], 8, 2, page, qt, ot, seed=page)


@pytest.mark.parametrize("before", [0, 1, 2, 15, 16, 17, 63, 64, 65, 119, 120, 121, 127, 128, 129, 255, 256, 257, 1000, 4097])
def test_tree_lengths(before):
    run_tree([9, 1], [before, 3], 4, 1, 16, seed=before)
    run_tree([9, 1], [before, 3], 4, 1, 16, "f32", "f32", mask="custom", seed=before)


@pytest.mark.parametrize("G,hkv,n", [(1, 1, 1), (1, 8, 5), (4, 2, 8), (4, 2, 31), (4, 2, 32), (4, 2, 33), (5, 3, 13), (7, 4, 19),
                                     (8, 1, 64), (8, 2, 17), (2, 2, 129), (1, 2, 300), (16, 1, 40), (1, 1, 512)])
@pytest.mark.parametrize("mask", ["random", "custom", "chain"])
def test_tree_shapes(G, hkv, n, mask):
    run_tree([n, max(1, n // 2)], [200, 0], G * hkv, hkv, 16, mask=mask, seed=n)
    if n <= 64:
        run_tree([n, 1], [70, 300], G * hkv, hkv, 8, "f32", "f32", mask=mask, seed=n + 1)


def test_tree_one_token_each_and_long():
    run_tree([1, 1, 1, 1], [0, 1, 777, 3000], 8, 2, 16)
    run_tree([6, 2], [9000, 20], 8, 2, 16, seed=5)
    run_tree([40, 2], [5000, 3333], 32, 4, 16, seed=6)
    run_tree([3, 4], [10, 20], 4, 2, 16, max_n=7)   # a bound above every count
    run_tree([1] * 300, [11] * 300, 4, 2, 16, seed=7)
    run_tree(([1] * 3 + [0]) * 350, list(range(40)) * 35, 2, 2, 4, seed=8)   # more sequences than one step of a scan takes
    run_tree([2, 1], [70, 3], 8, 2, 16, max_n=64)   # a bound above all tokens of the step


def test_tree_large_scores():
    """Scores far apart (softmax saturates) and all equal."""
    run_tree([8], [300], 4, 2, 16, "f32", "f32", scale=3.0)
    run_tree([8], [300], 4, 2, 16, scale=1e-6)


def test_tree_chain_is_dense_decode():
    import torch
    cache, qs, _, out, lse = run_tree([7, 3], [700, 40], 8, 2, 16, "bf16", "f32", mask="chain")
    o2, l2 = tsd.dense_decode(cache, qs, out_dtype=torch.float32)
    assert (out - o2).abs().max() < 2e-4 and (lse - l2).abs().max() < 1e-4


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("ot", ["bf16", "f32"])
def test_tree_masked_drafts_may_hold_anything(what, ot):
    """A draft's K and V rows of infinities or not-a-numbers reach those that see it, and nobody else."""
    import torch
    counts, before, hq, hkv, page, n = [6, 5], [200, 125], 4, 2, 16, 6
    lens = [a + c for a, c in zip(before, counts)]
    for tensor in ("k", "v", "kv"):
        cache, table = make_cache(lens, hkv, page)
        clean, _ = make_cache(lens, hkv, page)
        for b in range(2):
            p, s = table[b, (before[b] + 2) // page], (before[b] + 2) % page   # draft 2 of each sequence
            for x in tensor:
                getattr(cache, x)[p, :, s] = what
        q = torch.randn(11, hq, 128, device="cuda").bfloat16()
        rows = [S.tree_rows([-1, 0, 0, 2, 1, 4][:c]) for c in counts]
        m = i32(np.concatenate([S.pack_rows(r, 1) for r in rows]).view(np.int32))
        qs = tsd.Queries(q, q_indptr=i32([0, 6, 11]), max_tokens_per_seq=n)
        dt = torch.bfloat16 if ot == "bf16" else torch.float32
        out, lse = tsd.tree_decode(cache, qs, m, out_dtype=dt)
        ref, rl = tsd.tree_decode(clean, qs, m, out_dtype=dt)
        sees = torch.tensor([2 in r for rr in rows for r in rr], device="cuda")
        assert torch.equal(out[~sees], ref[~sees]) and torch.equal(lse[~sees], rl[~sees])
        assert torch.isfinite(out[~sees]).all()
        if what != what:
            assert torch.isnan(out[sees]).all()
            if tensor != "v":
                assert torch.isnan(lse[sees]).all()
            else:
                assert torch.equal(lse[sees], rl[sees])
        elif tensor == "v":
            if abs(what) == float("inf"):
                assert (out[sees] == what).all()
            assert torch.equal(lse[sees], rl[sees])


@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [5, 70])
def test_tree_sums_over_long_contexts(qt, n):
    """fp32 outputs over contexts long enough that sums leave tensor memory several times, with scores that grow along
    the context, so that what was summed is rescaled afterwards."""
    import torch
    counts, before, hq, hkv, page = [n, 3], [24990, 20], 16, 8, 16
    lens = [a + c for a, c in zip(before, counts)]
    cache, table = make_cache(lens, hkv, page, 9)
    for b, length in enumerate(lens):
        i = np.arange(length)
        ramp = torch.from_numpy(0.1 + 3.0 * i / length).cuda().to(torch.bfloat16)
        at = torch.from_numpy(table[b, i // page].astype(np.int64)).cuda(), torch.from_numpy(i % page).cuda()
        cache.k[at[0], :, at[1]] *= ramp[:, None, None]
    g = torch.Generator(device="cuda").manual_seed(11)
    q = torch.randn(sum(counts), hq, 128, generator=g, device="cuda").to(torch.float32 if qt == "f32" else torch.bfloat16)
    rng = np.random.default_rng(12)
    rows = [S.tree_rows(random_parents(rng, c, "random")) for c in counts]
    m = i32(np.concatenate([S.pack_rows(r, (n + 31) // 32) for r in rows]).view(np.int32))
    qs = tsd.Queries(q, q_indptr=i32([0, n, n + 3]), max_tokens_per_seq=n)
    out, lse = tsd.tree_decode(cache, qs, m, out_dtype=torch.float32)
    check_tree(cache, table, page, q, counts, lens, rows, out, lse, qs.sm_scale or 1 / math.sqrt(128))


@pytest.mark.parametrize("before", [6, 38, 59, 30, 2059])
@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_tree_nonfinite_drafts_anywhere_in_a_tile(what, qt, before):
    """Two drafts whose V rows hold anything, in the first, the second and both halves of a tile, or in two tiles."""
    import torch
    n, hkv, G, page = 9, 2, 3, 4
    cache, table = make_cache([before + n], hkv, page)
    clean, _ = make_cache([before + n], hkv, page)
    for d in (1, 5):
        cache.v[table[0, (before + d) // page], :, (before + d) % page] = what
    q = torch.randn(n, hkv * G, 128, device="cuda").to(torch.float32 if qt == "f32" else torch.bfloat16)
    rows = S.tree_rows([-1, 0, 0, 2, 1, 2, 5, 3, -1])
    m = i32(S.pack_rows(rows, 1).view(np.int32))
    qs = tsd.Queries(q, q_indptr=i32([0, n]), max_tokens_per_seq=n)
    for dt in (torch.float32, torch.bfloat16):
        out, lse = tsd.tree_decode(cache, qs, m, out_dtype=dt)
        ref, rl = tsd.tree_decode(clean, qs, m, out_dtype=dt)
        sees = torch.tensor([bool(r & {1, 5}) for r in rows], device="cuda")
        assert torch.equal(lse, rl)
        assert torch.equal(out[~sees], ref[~sees]) and torch.isfinite(out[~sees]).all()
        assert torch.isnan(out[sees]).all() if what != what else (out[sees] == what).all()


def test_tree_bad_pages_and_sequences():
    import torch
    counts, before, page = [4, 4, 2], [300, 60, 33], 16
    lens = [304, 64, 35]
    cache, table = make_cache(lens, 2, page)
    q = torch.randn(10, 4, 128, device="cuda")
    qs = lambda ip=[0, 4, 8, 10]: tsd.Queries(q, q_indptr=i32(ip), max_tokens_per_seq=4)
    st = i32([0])
    good, gl = tsd.tree_decode(cache, qs(), None, out_dtype=torch.float32)
    cache.page_table[0, 3] = 10 ** 6       # tokens 48 .. 63 drop out
    out, lse = tsd.tree_decode(cache, qs(), None, out_dtype=torch.float32, status=st)
    assert int(st) == tsd.DEV_BAD_PAGE and torch.equal(out[4:], good[4:]) and torch.equal(lse[4:], gl[4:])
    K, V = rows_of(cache, table, 0, 304, page)
    ok = np.r_[0:48, 64:304]
    ref, rl, _ = S.tree_attention(np64(q)[:4, :2], K[0][ok], V[0][ok], 284, S.tree_rows([-1, 0, 1, 2]), 1 / math.sqrt(128))
    assert np.abs(np64(out)[:4, :2] - ref).max() < 2e-5 and np.abs(np64(lse)[:4, :2] - rl).max() < 1e-4
    # a length above the bound, and more drafts than tokens: outputs of those sequences are not written
    cache.page_table[0, 3] = int(table[0, 3])
    st.zero_()
    cache.seq_lens[0], cache.seq_lens[2] = 10 ** 6, 1
    out.fill_(9.0)
    tsd.tree_decode(cache, qs(), None, out=out, status=st)
    assert int(st) == tsd.DEV_BAD_SEQ
    assert (out[:4] == 9).all() and (out[8:] == 9).all() and torch.equal(out[4:8], good[4:8])


def test_tree_tokens_of_no_sequence_are_left_as_they_were():
    import torch
    cache, table = make_cache([40, 30], 2, 16)
    q = torch.randn(12, 4, 128, device="cuda").bfloat16()
    out = torch.full((12, 4, 128), 9.0, device="cuda")
    lse = torch.full((12, 4), 9.0, device="cuda")
    tsd.tree_decode(cache, tsd.Queries(q, q_indptr=i32([2, 6, 9]), max_tokens_per_seq=4), None, out=out, lse=lse)
    for x in (out, lse):
        assert (x[:2] == 9).all() and (x[9:] == 9).all() and (x[2:9] != 9).any()


def test_a_step_without_tokens():
    import torch
    cache, _ = make_cache([40, 30], 2, 16, fill="other")
    before = cache.k.clone()
    ip = i32([0, 0, 0])
    x = torch.zeros(0, 4, 128, device="cuda")
    mask, depth = tsd.tree_mask(i32(np.zeros(0)), ip, 40)
    assert mask.shape == (0, 2) and depth.shape == (0,)
    q = tsd.rope_append(cache, tsd.RotaryEmbedding(), x, x[:, :2], x[:, :2], ip, 40, depth=depth)
    out, lse = tsd.tree_decode(cache, tsd.Queries(q, ip, 40), mask)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    # and one in which a single sequence has some
    ip = i32([0, 0, 3])
    x = torch.randn(3, 4, 128, device="cuda").bfloat16()
    mask, depth = tsd.tree_mask(i32([-1, 0, 1]), ip, 40)
    q = tsd.rope_append(cache, tsd.RotaryEmbedding(), x, x[:, :2], x[:, :2], ip, 40, depth=depth)
    out, lse = tsd.tree_decode(cache, tsd.Queries(q, ip, 40), mask)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all() and not torch.equal(before, cache.k)


def test_a_table_of_lengths_that_is_too_long_is_refused_on_the_host():
    import torch
    cache, _ = make_cache([40, 30], 2, 16)
    q = torch.zeros(6, 4, 128, device="cuda")
    with pytest.raises(ValueError):   # q_indptr of three sequences
        tsd.tree_decode(cache, tsd.Queries(q, q_indptr=i32([0, 2, 4, 6]), max_tokens_per_seq=3))
    with pytest.raises(ValueError):
        tsd.rope_append(cache, tsd.RotaryEmbedding(), q, q[:, :2], q[:, :2], i32([0, 2, 4, 6]), 3)
    with pytest.raises(ValueError):
        tsd.cache_compact(cache, i32([[0], [0]]), i32([0, 2, 4, 6]), 3)


def test_tree_refusals():
    import torch
    cache, _ = make_cache([40, 30], 2, 16)
    q = torch.zeros(6, 4, 128, device="cuda")
    ip = i32([0, 3, 6])
    qs = tsd.Queries(q, q_indptr=ip, max_tokens_per_seq=3)
    for kw in (dict(mask=i32(np.zeros((6, 2)))), dict(mask=torch.zeros(6, 1, device="cuda")), dict(out_dtype=torch.float16),
               dict(out=torch.zeros(6, 4, 64, device="cuda")), dict(lse=torch.zeros(6, 5, device="cuda")),
               dict(mask=torch.zeros(6, 1, dtype=torch.int32))):
        with pytest.raises((ValueError, TypeError)):
            tsd.tree_decode(cache, qs, **kw)
    with pytest.raises(ValueError):
        tsd.tree_decode(cache, tsd.Queries(q.cpu(), q_indptr=ip, max_tokens_per_seq=3))
    with pytest.raises(tsd.TsdError):
        tsd.tree_decode(cache, tsd.Queries(q, q_indptr=ip, max_tokens_per_seq=3, causal=False))
    big = tsd.Queries(torch.zeros(600, 4, 128, device="cuda"), q_indptr=i32([0, 0, 600]), max_tokens_per_seq=600)
    with pytest.raises(tsd.TsdError):
        tsd.tree_decode(cache, big)


# ---------------------------------------------------------------------------------------------------------------------
# Pages
# ---------------------------------------------------------------------------------------------------------------------
class Serving:
    """A pool on the GPU and its model on the CPU, with two layers whose pages carry labels."""

    def __init__(self, batch, page, max_len, pool, hkv=2, n_layers=2, seed=0):
        import torch
        self.rng = np.random.default_rng(seed)
        width = -(-max_len // page)
        self.table, self.lens = i32(np.full((batch, width), -1)), i32(np.zeros(batch))
        self.refs = i32(np.zeros(pool))
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kv = torch.randn(2 * n_layers, pool, hkv, page, 128, generator=g, device="cuda").to(torch.bfloat16)
        self.layers = tsd.LayerCaches([tsd.KVCache(self.kv[2 * i], self.kv[2 * i + 1], self.lens, max_len,
                                                   page_table=self.table) for i in range(n_layers)])
        self.model = S.Pool(self.table.cpu(), [0] * batch, [0] * pool, page, max_len, self.data())

    def data(self):
        return self.kv.transpose(0, 1).float().cpu().numpy()

    def check(self, ws=None):
        assert np.array_equal(self.table.cpu().numpy(), self.model.table)
        assert np.array_equal(self.refs.cpu().numpy(), self.model.refs)
        assert np.array_equal(self.lens.cpu().numpy(), self.model.lens)
        assert np.array_equal(self.data(), self.model.data)
        want = sum({"BAD_SEQ": tsd.DEV_BAD_SEQ, "NO_PAGES": tsd.DEV_NO_PAGES}[f] for f in self.model.flags)
        assert (status() if ws is None else tsd.read_device_status(ws)) == want
        self.model.flags.clear()
        held = self.model.table[self.model.table >= 0]
        assert np.array_equal(np.bincount(held, minlength=len(self.model.refs)), self.model.refs)

    def resize(self, new, **kw):
        tsd.cache_resize(self.layers, self.refs, i32(new), **kw)
        self.model.resize(list(new))
        self.check(kw.get("workspace"))

    def fork(self, src, dst):
        tsd.cache_fork(self.layers, self.refs, i32(src), i32(dst))
        self.model.fork(list(src), list(dst))
        self.check()


@pytest.mark.parametrize("batch,page,max_len,pool", [(1, 1, 9, 12), (3, 4, 40, 20), (17, 16, 300, 200), (5, 64, 500, 129),
                                                     (300, 8, 100, 3000), (1500, 2, 20, 9000)])
def test_pool_random_walk(batch, page, max_len, pool):
    s = Serving(batch, page, max_len, pool, n_layers=1 if batch > 100 else 2, seed=batch)
    ws = tsd.Workspace("cuda")
    for step in range(12):
        lens = s.model.lens
        what = s.rng.random(batch)
        new = np.where(what < 0.5, lens + s.rng.integers(0, max(2, max_len // 6), batch),
                       np.where(what < 0.7, lens, np.where(what < 0.85, lens // 2, 0)))
        new = np.minimum(new, max_len)
        if step % 5 == 4:
            new[s.rng.integers(batch)] = max_len + 1   # refused
        s.resize(new, **({"workspace": ws} if step % 2 else {}))
        n = int(s.rng.integers(0, max(1, batch // 2) + 1))
        s.fork(s.rng.integers(0, batch, n), s.rng.integers(0, batch, n))   # many are refused


def test_a_shared_page_is_copied_once_per_holder():
    s = Serving(5, 8, 64, 40)
    s.resize([21, 0, 0, 0, 0])
    s.fork([0, 0, 0], [1, 2, 4])
    assert s.model.refs.max() == 4
    s.resize([21, 22, 21, 0, 24])       # two of four holders grow
    assert s.model.refs[s.model.table[0, 2]] == 2
    s.resize([25, 22, 25, 0, 24])       # the last two leave it together: it is free
    s.resize([16, 22, 0, 0, 24])
    s.fork([4], [3])                    # a full last page is shared and never copied
    s.resize([16, 22, 0, 25, 24])
    assert s.model.table[3, 2] == s.model.table[4, 2]


def test_resize_exhausts_the_pool_exactly():
    s = Serving(4, 4, 100, 10)
    s.resize([20, 20, 0, 0])
    s.resize([20, 20, 1, 0])            # no page left
    s.resize([20, 16, 1, 0])            # one is released, to be had in the next call
    s.resize([20, 16, 1, 0])
    assert s.model.lens.tolist() == [20, 16, 1, 0]


def test_resize_large_pool_and_long_sequences():
    s = Serving(6, 1, 5000, 20011, hkv=1, n_layers=1)
    s.resize([5000, 1, 4999, 0, 77, 5000])
    s.resize([0, 1, 4999, 5000, 78, 2500])
    s.resize([5000, 5000, 0, 5000, 0, 0])


def test_resize_bad_table_entries():
    s = Serving(2, 4, 40, 12)
    s.resize([17, 9])
    s.table[0, 2] = 99
    s.refs[int(s.table[1, 2])] = 0
    keep = s.refs.clone()
    tsd.cache_resize(s.layers, s.refs, i32([4, 4]))
    assert status() == tsd.DEV_BAD_PAGE
    # page 99 is released by nobody, and a page that is free already stays at 0
    assert s.lens.tolist() == [4, 4] and int(s.refs.min()) == 0 and int((keep - s.refs).sum()) == 4


def compact_case(counts, before, keeps, page, hkv=2, n_layers=2, refs=None, bad=(), seed=0):
    import torch
    lens = [a + n for a, n in zip(before, counts)]
    caches, tables = [], None
    first, table = make_cache(lens, hkv, page, seed, fill="other")
    for i in range(n_layers):
        c, _ = make_cache(lens, hkv, page, seed + i, fill="other")
        k, v = torch.randn_like(c.k), torch.randn_like(c.v)
        caches.append(tsd.KVCache(k, v, first.seq_lens, first.max_seq_len, page_table=first.page_table))
    want = [(c.k.clone(), c.v.clone()) for c in caches]
    width = max(1, max(len(x) for x in keeps))
    keep = i32([list(x) + [-1] * (width - len(x)) for x in keeps])
    ip = i32(np.concatenate([[0], np.cumsum(counts)]))
    out = tsd.cache_compact(caches, keep, ip, max(counts), refs=refs(table) if refs else None)
    new = []
    for b, x in enumerate(keeps):
        if b in bad:
            new.append(lens[b])
            continue
        new.append(before[b] + len(x))
        at = lambda i: (int(table[b, (before[b] + i) // page]), (before[b] + i) % page) if page else (b, before[b] + i)
        for i, r in enumerate(x):
            for (kw, vw), c in zip(want, caches):
                # in the list's order a source is never overwritten before it is read
                (pd, sd), (ps, ss) = at(i), at(r)
                kw[pd, :, sd], vw[pd, :, sd] = kw[ps, :, ss].clone(), vw[ps, :, ss].clone()
    assert out.tolist() == new and first.seq_lens.tolist() == lens
    for (kw, vw), c in zip(want, caches):
        assert torch.equal(c.k, kw) and torch.equal(c.v, vw)


@pytest.mark.parametrize("page", [0, 1, 4, 16, 64])
def test_compact(page):
    rng = np.random.default_rng(page)
    counts = [16, 1, 0, 64, 33, 7, 300]
    before = [100, 0, 5, 3, 17, 15, 40]
    keeps = [sorted(rng.choice(n, rng.integers(0, n + 1), replace=False).tolist()) if n else [] for n in counts]
    keeps[4], keeps[5] = list(range(33)), [1, 2, 3, 4, 5, 6]     # all; every target a later source
    compact_case(counts, before, keeps, page)
    compact_case(counts, before, keeps, page, hkv=3, n_layers=5)


def test_compact_bad_lists_leave_their_sequence():
    compact_case([8, 8, 8, 8, 8], [10] * 5, [[1, 3], [3, 1], [2, 8], [5, 5], [0, -7]], 4, bad=(1, 2, 3, 4))
    assert status() == tsd.DEV_BAD_INDEX
    compact_case([8, 8], [10, 10], [[0, 2], [4, 6]], 4,
                 refs=lambda t: i32(np.bincount(np.r_[t[0, :5], t[1, :5], t[1, 2]], minlength=13)), bad=(1,))
    assert status() == tsd.DEV_SHARED_PAGE


def test_cache_call_refusals():
    import torch
    s = Serving(3, 4, 40, 12)
    cont, _ = make_cache([5, 6, 7], 2, 0, fill="other")
    one = i32([1])
    for call in (lambda: tsd.cache_resize(s.layers, s.refs[:-1], i32([1, 1, 1])),
                 lambda: tsd.cache_resize(s.layers, s.refs, i32([1, 1])),
                 lambda: tsd.cache_resize(s.layers, s.refs.long(), i32([1, 1, 1])),
                 lambda: tsd.cache_resize(cont, s.refs, i32([1, 1, 1])),
                 lambda: tsd.cache_fork(s.layers, s.refs, one, i32([1, 2])),
                 lambda: tsd.cache_fork(s.layers, s.refs, one, torch.ones(1, device="cuda")),
                 lambda: tsd.cache_compact(s.layers, i32([[1], [1]])),
                 lambda: tsd.cache_compact(s.layers, i32([[0], [0], [0]]), refs=s.refs[1:])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(tsd.TsdError):
        tsd.cache_compact(s.layers, i32([[0], [0], [0]]), out_lens=s.lens)
    tsd.cache_fork(s.layers, s.refs, one[:0], one[:0])   # no pairs: nothing happens
    s.check()


# ---------------------------------------------------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------------------------------------------------
def step_setup(seed=0):
    """Three sequences with filled caches, and one drafting step's inputs."""
    import torch
    s = Serving(4, 16, 256, 80, hkv=2, n_layers=2, seed=seed)
    s.resize([100, 37, 0, 0])
    s.fork([0], [3])                                    # sequence 3 goes on from sequence 0
    counts = [6, 9, 0, 5]
    rng = np.random.default_rng(seed)
    par = [random_parents(rng, n, "random") for n in counts]
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda h: [torch.randn(20, h, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    return s, counts, par, i32(sum(par, [])), i32(np.concatenate([[0], np.cumsum(counts)])), mk(8), mk(2), mk(2)


def one_step(s, parents, ip, n_max, q, k, v, keep, grown):
    rope = tsd.RotaryEmbedding(theta=500000.0)
    tsd.cache_resize(s.layers, s.refs, grown)
    mask, depth = tsd.tree_mask(parents, ip, n_max)
    outs = []
    for i, cache in enumerate(s.layers.caches):
        qr = tsd.rope_append(cache, rope, q[i], k[i], v[i], ip, n_max, depth=depth)
        outs.append((qr,) + tsd.tree_decode(cache, tsd.Queries(qr, ip, n_max), mask))
    lens = tsd.cache_compact(s.layers, keep, ip, n_max, refs=s.refs)
    held = s.table.clone(), s.lens.clone()
    tsd.cache_resize(s.layers, s.refs, lens)
    return mask, depth, outs, lens, held


def test_a_speculative_step():
    s, counts, par, parents, ip, q, k, v = step_setup()
    before = s.model.lens.copy()
    keep = i32([[0, 2, -1], [1, 3, 8], [-1, -1, -1], [-1, -1, -1]])
    old = s.data()
    mask, depth, outs, lens, (table, now) = one_step(s, parents, ip, 9, q, k, v, keep, i32(before + np.array(counts)))
    rows = [S.tree_rows(p) for p in par]
    s.model.resize((before + np.array(counts)).tolist())
    assert np.array_equal(table.cpu().numpy(), s.model.table)
    assert s.model.table[0, 6] != s.model.table[3, 6]        # the shared half page was copied
    freq, ms = S.rope_frequencies(128, 500000.0)
    data = s.model.data
    t = 0
    for b, n in enumerate(counts):
        for j in range(n):
            pos = np.array([before[b] + len(rows[b][j]) - 1.0])
            p, slot = s.model.table[b, (before[b] + j) // 16], (before[b] + j) % 16
            for i in range(2):
                ref = S.rope_rotate(np64(k[i])[t + j:t + j + 1], pos, freq, ms, False)[0]
                data[p, 2 * i, :, slot], data[p, 2 * i + 1, :, slot] = ref, np64(v[i])[t + j]
        for i in range(2):
            qr = S.rope_rotate(np64(q[i])[t:t + n], before[b] + np.array([len(r) - 1.0 for r in rows[b]]), freq, ms, False)
            i_all = np.arange(before[b] + n)
            pages, slots = s.model.table[b, i_all // 16].astype(int), i_all % 16
            for g in range(2):
                K, V = data[pages, 2 * i, g, slots], data[pages, 2 * i + 1, g, slots]
                ref, rl, spread = S.tree_attention(qr[:, 4 * g:4 * g + 4], K, V, before[b], rows[b], 1 / math.sqrt(128))
                o, l = np64(outs[i][1])[t:t + n, 4 * g:4 * g + 4], np64(outs[i][2])[t:t + n, 4 * g:4 * g + 4]
                # q and K are rounded to bf16 after the rotation, 2^-8 each: a score moves by 2^-7 sum |q k| scale
                dz = 2.0 ** -7 / math.sqrt(128) * (np.abs(qr[:, 4 * g:4 * g + 4]) @ np.abs(K).T).max(-1, initial=0.0)
                assert (np.abs(o - ref) <= (2 * dz[..., None] + 2.0 ** -7) * spread + 2.0 ** -8 * np.abs(ref)).all()
                assert (np.abs(l - rl) <= dz + 1e-5).all()
        t += n
    assert lens.tolist() == [102, 40, 0, 100]
    s.model.resize(lens.tolist())
    assert np.array_equal(s.table.cpu().numpy(), s.model.table) and np.array_equal(s.refs.cpu().numpy(), s.model.refs)
    assert np.array_equal(s.lens.cpu().numpy(), s.model.lens)
    # the accepted rows lie behind the committed ones, rounded keys of the accepted drafts
    got = s.data()
    for b, kept in ((0, [0, 2]), (1, [1, 3, 8])):
        t0 = int(ip[b])
        for i, r in enumerate(kept):
            p, slot = s.model.table[b, (before[b] + i) // 16], (before[b] + i) % 16
            assert np.array_equal(got[p, 1, :, slot], np64(v[0])[t0 + r])
            assert np.array_equal(got[p, 3, :, slot], np64(v[1])[t0 + r])
    assert status() == 0


def test_steps_captured_and_replayed_and_on_streams():
    """The whole step in two CUDA graphs of different sizes, replayed at once on two streams, and an
    eager step on a third: each gives what an eager step alone gives."""
    import torch
    setups = [step_setup(seed) for seed in (0, 1, 2)]
    keeps = i32([[0, 2, -1], [1, 3, 8], [-1, -1, -1], [-1, -1, -1]])
    eager = []
    for s, counts, par, parents, ip, q, k, v in setups:
        grown = i32(s.model.lens + np.array(counts))
        saved = [x.clone() for x in (s.table, s.lens, s.refs, s.kv)]
        r = one_step(s, parents, ip, 9, q, k, v, keeps, grown)
        torch.cuda.synchronize()
        eager.append(([x.clone() for o in r[2] for x in o], [x.clone() for x in (s.table, s.lens, s.refs, s.kv)], saved, grown))

    def restore(i):
        s = setups[i][0]
        for x, y in zip((s.table, s.lens, s.refs, s.kv), eager[i][2]):
            x.copy_(y)

    graphs, results = [], []
    for i in range(2):
        s, counts, par, parents, ip, q, k, v = setups[i]
        restore(i)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = one_step(s, parents, ip, 9, q, k, v, keeps, eager[i][3])
        graphs.append(g)
        results.append([x for o in r[2] for x in o])
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        for i in range(3):
            restore(i)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        s, counts, par, parents, ip, q, k, v = setups[2]
        with torch.cuda.stream(streams[2]):
            r = one_step(s, parents, ip, 9, q, k, v, keeps, eager[2][3])
        torch.cuda.synchronize()
        for i, got in enumerate(results + [[x for o in r[2] for x in o]]):
            assert all(torch.equal(a, b) for a, b in zip(got, eager[i][0]))
            s = setups[i][0]
            assert all(torch.equal(a, b) for a, b in zip((s.table, s.lens, s.refs, s.kv), eager[i][1]))
    del graphs
    assert status() == 0


def test_a_stream_argument():
    import torch
    st = torch.cuda.Stream()
    s, counts, par, parents, ip, q, k, v = step_setup(3)
    rope = tsd.RotaryEmbedding()
    tsd.cache_resize(s.layers, s.refs, i32(s.model.lens + np.array(counts)))
    mask, depth = tsd.tree_mask(parents, ip, 9)
    c = s.layers.caches[0]
    want = tsd.rope_append(c, rope, q[0], k[0], v[0], ip, 9, depth=depth)
    want = (want,) + tsd.tree_decode(c, tsd.Queries(want, ip, 9), mask)
    torch.cuda.synchronize()
    m2, d2 = tsd.tree_mask(parents, ip, 9, stream=st)
    got = tsd.rope_append(c, rope, q[0], k[0], v[0], ip, 9, depth=d2, stream=st)
    got = (got,) + tsd.tree_decode(c, tsd.Queries(got, ip, 9), m2, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_workspace_shared_with_sparse_decode():
    """tree_decode scribbles over scratch that sparse decode needs zeroed: a Workspace keeps them apart."""
    import torch
    cache, table = make_cache([300, 200], 2, 16)
    q = torch.randn(2, 4, 128, device="cuda").bfloat16()
    qs = tsd.Queries(q)
    ws = tsd.Workspace("cuda")
    ref = tsd.decode_step(cache, qs, 32)[0]
    for _ in range(3):
        assert torch.equal(tsd.decode_step(cache, qs, 32, workspace=ws)[0], ref)
        a = tsd.tree_decode(cache, qs, workspace=ws)[0]
        assert torch.equal(a, tsd.tree_decode(cache, qs)[0])
    assert tsd.read_device_status(ws) == 0
