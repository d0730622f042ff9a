"""tree_decode where units consist mostly of drafts, or where lists see nothing for many tiles, against the formula
in 64 bits (torch, on the GPU).

Tolerances, as for the other tests of tree_decode: a score is a sum of 128 products in fp32, off by
dz <= 130 2^-24 scale sum |q_d k_d| and by 2^-16 2^-8 for the exponent arithmetic; dz in every exponent changes a weighted
mean by at most 2 dz sum p|V|; the weights' rounding is 2^-8 of sum p|V| (bf16 outputs) or 2^-22 (fp32 outputs), and
the output's own is 2^-8 or 2^-23 of the value.
"""

import math

import numpy as np
import pytest

import top_sparse_decode_topk_b200 as tsd
from tests.test_gpu_speculative import i32, status

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_flags_left():
    status()
    yield
    assert status() == 0


def filled(lens, hkv, page, seed, spare=5):
    """A paged cache whose pages lie in random order, with all rows finite; (cache, table)."""
    import torch
    rng = np.random.default_rng(seed)
    need = [-(-x // page) for x in lens]
    order, at = rng.permutation(sum(need) + spare), 0
    table = np.full((len(lens), max(1, max(need))), -1, np.int64)
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda: torch.randn(len(order), hkv, page, 128, generator=g, device="cuda").to(torch.bfloat16)
    return tsd.KVCache(mk(), mk(), i32(lens), max(lens), page_table=i32(table)), table


def expected(cache, row, page, q, t0, n, length, sees, scale, gone=()):
    """One sequence, whose pages are `row`, in 64 bits: out and spread [n, Hq, 128], lse and size [n, Hq].  sees: bool [n, n] (draft, draft);
    gone: positions whose pages cannot be read."""
    import torch
    hkv, hq = cache.num_kv_heads, q.shape[1]
    G, i = hq // hkv, np.arange(length)
    pages, slots = torch.from_numpy(row[i // page]).cuda(), torch.from_numpy(i % page).cuda()
    K, V = (x[pages, :, slots].double().transpose(0, 1) for x in (cache.k, cache.v))   # [Hkv, length, 128]
    see = torch.ones(n, length, dtype=torch.bool, device="cuda")
    see[:, length - n:] = torch.from_numpy(sees).cuda()
    if len(gone):
        see[:, torch.from_numpy(np.asarray(gone)).cuda()] = False
    qq = q[t0:t0 + n].double().view(n, hkv, G, 128)
    z = scale * torch.einsum("nhgd,hld->nhgl", qq, K)
    size = scale * torch.einsum("nhgd,hld->nhgl", qq.abs(), K.abs()).amax(-1)
    z.masked_fill_(~see[:, None, None], -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.where(torch.isneginf(lse)[..., None], 0.0, torch.exp(z - lse[..., None]))
    flat = lambda x: x.reshape(n, hq, *x.shape[3:])
    return tuple(flat(x) for x in (torch.einsum("nhgl,hld->nhgd", p, V), torch.einsum("nhgl,hld->nhgd", p, V.abs()), lse, size))


def compare(got, lse, ref, spread, rl, size, bf16_out):
    import torch
    dz = size * 130 * 2.0 ** -24 + 2.0 ** -24
    w, o = (2.0 ** -8, 2.0 ** -8) if bf16_out else (2.0 ** -22, 2.0 ** -23)
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty) and not got[empty].any()
    over = (got.double() - ref).abs() - ((2 * dz[..., None] + w) * spread + o * ref.abs())
    assert not (over > 0).any() and torch.isfinite(got).all(), over.max()
    gap = (lse.double() - rl).abs() - (dz + 2.0 ** -22 * (4 + rl.abs()))
    assert not (gap[~empty] > 0).any(), gap[~empty].max()


def run(counts, before, hq, hkv, qt, ot, kind, page=16, seed=0, check=None, bad=()):
    """bad: positions (first of a page) whose table entries are out of range, in every sequence."""
    import torch
    rng = np.random.default_rng(seed)
    lens = [a + n for a, n in zip(before, counts)]
    cache, table = filled(lens, hkv, page, seed)
    gone = np.concatenate([np.arange(p, p + page) for p in bad]) if len(bad) else ()
    for p in bad:
        cache.page_table[:, p // page] = 10 ** 8
    n_max, W = max(counts), (max(counts) + 31) // 32
    T = sum(counts)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn(T, hq, 128, generator=g, device="cuda").to(torch.bfloat16 if qt == "bf16" else torch.float32)
    sees = []
    for n in counts:
        if kind == "chain":
            sees.append(np.tril(np.ones((n, n), bool)))
        else:   # any bits: rows that see nothing, rows that see late drafts alone, rows that see some
            m = rng.random((n, n)) < 0.2
            m[rng.random(n) < 0.3] = False
            late = rng.random(n) < 0.3
            m[late, :n * 4 // 5] = False
            sees.append(m)
    mask = None
    if kind != "chain":
        words = np.zeros((T, W * 32), bool)
        t = 0
        for m in sees:
            words[t:t + len(m), :m.shape[1]] = m
            t += len(m)
        mask = i32(np.packbits(words, axis=1, bitorder="little").view(np.int32))
    ip = i32(np.concatenate([[0], np.cumsum(counts)]))
    st = i32([0])
    dt = torch.bfloat16 if ot == "bf16" else torch.float32
    out, lse = tsd.tree_decode(cache, tsd.Queries(q, ip, n_max), mask, out_dtype=dt, status=st)
    assert int(st) == (tsd.DEV_BAD_PAGE if len(bad) else 0)
    t = 0
    for b, n in enumerate(counts):
        if check is None or b in check:
            compare(out[t:t + n], lse[t:t + n], *expected(cache, table[b], page, q, t, n, lens[b], sees[b], 1 / math.sqrt(128), gone),
                    ot == "bf16")
        t += n
    return out, lse


@pytest.mark.parametrize("kind", ["chain", "custom"])
@pytest.mark.parametrize("ot", ["f32", "bf16"])
@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("batch,n,before,hq,hkv", [(16, 300, 0, 32, 8), (64, 500, 0, 8, 8), (2, 300, 17, 64, 8), (64, 500, 40, 32, 8),
                                                   (3, 512, 0, 4, 1), (5, 257, 64, 2, 2)])
def test_many_drafts(batch, n, before, hq, hkv, qt, ot, kind):
    """Segments that start among the drafts and are longer than what is summed in tensor memory."""
    rng = np.random.default_rng(n)
    counts = [n] * batch
    for b in range(1, batch, 3):
        counts[b] = int(rng.integers(130, n + 1))
    run(counts, [before] * batch, hq, hkv, qt, ot, kind, seed=n + before, check=range(0, batch, max(1, batch // 8)))


@pytest.mark.parametrize("kind", ["chain", "custom"])
@pytest.mark.parametrize("qt", ["bf16", "f32"])
def test_a_bad_page_in_each_of_the_first_tiles(qt, kind):
    """Rows behind a unit's last list are masked in every tile with a bad page, while its lists see the other rows."""
    bad = list(range(16, 1600, 32))
    run([3] * 40, [4000] * 40, 8, 2, qt, "f32", kind, seed=3, check=(0, 7, 21, 39), bad=bad)
    run([40] * 24, [2500] * 24, 8, 2, qt, "f32", kind, seed=4, check=(0, 7, 23), bad=bad)


@pytest.mark.parametrize("qt", ["bf16", "f32"])
def test_nothing_but_bad_pages_before_the_drafts(qt):
    """All lists see their first token late."""
    run([70] * 30, [1600] * 30, 8, 2, qt, "f32", "custom", seed=5, check=(0, 11, 29), bad=list(range(0, 1600, 16)))


@pytest.mark.parametrize("qt,ot", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_units_of_one_tile_between_longer_ones(qt, ot):
    """Dozens of units of one tile in a CTA's share, with longer ones among and behind them."""
    rng = np.random.default_rng(8)
    lens = [int(rng.integers(1, 33)) for _ in range(700)]
    for b in (5, 200, 201, 350, 699):
        lens[b] = int(rng.integers(100, 900))
    counts = [min(n, int(rng.integers(1, 4))) for n in lens]
    run(counts, [n - c for n, c in zip(lens, counts)], 16, 8, qt, ot, "custom", seed=9,
        check=list(range(0, 700, 29)) + [5, 200, 201, 202, 350, 699])


@pytest.mark.parametrize("qt,ot", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_a_share_with_not_a_number_alone(qt, ot):
    """The unit is cut where its drafts begin, and in that share a list sees nothing but a key of NaNs: its maximum
    there is -inf as if it saw nothing, its sum is not a number, and neither may get lost in the merge."""
    import torch
    dts = {"bf16": torch.bfloat16, "f32": torch.float32}
    for before in (32, 64, 128, 192, 256, 320):   # a whole number of tiles; shares of two or three
        cache, table = filled([before + 3], 1, 16, before)
        p = int(table[0, before // 16])
        cache.k[p, :, 1] = float("nan")           # draft 1
        q = torch.randn(3, 2, 128, device="cuda").to(dts[qt])
        mask = i32([[1], [2], [5]])               # draft 1 sees itself alone among the drafts; the others do not see it
        out, lse = tsd.tree_decode(cache, tsd.Queries(q, i32([0, 3]), 3), mask, out_dtype=dts[ot])
        assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
        assert torch.isfinite(out[[0, 2]]).all() and torch.isfinite(lse[[0, 2]]).all()
