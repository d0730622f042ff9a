"""Cases, plain forms and calls of the operators of a speculative decoding step over a paged bf16 cache.

rope_append   rotary positions of new queries and keys, and the new K and V rows written into the cache
tree_mask     ancestor bits and depths of trees of drafted tokens, from their parents
tree_decode   attention of drafted tokens over the cache and over their own ancestors
cache_fork    sequences that start as copies of others and share their pages
cache_resize  pages taken (with copy on write of a shared last page) and released
cache_compact accepted drafts moved to the front of a sequence's drafts, in every layer

`own` chooses between the plain forms, elementary torch operations, and the framework's calls.
"""

import math
import random

import numpy as np
import torch

own = False

D = 128   # head dimension of the cache
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one user, eight drafted tokens of a shallow tree: tree bookkeeping and one layer's append, a matter of latency
        dict(name="rope_tree_tiny", op="rope", tree=True, batch=1, hq=8, hkv=2, len_lo=4096, len_hi=4096, n_lo=8,
             n_hi=8, page=16, dtype="bf16", rotary_dim=128, interleaved=False, theta=500000.0, scaling="none",
             fused=True, lens_seed=1),
        # a prefill chunk of eight sequences, yarn-scaled for contexts of 128K: bound by memory
        dict(name="rope_prefill", op="rope", tree=False, batch=8, hq=32, hkv=8, len_lo=4096, len_hi=16384, n_lo=4096,
             n_hi=4096, page=16, dtype="bf16", rotary_dim=128, interleaved=False, theta=1000000.0, scaling="yarn",
             fused=True, lens_seed=2),
        # a ragged batch of trees, fp32 activations, interleaved pairs over half of the head, far positions
        dict(name="rope_tree_ragged", op="rope", tree=True, batch=37, hq=28, hkv=4, len_lo=100, len_hi=131072, n_lo=1,
             n_hi=61, page=32, dtype="f32", rotary_dim=64, interleaved=True, theta=10000.0, scaling="banded",
             fused=False, lens_seed=3),
        # one user verifying eight drafts over 4K tokens: latency
        dict(name="tree_tiny", op="tree", batch=1, hq=8, hkv=2, len_lo=4096, len_hi=4096, n_lo=8, n_hi=8, page=16,
             dtype="bf16", out="bf16", mask="tree", lens_seed=4),
        # eight users, sixteen drafts each, 32K contexts: bound by the cache's bytes
        dict(name="tree_32k", op="tree", batch=8, hq=32, hkv=8, len_lo=32768, len_hi=32768, n_lo=16, n_hi=16, page=16,
             dtype="bf16", out="bf16", mask="tree", lens_seed=5),
        # four users, thirty-two drafts each, 128K contexts, eight query heads per kv head: bytes and products balance
        dict(name="tree_128k", op="tree", batch=4, hq=64, hkv=8, len_lo=131072, len_hi=131072, n_lo=32, n_hi=32,
             page=16, dtype="bf16", out="bf16", mask="tree", lens_seed=6),
        # a ragged batch with custom masks (rows that see nothing among them), fp32 queries and outputs, seven heads a group
        dict(name="tree_ragged", op="tree", batch=13, hq=28, hkv=4, len_lo=1, len_hi=20011, n_lo=1, n_hi=33, page=32,
             dtype="f32", out="f32", mask="custom", lens_seed=7),
        # accepted drafts of eight users kept in one layer's cache
        dict(name="compact_one_layer", op="compact", batch=8, hkv=8, layers=1, len_lo=1000, len_hi=2000, n_lo=16,
             n_hi=16, page=16, lens_seed=8),
        # accepted drafts of a full batch kept in all layers at once
        dict(name="compact_all_layers", op="compact", batch=64, hkv=8, layers=16, len_lo=10, len_hi=100, n_lo=40,
             n_hi=64, page=16, lens_seed=9),
        # one prompt answered four ways: fork, then room for the next tokens
        dict(name="branch_one_prompt", op="branch", parents=1, ways=4, hkv=8, layers=1, len_lo=3001, len_hi=3001,
             grow=8, page=16, spare=64, lens_seed=10),
        # sixty-four prompts, four ways each, every layer's half-filled page copied
        dict(name="branch_batch", op="branch", parents=64, ways=4, hkv=8, layers=16, len_lo=100, len_hi=250, grow=20,
             page=16, spare=500, lens_seed=11),
        # a serving loop's turn: some sequences grow, some shrink to what was accepted, some end, over a large pool
        dict(name="resize_batch", op="resize", batch=256, hkv=1, len_lo=0, len_hi=8000, page=16, spare=70000,
             lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "tree", "compact", "branch", "resize"])
    page = rng.choice([1, 2, 4, 8, 16, 16, 32, 64])
    c = dict(op=op, page=page, lens_seed=rng.randrange(1 << 30))
    if op == "rope":
        hkv = rng.choice([1, 2, 3, 4, 8])
        tree = rng.random() < 0.5
        batch = _log_int(rng, 1, 64)
        n_hi = _log_int(rng, 1, 128 if tree else 4096)
        n_hi = max(1, min(n_hi, 32768 // batch))
        c.update(tree=tree, batch=batch, hkv=hkv, hq=hkv * rng.choice([1, 2, 4, 5, 7]), n_lo=rng.randint(1, n_hi),
                 n_hi=n_hi, len_lo=n_hi, len_hi=n_hi + _log_int(rng, 1, 131072 // batch + 1),
                 dtype=rng.choice(["bf16", "f32"]), rotary_dim=rng.choice([128, 128, 64, 32, 96, 2, 50]),
                 interleaved=rng.random() < 0.5, theta=rng.choice([10000.0, 500000.0, 1000000.0]),
                 scaling=rng.choice(["none", "linear", "ntk", "banded", "yarn"]), fused=rng.random() < 0.5)
    elif op == "tree":
        hkv = rng.choice([1, 2, 3, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
        batch = _log_int(rng, 1, 32)
        n_hi = _log_int(rng, 1, 128)
        len_hi = _log_int(rng, 1, max(2, min(131072, 500_000_000 // (batch * hq * n_hi), 500_000 // batch)))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        c.update(batch=batch, hkv=hkv, hq=hq, n_lo=rng.randint(1, n_hi), n_hi=n_hi, len_lo=rng.randint(1, len_hi),
                 len_hi=len_hi, dtype=dtype, out=rng.choice(["bf16", "f32"]),
                 mask=rng.choice(["tree", "tree", "custom", "chain"]))
    elif op == "compact":
        n_hi = _log_int(rng, 1, 128)
        c.update(batch=_log_int(rng, 1, 64), hkv=rng.choice([1, 2, 3, 8]), layers=_log_int(rng, 1, 16), n_lo=rng.randint(1, n_hi),
                 n_hi=n_hi, len_lo=1, len_hi=_log_int(rng, 2, 200))
    elif op == "branch":
        len_hi = _log_int(rng, 1, 250)
        c.update(parents=_log_int(rng, 1, 64), ways=rng.randint(2, 4), hkv=rng.choice([1, 2, 4, 8]),
                 layers=_log_int(rng, 1, 12), len_lo=rng.randint(1, len_hi), len_hi=len_hi, grow=rng.randint(1, 20),
                 spare=rng.randint(0, 500))
    else:
        len_hi = _log_int(rng, 16, 8000)
        c.update(batch=_log_int(rng, 1, 256), hkv=1, len_lo=0, len_hi=len_hi, spare=rng.randint(0, 70000))
    return c


def _lengths(case):
    """Tokens in the cache before the drafts, and drafts, of every sequence: the case's own, whatever the seed."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "branch":
        return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["parents"])], None
    total = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    if case["op"] == "resize":
        # a third grows a little, a third gives back its rejected tail, some end, some stay
        new = [r.choice([t + r.randint(1, 64), max(0, t - r.randint(1, 64)), t, 0 if r.random() < 0.3 else t + 1]) for t in total]
        return total, new
    n = [r.randint(case["n_lo"], case["n_hi"]) for _ in total]
    if case["op"] == "tree":
        total = [max(t, k) for t, k in zip(total, n)]   # a sequence may consist of its drafts alone
    else:
        total = [t + k for t, k in zip(total, n)]
    return [t - k for t, k in zip(total, n)], n


def _parents(r, n, kind):
    """Parents of n drafts, root's children at -1; most drafts extend a recent one."""
    return [-1 if i == 0 or r.random() < 0.15 else r.randint(max(0, i - 6), i - 1) for i in range(n)] if kind != "chain" \
        else list(range(-1, n - 1))


def _mask_rows(case, n, b):
    """Visible drafts of each draft of sequence b, as sets."""
    r = random.Random(case["lens_seed"] * 1009 + b)
    if case.get("mask") == "custom":
        return [{i for i in range(n) if r.random() < 0.3} if r.random() < 0.9 else set() for _ in range(n)]
    rows = []
    for j, p in enumerate(_parents(r, n, case.get("mask", "tree"))):
        rows.append({j} | (rows[p] if p >= 0 else set()))
    return rows


def _keep(case, n, b):
    """Accepted drafts: a run of the first ones, then some from behind the places that they are moved to, so that a
    second pass over the same cache moves the same rows."""
    r = random.Random(case["lens_seed"] * 1013 + b)
    cnt = r.randint(0, max(1, n // 4))
    run = r.randint(0, cnt)
    return list(range(run)) + sorted(r.sample(range(cnt, n), min(cnt - run, n - cnt)))[: cnt - run]


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages_of(length, page):
    return (length + page - 1) // page


def _table(lens, page, seed, spare=3, width=None):
    """A shuffled page table [batch, width], -1 behind a sequence's pages, and the number of pages of the pool."""
    need = [_pages_of(t, page) for t in lens]
    width = width or max(1, max(need))
    pool = sum(need) + spare
    order = np.random.default_rng(seed * 31 + 5).permutation(pool)
    table, at = np.full((len(lens), width), -1, np.int32), 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, pool


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    return {"rope": _prepare_rope, "tree": _prepare_tree, "compact": _prepare_compact, "branch": _prepare_branch,
            "resize": _prepare_resize}[case["op"]](case, seed, g, s)


def _prepare_drafts(case, seed, s):
    base, n = _lengths(case)
    total = [x + y for x, y in zip(base, n)]
    table, pool = _table(total, case["page"], seed)
    s.update(table=torch.from_numpy(table).cuda(), lens=_i32(total), indptr=_i32(np.concatenate([[0], np.cumsum(n)])),
             max_n=max(n), max_len=max(total), tokens=sum(n))
    return base, n, total, table, pool


def _prepare_rope(case, seed, g, s):
    base, n, total, table, pool = _prepare_drafts(case, seed, s)
    T, hq, hkv, dt = s["tokens"], case["hq"], case["hkv"], DTYPES[case["dtype"]]
    if case["fused"]:   # the three are slices of one projection's output
        qkv = torch.randn(T, (hq + 2 * hkv) * D, generator=g, device="cuda").to(dt).view(T, hq + 2 * hkv, D)
        s.update(q=qkv[:, :hq], k_new=qkv[:, hq:hq + hkv], v_new=qkv[:, hq + hkv:])
    else:
        s.update(q=torch.randn(T, hq, D, generator=g, device="cuda").to(dt),
                 k_new=torch.randn(T, hkv, D, generator=g, device="cuda").to(dt),
                 v_new=torch.randn(T, hkv, D, generator=g, device="cuda").to(dt))
    s["k"] = torch.zeros(pool, hkv, case["page"], D, dtype=torch.bfloat16, device="cuda")
    s["v"] = torch.zeros_like(s["k"])
    if case["tree"]:
        rs = [random.Random(seed * 65537 + b) for b in range(len(n))]
        s["parents"] = _i32([p for r, k in zip(rs, n) for p in _parents(r, k, "tree")])
    freq, s["mscale"] = _frequencies(case)
    s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
    return s


# A scaled case's constants: contexts of 128K over 32K trained positions
SCALE = dict(factor=4.0, original_max_len=32768, low_freq_factor=1.0, high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0)


def _frequencies(case):
    """Angle per position of each pair, in 64 bits, and the factor on cosines and sines."""
    R, theta, f = case["rotary_dim"], case["theta"], SCALE["factor"]
    L, kind = SCALE["original_max_len"], case["scaling"]
    if kind == "ntk" and R > 2:
        theta *= f ** (R / (R - 2))
    w = np.float64(theta) ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    if kind == "linear":
        w = w / f
    elif kind == "banded":
        turns = L * w / (2 * math.pi)
        t = (turns - SCALE["low_freq_factor"]) / (SCALE["high_freq_factor"] - SCALE["low_freq_factor"])
        t = np.clip(t, 0, 1)
        w = (1 - t) * w / f + t * w
    elif kind == "yarn":
        dim = lambda turns: R * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(dim(SCALE["beta_fast"])), 0), min(math.ceil(dim(SCALE["beta_slow"])), R - 1)
        t = np.clip((np.arange(R // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        w = w / f * t + w * (1 - t)
        return w, 0.1 * math.log(f) + 1
    return w, 1.0


def _prepare_tree(case, seed, g, s):
    base, n, total, table, pool = _prepare_drafts(case, seed, s)
    T, hq, hkv, page = s["tokens"], case["hq"], case["hkv"], case["page"]
    s["q"] = (1.5 * torch.randn(T, hq, D, generator=g, device="cuda")).to(DTYPES[case["dtype"]])
    s["k"] = torch.randn(pool, hkv, page, D, generator=g, device="cuda", dtype=torch.bfloat16)
    s["v"] = torch.randn(pool, hkv, page, D, generator=g, device="cuda", dtype=torch.bfloat16)
    # a sink: every sequence's first key lies along its queries
    at = 0
    for b, k in enumerate(n):
        qm = s["q"][at:at + k].float().view(k, hkv, hq // hkv, D).mean((0, 2))
        s["k"][table[b, 0], :, 0] = (6 * math.sqrt(D) * qm / qm.norm(dim=-1, keepdim=True) ** 2).to(torch.bfloat16)
        at += k
    # slots that hold no token: whatever an earlier owner left, not-a-numbers among it
    free = torch.ones(pool * page, dtype=torch.bool, device="cuda")
    for b, t in enumerate(total):
        i = np.arange(t)
        free[torch.from_numpy(table[b, i // page].astype(np.int64) * page + i % page).cuda()] = False
    for x in (s["k"], s["v"]):
        x.masked_fill_(free.view(pool, 1, page, 1), float("nan"))
    W = (s["max_n"] + 31) // 32
    words = np.zeros((T, W), np.uint32)
    at = 0
    for b, k in enumerate(n):
        for j, row in enumerate(_mask_rows(case, k, b)):
            for i in row:
                words[at + j, i >> 5] |= np.uint32(1 << (i & 31))
        at += k
    s["mask"] = torch.from_numpy(words.view(np.int32)).cuda()
    return s


def _prepare_compact(case, seed, g, s):
    base, n, total, table, pool = _prepare_drafts(case, seed, s)
    shape = (case["layers"], pool, case["hkv"], case["page"], D)
    s["k"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    s["v"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    keep = [_keep(case, k, b) for b, k in enumerate(n)]
    width = max(1, max(len(x) for x in keep))
    s["keep"] = _i32([x + [-1] * (width - len(x)) for x in keep])
    return s


def _prepare_pool(case, s, lens, table, pool, width):
    """Table, reference counts and lengths in one buffer, and what they are at the start of every pass."""
    refs = np.zeros(pool, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    flat = np.concatenate([table.reshape(-1), refs, np.asarray(lens, np.int32)])
    s["start"] = torch.from_numpy(flat).cuda()
    s["now"] = s["start"].clone()
    B = len(lens)
    s["table"] = s["now"][:B * width].view(B, width)
    s["refs"] = s["now"][B * width:B * width + pool]
    s["lens"] = s["now"][B * width + pool:]


def _prepare_branch(case, seed, g, s):
    lens, _ = _lengths(case)
    P, ways, page = case["parents"], case["ways"], case["page"]
    s["max_len"] = max(lens) + case["grow"]
    width = _pages_of(s["max_len"], page)
    room = P * ways * (2 + _pages_of(case["grow"], page)) + case["spare"]
    lens = lens + [0] * (P * (ways - 1))
    table, pool = _table(lens, page, seed, spare=room, width=width)
    _prepare_pool(case, s, lens, table, pool, width)
    shape = (case["layers"], pool, case["hkv"], page, D)
    s["k"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    s["v"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    s["src"] = _i32([p for p in range(P) for _ in range(ways - 1)])
    s["dst"] = _i32(list(range(P, P * ways)))
    s["new_lens"] = _i32([lens[p] + case["grow"] for p in list(range(P)) + [p for p in range(P) for _ in range(ways - 1)]])
    return s


def _prepare_resize(case, seed, g, s):
    lens, new = _lengths(case)
    s["max_len"] = max(1, max(lens + new))
    width = _pages_of(s["max_len"], case["page"])
    room = sum(max(0, _pages_of(b, case["page"]) - _pages_of(a, case["page"])) for a, b in zip(lens, new))
    table, pool = _table(lens, case["page"], seed, spare=room + case["spare"] + 1, width=width)
    _prepare_pool(case, s, lens, table, pool, width)
    s["k"] = torch.zeros(1, pool, case["hkv"], case["page"], D, dtype=torch.bfloat16, device="cuda")
    s["v"] = torch.zeros_like(s["k"])
    s["new_lens"] = _i32(new)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------------
def run(s):
    return {"rope": _run_rope, "tree": _run_tree, "compact": _run_compact, "branch": _run_branch,
            "resize": _run_resize}[s["case"]["op"]](s)


def _caches(tsd, s):
    """The program's cache descriptors, made once."""
    if "caches" not in s:
        layers = [(s["k"], s["v"])] if s["k"].dim() == 4 else list(zip(s["k"], s["v"]))
        s["caches"] = tsd.LayerCaches(tsd.KVCache(k, v, s["lens"], s["max_len"], page_table=s["table"]) for k, v in layers)
    return s["caches"]


def _token_places(s):
    """Sequence, index among the sequence's new tokens, and position in the cache of every new token."""
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(s["indptr"][1:].long(), t, right=True)
    j = t - s["indptr"].long()[b]
    n = (s["indptr"][1:] - s["indptr"][:-1]).long()
    return b, j, s["lens"].long()[b] - n[b] + j, n


def _run_rope(s):
    c = s["case"]
    if own:
        import top_sparse_decode_topk_b200 as tsd
        if "rope" not in s:
            kw = {} if c["scaling"] == "none" else dict(scaling=c["scaling"], **SCALE)
            s["rope"] = tsd.RotaryEmbedding(rotary_dim=c["rotary_dim"], theta=c["theta"], interleaved=c["interleaved"], **kw)
        cache = _caches(tsd, s).caches[0]
        mask = depth = None
        if c["tree"]:
            mask, depth = tsd.tree_mask(s["parents"], s["indptr"], s["max_n"])
        q = tsd.rope_append(cache, s["rope"], s["q"], s["k_new"], s["v_new"], q_indptr=s["indptr"],
                            max_tokens_per_seq=s["max_n"], depth=depth)
        return [q, s["k"], s["v"]] + ([mask, depth] if c["tree"] else [])
    b, j, row, n = _token_places(s)
    pos, more = row, []
    if c["tree"]:
        mask, depth = _plain_tree_mask(s, b, j)
        pos, more = row - j + depth.long(), [mask, depth]
    angle = pos.double()[:, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["mscale"]).float()[:, None], (torch.sin(angle) * s["mscale"]).float()[:, None]
    page, slot = s["table"][b, row // c["page"]].long(), row % c["page"]
    s["k"][page, :, slot] = _plain_rotate(s["k_new"], cos, sin, c).to(torch.bfloat16)
    s["v"][page, :, slot] = s["v_new"].to(torch.bfloat16)
    return [_plain_rotate(s["q"], cos, sin, c).to(s["q"].dtype), s["k"], s["v"]] + more


def _plain_rotate(x, cos, sin, c):
    R = c["rotary_dim"]
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((rot, x[..., R:]), -1)


def _plain_tree_mask(s, b, j):
    B, N = s["lens"].numel(), s["max_n"]
    W = (N + 31) // 32
    reach = torch.eye(N, device="cuda").repeat(B, 1, 1)
    p = s["parents"].long()
    reach[b, j, p.clamp(min=0)] += (p >= 0).float()
    step = 1
    while step < N:   # paths of up to `step` edges, doubled
        reach = (reach @ reach > 0).float()
        step *= 2
    rows = reach[b, j]                                   # [T, N]
    depth = (rows.sum(-1) - 1).to(torch.int32)
    bits = torch.nn.functional.pad(rows, (0, 32 * W - N)).view(-1, W, 32).long() << torch.arange(32, device="cuda")
    return bits.sum(-1).to(torch.int32), depth


def _run_tree(s):
    c = s["case"]
    if own:
        import top_sparse_decode_topk_b200 as tsd
        if "queries" not in s:
            s["queries"] = tsd.Queries(s["q"], q_indptr=s["indptr"], max_tokens_per_seq=s["max_n"])
        return list(tsd.tree_decode(_caches(tsd, s).caches[0], s["queries"], None if c["mask"] == "chain" else s["mask"],
                                    out_dtype=DTYPES[c["out"]]))
    page, hkv, hq = c["page"], c["hkv"], c["hq"]
    B, N, L, G = s["lens"].numel(), s["max_n"], s["max_len"], hq // hkv
    b, j, _, n = _token_places(s)
    lens = s["lens"].long()
    base = lens - n
    pos = torch.arange(L, device="cuda")
    inside = pos < lens[:, None]                                                          # [B, L]
    rows = s["table"][:, pos // page].long().clamp(min=0), (pos % page).expand(B, L)
    hole = ~inside[:, :, None, None]
    k = s["k"][rows[0], :, rows[1]].float().masked_fill(hole, 0).permute(0, 2, 3, 1)      # [B, Hkv, D, L]
    v = s["v"][rows[0], :, rows[1]].float().masked_fill(hole, 0).permute(0, 2, 1, 3)      # [B, Hkv, L, D]
    q = torch.zeros(B, N, hq, D, device="cuda")
    q[b, j] = s["q"].float()
    q = q.view(B, N, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, N * G, D)
    words = torch.zeros(B, N, s["mask"].shape[1], dtype=torch.int64, device="cuda")
    words[b, j] = s["mask"].long()
    i = (pos - base[:, None]).clamp(min=0, max=32 * words.shape[2] - 1)                   # [B, L]: draft index
    bit = torch.gather(words, 2, (i >> 5)[:, None].expand(B, N, L)) >> (i & 31)[:, None] & 1
    seen = inside[:, None] & ((pos < base[:, None])[:, None] | (bit == 1))                # [B, N, L]
    seen = seen[:, None, :, None].expand(B, hkv, N, G, L).reshape(B, hkv, N * G, L)
    z = (q @ k).mul_(1.0 / math.sqrt(D)).masked_fill_(~seen, float("-inf"))
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).squeeze(-1)
    out = out.view(B, hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, hq, D)[b, j]
    lse = lse.view(B, hkv, N, G).permute(0, 2, 1, 3).reshape(B, N, hq)[b, j]
    return [out.to(DTYPES[c["out"]]), lse]


def _run_compact(s):
    c = s["case"]
    if own:
        import top_sparse_decode_topk_b200 as tsd
        lens = tsd.cache_compact(_caches(tsd, s), s["keep"], q_indptr=s["indptr"], max_tokens_per_seq=s["max_n"])
        return [s["k"], s["v"], lens]
    page, keep = c["page"], s["keep"].long()
    B, M = keep.shape
    n = (s["indptr"][1:] - s["indptr"][:-1]).long()
    base = s["lens"].long() - n
    i = torch.arange(M, device="cuda").expand(B, M)
    used = keep >= 0
    dst = base[:, None] + torch.minimum(i, n[:, None] - 1)          # an unused entry writes a row of its own sequence
    src = torch.where(used, base[:, None] + keep, dst)              # back to itself
    at = lambda r: (torch.gather(s["table"].long(), 1, r // page), r % page)
    (ps, ss), (pd, sd) = at(src), at(dst)
    for x in (s["k"], s["v"]):
        x[:, pd, :, sd] = x[:, ps, :, ss]
    return [s["k"], s["v"], (base + used.sum(-1)).to(torch.int32)]


def _run_branch(s):
    s["now"].copy_(s["start"])   # the same branching again on every pass
    if own:
        import top_sparse_decode_topk_b200 as tsd
        caches = _caches(tsd, s)
        tsd.cache_fork(caches, s["refs"], s["src"], s["dst"])
        tsd.cache_resize(caches, s["refs"], s["new_lens"])
    else:
        src, dst, page = s["src"].long(), s["dst"].long(), s["case"]["page"]
        pages = (s["lens"][src] + page - 1) // page
        rows = torch.where(torch.arange(s["table"].shape[1], device="cuda") < pages[:, None], s["table"][src], -1)
        s["table"][dst] = rows
        s["lens"][dst] = s["lens"][src]
        s["refs"].scatter_add_(0, rows.clamp(min=0).long().flatten(), (rows >= 0).to(torch.int32).flatten())
        _plain_resize(s)
    return [s["k"], s["v"], s["table"], s["refs"], s["lens"]]


def _run_resize(s):
    s["now"].copy_(s["start"])
    if own:
        import top_sparse_decode_topk_b200 as tsd
        tsd.cache_resize(_caches(tsd, s), s["refs"], s["new_lens"])
    else:
        _plain_resize(s)
    return [s["table"], s["refs"], s["lens"]]


def _plain_resize(s):
    page, table, refs, lens, new = s["case"]["page"], s["table"], s["refs"], s["lens"], s["new_lens"]
    P = refs.numel()
    have, want = ((lens + page - 1) // page)[:, None], ((new + page - 1) // page)[:, None]
    at = torch.arange(table.shape[1], device="cuda")
    held = table.clamp(min=0).long()
    shared = (refs[held] > 1) & (at == have - 1) & (lens % page != 0)[:, None] & (new > lens)[:, None]
    take = shared | ((at >= have) & (at < want))
    drop = (at >= want) & (at < have)
    # free pages, the lowest first; the sequences are served in order while pages last
    order = torch.argsort((refs != 0).to(torch.int32), stable=True)
    ends = take.sum(-1).cumsum(0)
    served = (ends <= (refs == 0).sum()) | (take.sum(-1) == 0)
    take, shared, drop = take & served[:, None], shared & served[:, None], drop & served[:, None]
    rank = take.flatten().cumsum(0).view_as(take) - 1
    fresh = order[rank.clamp(min=0, max=P - 1)]
    # the shared last pages are copied; a sequence without one copies a page in use onto itself
    last = (have - 1).clamp(min=0).long()
    cow = torch.gather(shared, 1, last).squeeze(1)
    old = torch.where(lens > 0, torch.gather(held, 1, last).squeeze(1), refs.argmax())
    to = torch.where(cow, torch.gather(fresh, 1, last).squeeze(1), old)
    if s["case"]["op"] == "branch":
        for x in (s["k"], s["v"]):
            x[:, to] = x[:, old]
    gone = shared | drop
    refs.scatter_add_(0, held.flatten(), -gone.to(torch.int32).flatten())
    refs.scatter_add_(0, fresh.flatten(), take.to(torch.int32).flatten())
    table.copy_(torch.where(take, fresh.to(torch.int32), torch.where(drop, -1, table)))
    lens.copy_(torch.where(served, new, lens))


# ---------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    base, n = _lengths(case)
    if case["op"] == "rope":
        e, T = (2 if case["dtype"] == "bf16" else 4), sum(n)
        byts = T * D * (2 * case["hq"] * e + case["hkv"] * (2 * e + 4)) + 4 * (2 * T + 3 * len(n))
        if case["tree"]:
            byts += 4 * T * (2 + (max(n) + 31) // 32)
        return {"bytes": byts, "flops": 3 * T * (case["hq"] + case["hkv"]) * case["rotary_dim"]}
    if case["op"] == "tree":
        T, e, o = sum(n), (2 if case["dtype"] == "bf16" else 4), (2 if case["out"] == "bf16" else 4)
        rows = sum(x + y for x, y in zip(base, n)) * case["hkv"]
        pairs = sum(x * y + sum(len(r) for r in _mask_rows(case, y, b)) for b, (x, y) in enumerate(zip(base, n)))
        byts = 4 * D * rows + T * case["hq"] * (D * (e + o) + 4) + 4 * T * ((max(n) + 31) // 32) \
            + 4 * sum(_pages_of(x + y, case["page"]) for x, y in zip(base, n))
        return {"bytes": byts, "flops": 4 * D * pairs * case["hq"]}
    if case["op"] == "compact":
        keep = [_keep(case, k, b) for b, k in enumerate(n)]
        moved = sum(1 for x in keep for i, r in enumerate(x) if i != r)
        return {"bytes": moved * case["hkv"] * case["layers"] * 2 * 4 * D + 4 * sum(map(len, keep)) + 12 * len(n), "flops": 0}
    page = case["page"]
    if case["op"] == "branch":
        lens = base * case["ways"]
        new = [x + case["grow"] for x in lens]
        pool = sum(_pages_of(x, page) for x in base) + case["parents"] * case["ways"] * (2 + _pages_of(case["grow"], page)) + case["spare"]
        copied = sum(page for x in lens if x % page) * case["hkv"] * case["layers"] * 2 * 4 * D
        shared = sum(_pages_of(x, page) for x in lens[case["parents"]:])
        return {"bytes": copied + 8 * shared + 4 * pool + 4 * len(lens) * 3, "flops": 0}
    lens, new = base, n
    touched = sum(abs(_pages_of(a, page) - _pages_of(b, page)) for a, b in zip(lens, new))
    room = sum(max(0, _pages_of(b, page) - _pages_of(a, page)) for a, b in zip(lens, new))
    pool = sum(_pages_of(x, page) for x in lens) + room + case["spare"] + 1
    return {"bytes": 4 * pool + 12 * touched + 12 * len(lens), "flops": 0}


# ---------------------------------------------------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "compact": _exact_compact, "branch": _exact_pool,
            "resize": _exact_pool}[case["op"]](case, s)


def _exact_rope(case, s):
    if s["tokens"] * (case["hq"] + 2 * case["hkv"]) > 4_000_000:
        return None
    R, page = case["rotary_dim"], case["page"]
    indptr, lens, table = s["indptr"].tolist(), s["lens"].tolist(), s["table"].cpu().numpy()
    parents = s["parents"].tolist() if case["tree"] else None
    W = (s["max_n"] + 31) // 32
    words, depth, pos, place = [], [], [], []
    for b, length in enumerate(lens):
        t0, n = indptr[b], indptr[b + 1] - indptr[b]
        for j in range(n):
            row, at = [], j
            while case["tree"] and at >= 0:
                row.append(at)
                at = parents[t0 + at]
            w = [sum(1 << (i & 31) for i in row if i >> 5 == u) for u in range(W)]
            words.append([x - (1 << 32) if x >= 1 << 31 else x for x in w])
            depth.append(len(row) - 1)
            pos.append(length - n + (depth[-1] if case["tree"] else j))
            r = length - n + j
            place.append((int(table[b, r // page]), r % page))
    # rotation as a product of complex numbers
    turn = torch.polar(torch.full((1,), s["mscale"], dtype=torch.float64, device="cuda"),
                       torch.tensor(pos, dtype=torch.float64, device="cuda")[:, None] * s["freq"])[:, None]
    halves = (lambda x: (x[..., 0:R:2], x[..., 1:R:2])) if case["interleaved"] else (lambda x: (x[..., :R // 2], x[..., R // 2:R]))

    def rotated(x):
        x = x.double()
        z = torch.complex(*halves(x)) * turn
        y = x.clone()
        for part, value in zip(halves(y), (z.real, z.imag)):
            part.copy_(value)
        return y

    k, v = s["k"].double(), s["v"].double()
    p, o = (torch.tensor(x, device="cuda") for x in zip(*place))
    k[p, :, o], v[p, :, o] = rotated(s["k_new"]), s["v_new"].double()
    return [rotated(s["q"]), k, v] + ([_i32(words), _i32(depth)] if case["tree"] else [])


def _exact_tree(case, s):
    base, n = _lengths(case)
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    out = torch.zeros(s["tokens"], hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], hq), float("-inf"), dtype=torch.float64, device="cuda")
    t = 0
    for b, (c, m) in enumerate(zip(base, n)):
        i = torch.arange(c + m, device="cuda")
        pages = s["table"][b].long()[i // page]
        k, v = (x[pages, :, i % page].double().transpose(0, 1) for x in (s["k"], s["v"]))   # [Hkv, len, D]
        for row in _mask_rows(case, m, b):
            q = s["q"][t].double().view(hkv, hq // hkv, D)
            d = torch.tensor(sorted(row), dtype=torch.long, device="cuda") + c
            z = torch.cat((q @ k[:, :c].transpose(1, 2), q @ k[:, d].transpose(1, 2)), -1) / math.sqrt(D)
            if z.shape[-1]:
                l = torch.logsumexp(z, -1, keepdim=True)
                p = torch.exp(z - l)
                out[t] = (p[..., :c] @ v[:, :c] + p[..., c:] @ v[:, d]).view(hq, D)
                lse[t] = l.view(hq)
            t += 1
    return [out, lse]


def _exact_compact(case, s):
    base, n = _lengths(case)
    page, table = case["page"], s["table"].cpu().numpy()
    src, dst, lens = [], [], []
    for b, m in enumerate(n):
        keep = _keep(case, m, b)
        lens.append(base[b] + len(keep))
        for i, r in enumerate(keep):
            src.append((int(table[b, (base[b] + r) // page]), (base[b] + r) % page))
            dst.append((int(table[b, (base[b] + i) // page]), (base[b] + i) % page))
    k, v = s["k"].double(), s["v"].double()
    if src:
        (ps, ss), (pd, sd) = ([torch.tensor(x, device="cuda") for x in zip(*y)] for y in (src, dst))
        k[:, pd, :, sd], v[:, pd, :, sd] = s["k"].double()[:, ps, :, ss], s["v"].double()[:, ps, :, ss]
    return [k, v, _i32(lens)]


def _exact_pool(case, s):
    page = case["page"]
    table, refs, lens = (s[x].cpu().numpy().copy() for x in ("table", "refs", "lens"))
    k, v = s["k"].double(), s["v"].double()
    if case["op"] == "branch":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            lens[b] = lens[a]
            for i in range(_pages_of(int(lens[a]), page)):
                table[b, i] = table[a, i]
                refs[table[a, i]] += 1
    before, free = refs.copy(), iter(np.flatnonzero(refs == 0).tolist())
    for b, want in enumerate(s["new_lens"].tolist()):
        have, need = _pages_of(int(lens[b]), page), _pages_of(want, page)
        if want > lens[b] and lens[b] % page and before[table[b, have - 1]] > 1:
            old, new = int(table[b, have - 1]), next(free)
            k[:, new], v[:, new] = k[:, old], v[:, old]
            refs[old] -= 1
            refs[new] = 1
            table[b, have - 1] = new
        for i in range(have, need):
            table[b, i] = next(free)
            refs[table[b, i]] = 1
        for i in range(need, have):
            refs[table[b, i]] -= 1
            table[b, i] = -1
        lens[b] = want
    head = [k, v] if case["op"] == "branch" else []
    return head + [_i32(table), _i32(refs), _i32(lens)]
