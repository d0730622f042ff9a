"""Float64 definitions of the speculative-decoding operators (include/tsd.h, last section)."""

import math

import numpy as np


def rope_frequencies(rotary_dim, theta, scaling=None, factor=1.0, original_max_len=0.0, low_freq_factor=1.0,
                     high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0, attention_factor=0.0):
    """(radians per position of each pair, factor on cosines and sines)."""
    R = rotary_dim
    if scaling == "ntk" and R > 2:
        theta = theta * factor ** (R / (R - 2))
    out, mscale = [], 1.0
    if scaling == "yarn":
        mscale = attention_factor or 0.1 * math.log(factor) + 1.0
        dim_of = lambda turns: R * math.log(original_max_len / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(dim_of(beta_fast)), 0), min(math.ceil(dim_of(beta_slow)), R - 1)
    for i in range(R // 2):
        f = theta ** (-2.0 * i / R)
        if scaling == "linear":
            f /= factor
        elif scaling == "banded":
            turns = original_max_len * f / (2 * math.pi)
            if turns <= low_freq_factor:
                f /= factor
            elif turns < high_freq_factor:
                t = (turns - low_freq_factor) / (high_freq_factor - low_freq_factor)
                f = (1 - t) * f / factor + t * f
        elif scaling == "yarn":
            t = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f / factor * t + f * (1 - t)
        out.append(f)
    return np.array(out), mscale


def rope_rotate(x, pos, freq, mscale, interleaved):
    """x [T, H, 128], pos [T]."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(freq))
        c, s = mscale * np.cos(pos * f)[:, None], mscale * np.sin(pos * f)[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def tree_rows(parents):
    """The drafts each draft sees, itself and its ancestors, as sets (parents of one sequence)."""
    rows = []
    for j, p in enumerate(parents):
        rows.append({j} | (rows[p] if 0 <= p < j else set()))
    return rows


def pack_rows(rows, words):
    out = np.zeros((len(rows), words), np.uint32)
    for j, r in enumerate(rows):
        for i in r:
            out[j, i >> 5] |= np.uint32(1 << (i & 31))
    return out


def tree_attention(q, K, V, base, rows, scale):
    """One sequence and kv head: q [n, G, 128], K, V [len, 128]; draft j sees [0, base) and base + rows[j].
    Returns out [n, G, 128], lse [n, G], spread [n, G, 128] = sum_i p_i |V_i| (what rounding errors of
    the weights are relative to)."""
    n, G, D = q.shape
    out, spread = np.zeros((n, G, D)), np.zeros((n, G, D))
    lse = np.full((n, G), -np.inf)
    for j in range(n):
        idx = np.concatenate([np.arange(base), base + np.array(sorted(rows[j]), int)]).astype(int)
        if not idx.size:
            continue
        z = scale * (q[j] @ K[idx].T)
        m = z.max(-1, keepdims=True)
        p = np.exp(z - m)
        s = p.sum(-1, keepdims=True)
        out[j], spread[j] = (p / s) @ V[idx], (p / s) @ np.abs(V[idx])
        lse[j] = (m + np.log(s))[:, 0]
    return out, lse, spread


class Pool:
    """Page table, lengths and reference counts of a paged cache, and the page contents as labels."""

    def __init__(self, table, lens, refs, page, max_len, data=None):
        self.table, self.lens, self.refs = (np.array(np.asarray(x), np.int64) for x in (table, lens, refs))
        self.page, self.max_len = page, max_len
        self.data = None if data is None else data.copy()   # [..., pages at axis 0]
        self.flags = set()

    def pages(self, n):
        return -(-int(n) // self.page)

    def fork(self, src, dst):
        B = len(self.lens)
        start = self.lens.copy()
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < B and 0 <= d < B) or s == d or d in dst[:i] or s in dst or start[d] != 0:
                self.flags.add("BAD_SEQ")
                continue
            n = self.pages(start[s])
            self.table[d] = -1
            self.table[d, :n] = self.table[s, :n]
            for p in self.table[s, :n]:
                self.refs[p] += 1
            self.lens[d] = start[s]

    def resize(self, new_lens):
        start = self.refs.copy()
        free = np.flatnonzero(start == 0).tolist()
        at = 0
        for b, new in enumerate(new_lens):
            old = int(self.lens[b])
            if not 0 <= new <= self.max_len:
                self.flags.add("BAD_SEQ")
                continue
            have, end = self.pages(old), self.pages(new)
            cow = new > old and old % self.page != 0 and start[self.table[b, have - 1]] > 1
            want = max(0, end - have) + int(cow)
            mine, at = free[at:at + want], at + want
            if want and at > len(free):
                self.flags.add("NO_PAGES")
                continue
            if cow:
                p = self.table[b, have - 1]
                self.refs[p] -= 1
                q = mine.pop(0)
                self.table[b, have - 1] = q
                self.refs[q] = 1
                if self.data is not None:
                    self.data[q] = self.data[p]
            for i, p in zip(range(have, end), mine):
                self.table[b, i] = p
                self.refs[p] = 1
            for i in range(end, have):
                self.refs[self.table[b, i]] -= 1
                self.table[b, i] = -1
            self.lens[b] = new
