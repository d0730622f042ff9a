"""The speculative-decoding entry points without a GPU: sizes, and bad arguments refused on the host."""

import ctypes
import math

import numpy as np
import pytest

import top_sparse_decode_topk_b200 as tsd
from oracle import speculative as S
from tests.test_abi import FAKE, fake_pointer_call, lib, make_cache, make_queries   # noqa: F401
from top_sparse_decode_topk_b200 import _LayerC, _RopeC, _RopeScalingC

INVALID, UNSUPPORTED, SMALL = tsd.TSD_ERR_INVALID_ARGUMENT, tsd.TSD_ERR_UNSUPPORTED, tsd.TSD_ERR_WORKSPACE_TOO_SMALL


def rope(rotary_dim=128):
    r = _RopeC()
    r.rotary_dim = rotary_dim
    return r


def append(lib, c=None, q=None, r=None, q_stride=4096, k=FAKE, k_stride=1024, v=FAKE, v_stride=1024, pos=None, depth=None,
           out=FAKE):
    c, q, r = c or make_cache(), q or make_queries(), r or rope()
    return lib.tsd_rope_append(ctypes.byref(c), ctypes.byref(q), ctypes.byref(r), q_stride, k, k_stride, v, v_stride, pos,
                               depth, out, None, None)


@fake_pointer_call
@pytest.mark.parametrize("kw,status", [
    (dict(c=make_cache(head_dim=64)), UNSUPPORTED),
    (dict(q=make_queries(tokens=7)), INVALID),
    (dict(q=make_queries(q_dtype=5)), UNSUPPORTED),
    (dict(r=rope(0)), UNSUPPORTED),
    (dict(r=rope(63)), UNSUPPORTED),
    (dict(r=rope(130)), UNSUPPORTED),
    (dict(q_stride=4095), INVALID),
    (dict(q_stride=4100), INVALID),            # not whole 16-byte pieces of bf16
    (dict(k_stride=1000), INVALID),
    (dict(v_stride=0), INVALID),
    (dict(k=None), INVALID),
    (dict(v=FAKE + 8), INVALID),
    (dict(out=None), INVALID),
    (dict(out=FAKE + 4), INVALID),
    (dict(pos=FAKE, depth=FAKE), INVALID),
])
def test_append_errors_before_launch(lib, kw, status):
    assert append(lib, **kw) == status


@pytest.mark.parametrize("R,theta,scaling,status", [
    (128, 1.0, None, INVALID), (128, math.inf, None, INVALID), (128, math.nan, None, INVALID),
    (3, 1e4, None, UNSUPPORTED), (0, 1e4, None, UNSUPPORTED), (256, 1e4, None, UNSUPPORTED),
    (128, 1e4, (9, 2, 1, 1, 4, 32, 1, 0), INVALID), (128, 1e4, (1, 0.5, 0, 0, 0, 0, 0, 0), INVALID),
    (128, 1e4, (1, math.nan, 0, 0, 0, 0, 0, 0), INVALID), (128, 1e4, (3, 2, 0, 1, 4, 0, 0, 0), INVALID),
    (128, 1e4, (3, 2, 8192, 4, 4, 0, 0, 0), INVALID), (128, 1e4, (4, 2, 8192, 0, 0, 1, 1, 0), INVALID),
    (128, 1e4, (4, 2, 8192, 0, 0, 32, 0, 0), INVALID), (128, 1e4, (4, 2, 8192, 0, 0, 32, 1, -1), INVALID),
])
def test_rope_init_errors(lib, R, theta, scaling, status):
    r = _RopeC()
    sc = None if scaling is None else ctypes.byref(_RopeScalingC(*scaling))
    assert lib.tsd_rope_init(ctypes.byref(r), R, theta, 0, sc) == status
    assert lib.tsd_rope_init(None, 128, 1e4, 0, None) == INVALID


@pytest.mark.parametrize("kw", [
    {}, dict(rotary_dim=2), dict(rotary_dim=50, theta=5e5), dict(scaling="linear", factor=8.0),
    dict(scaling="ntk", factor=4.0, rotary_dim=64), dict(scaling="ntk", factor=4.0, rotary_dim=2),
    dict(scaling="banded", factor=8.0, original_max_len=8192.0, theta=5e5),
    dict(scaling="yarn", factor=4.0, original_max_len=32768.0, theta=1e6),
    dict(scaling="yarn", factor=4.0, original_max_len=100.0, attention_factor=0.7),
])
def test_rope_frequencies(kw):
    """turn[i] against the oracle's frequencies: pow and log in 64 bits are within a few units of 2^-53 (64 of them
    with the exponent's own rounding, 20 such steps), and a turn is a multiple of 2^-64, off by at most half of
    one: pi 2^-64 radians."""
    r = tsd.RotaryEmbedding(**kw)
    o = dict(kw)
    freq, mscale = S.rope_frequencies(o.pop("rotary_dim", 128), o.pop("theta", 10000.0), **o)
    got = np.array([t / 2.0 ** 64 * 2 * math.pi for t in r.turns])
    assert got.shape == freq.shape and (np.abs(got - freq) <= 64 * 2.0 ** -53 * 20 * freq + math.pi * 2.0 ** -64).all()
    assert abs(r.mscale - mscale) <= 2.0 ** -24 * mscale


def test_rope_refuses_unknown_scaling():
    with pytest.raises(ValueError):
        tsd.RotaryEmbedding(scaling="other")
    with pytest.raises(tsd.TsdError):
        tsd.RotaryEmbedding(rotary_dim=127)


@fake_pointer_call
def test_tree_mask_errors_before_launch(lib):
    call = lambda b=8, ip=FAKE, t=64, n=16, p=FAKE, m=FAKE, d=FAKE: lib.tsd_tree_mask(b, ip, t, n, p, m, d, None, None)
    assert call(b=0) == INVALID and call(t=0) == INVALID and call(p=None) == INVALID and call(m=None) == INVALID
    assert call(n=0) == INVALID and call(n=513) == UNSUPPORTED
    assert call(ip=None) == INVALID   # one draft each: num_tokens must equal batch


@fake_pointer_call
def test_tree_decode_errors_before_launch(lib):
    def call(c=None, q=None, out=FAKE, dt=0, ws=FAKE, nbytes=1 << 40):
        c, q = c or make_cache(), q or make_queries(tokens=64, q_indptr=FAKE, max_tokens=16)
        return lib.tsd_tree_decode(ctypes.byref(c), ctypes.byref(q), FAKE, out, dt, None, ws, nbytes, None, None)
    assert call(c=make_cache(page_size=24)) == UNSUPPORTED
    assert call(q=make_queries(sm_scale=0.0)) == INVALID
    assert call(q=make_queries(tokens=1024, q_indptr=FAKE, max_tokens=513)) == UNSUPPORTED
    assert call(out=None) == INVALID and call(out=FAKE + 8) == INVALID and call(dt=7) == UNSUPPORTED
    assert call(ws=None) == INVALID and call(ws=FAKE + 16) == INVALID and call(nbytes=16) == SMALL
    q = make_queries(tokens=64, q_indptr=FAKE, max_tokens=16)
    q.causal = 0
    assert call(q=q) == INVALID
    assert lib.tsd_tree_decode(None, ctypes.byref(q), None, FAKE, 0, None, FAKE, 1 << 40, None, None) == INVALID
    assert lib.tsd_tree_decode_workspace_size(ctypes.byref(make_cache(head_dim=64)), ctypes.byref(make_queries()), 0) == 0
    assert lib.tsd_tree_decode_workspace_size(ctypes.byref(make_cache()), ctypes.byref(make_queries()), 0) > 0
    assert lib.tsd_tree_decode_workspace_size(ctypes.byref(make_cache()), ctypes.byref(make_queries()), 7) == 0


def layers(n, k=FAKE, v=FAKE):
    return (_LayerC * n)(*[_LayerC(k, v) for _ in range(n)])


@fake_pointer_call
def test_cache_calls_errors_before_launch(lib):
    c, cont = make_cache(), make_cache(layout=1, page_table=None)
    fork = lambda c=c, r=FAKE, n=2, s=FAKE, d=FAKE: lib.tsd_cache_fork(ctypes.byref(c), r, n, s, d, None, None)
    assert fork(c=cont) == UNSUPPORTED and fork(r=None) == INVALID and fork(n=-1) == INVALID
    assert fork(s=None) == INVALID and fork(d=None) == INVALID and fork(n=0, s=None, d=None) == tsd.TSD_OK

    def resize(c=c, n=2, ls=None, r=FAKE, nl=FAKE, ws=FAKE, nbytes=1 << 40):
        return lib.tsd_cache_resize(ctypes.byref(c), n, layers(max(n, 1)) if ls is None else ls, r, nl, ws, nbytes, None,
                                    None)
    assert resize(c=cont) == UNSUPPORTED and resize(n=0) == INVALID and resize(n=129) == UNSUPPORTED
    assert resize(ls=layers(2, v=None)) == INVALID and resize(ls=layers(2, k=FAKE + 8)) == INVALID
    assert resize(r=None) == INVALID and resize(nl=None) == INVALID and resize(ws=None) == INVALID
    assert resize(ws=FAKE + 16) == INVALID and resize(nbytes=64) == SMALL
    assert lib.tsd_cache_resize_workspace_size(ctypes.byref(c)) >= 4 * c.num_pages
    assert lib.tsd_cache_resize_workspace_size(ctypes.byref(cont)) == 0
    assert lib.tsd_cache_resize_workspace_size(None) == 0

    def compact(c=c, n=2, ls=None, ip=FAKE, t=64, m=16, keep=FAKE, k=4, out=FAKE + 0x900000):
        return lib.tsd_cache_compact(ctypes.byref(c), n, layers(max(n, 1)) if ls is None else ls, ip, t, m, keep, k, None,
                                     out, None, None)
    assert compact(n=0) == INVALID and compact(n=129) == UNSUPPORTED and compact(keep=None) == INVALID
    assert compact(k=0) == INVALID and compact(out=None) == INVALID and compact(m=-1) == INVALID
    assert compact(ip=None) == INVALID and compact(c=make_cache(head_dim=64)) == UNSUPPORTED
    assert compact(out=FAKE + 0x300000) == INVALID          # seq_lens itself
    assert compact(out=FAKE + 0x300000 + 28) == INVALID     # its last entry


def test_layers_must_agree():
    import torch
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    kv = lambda pages=5: tsd.KVCache(torch.zeros(pages, 1, 4, 128, dtype=torch.bfloat16),
                                     torch.zeros(pages, 1, 4, 128, dtype=torch.bfloat16), lens, 16, page_table=table)
    assert len(tsd.LayerCaches([kv(), kv()]).caches) == 2
    with pytest.raises(ValueError):
        tsd.LayerCaches([kv(), kv(6)])
    with pytest.raises(ValueError):
        tsd.LayerCaches([kv(), tsd.KVCache(kv().k, kv().v, lens.clone(), 16, page_table=table)])
    with pytest.raises(ValueError):
        tsd.LayerCaches([])
