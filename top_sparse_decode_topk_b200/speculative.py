"""Speculative decoding over the paged cache: binding of the last section of include/tsd.h.

    caches = LayerCaches(per_layer_caches)             # one page table, one seq_lens
    cache_resize(caches, refs, seq_lens + n)           # pages for the drafts (copy on write)
    mask, depth = tree_mask(parents, q_indptr, n_max)  # ancestors of every draft
    for layer ...:
        q = rope_append(cache, rope, q, k, v, q_indptr, n_max, depth=depth)
        out, lse = tree_decode(cache, Queries(q, q_indptr, n_max), mask)
    new_lens = cache_compact(caches, keep, q_indptr, n_max, refs=refs)
    cache_resize(caches, refs, new_lens)               # the rejected drafts' pages go back
    cache_fork(caches, refs, src, dst)                 # sequences that share src's pages

All tensors are on the cache's device.  Nothing here waits for the device, so every call can be
captured into a CUDA graph (call it once before, so that the status word below exists).

Outputs and scratch are allocated per call on the call's stream unless the caller passes them, so
calls on several streams and several captured graphs share nothing.  Device-detected problems set
bits in `status` (an int32 tensor), else in the workspace when one is passed, else in a word kept per
device; ``read_device_status`` reads the latter two.  `stream` defaults to the current stream; tensors
made on another stream have to be ready on it, as for every call of this package.
"""

from __future__ import annotations

import ctypes
from typing import Optional

from . import (DEV_BAD_SEQ, TSD_BF16, TSD_ERR_INVALID_ARGUMENT, TSD_F32, KVCache, Queries, TsdError, Workspace,  # noqa: F401
               _check, _KvCacheC, _LayerC, _QueriesC, _RopeC, _RopeScalingC, _shape_key, load_library)

_SCALING = {"linear": 1, "ntk": 2, "banded": 3, "yarn": 4}

_STATUS = {}   # device index -> the status word of calls without one of their own


class _Call:
    """The device and stream of one call: `with` makes them current where they are not already."""

    def __init__(self, device, stream):
        import torch
        self.device = device
        self.guards = []
        if torch.cuda.current_device() != device.index:
            self.guards.append(torch.cuda.device(device))
        if stream is not None:
            self.guards.append(torch.cuda.stream(stream))
        else:
            stream = torch.cuda.current_stream(device)
        self.ptr = stream.cuda_stream

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _status_ptr(status, device):
    import torch
    if status is not None:
        if status.dtype != torch.int32 or status.device != device or status.numel() < 1:
            raise ValueError("status must be an int32 tensor on the cache's device")
        return status.data_ptr()
    word = _STATUS.get(device.index)
    if word is None:
        word = _STATUS[device.index] = torch.zeros(64, dtype=torch.int32, device=device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(device).synchronize()   # once: other streams may use it at once
    return word.data_ptr()


def _int32(t, name, device, *shape):
    """A contiguous int32 tensor on `device` of the given shape (None: any extent)."""
    import torch
    if t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on {device}")
    if t.dim() != len(shape) or any(want is not None and int(have) != want for have, want in zip(t.shape, shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    return t.data_ptr()


def _indptr(q_indptr, batch, device):
    return None if q_indptr is None else _int32(q_indptr, "q_indptr", device, batch + 1)


class RotaryEmbedding:
    """Rotary positions: dims [0, rotary_dim) of a head turn by theta^(-2i / rotary_dim) per position,
    as pairs (i, i + rotary_dim / 2) or, interleaved, (2i, 2i + 1).

    scaling: None, "linear", "ntk", "banded" or "yarn" (include/tsd.h, tsd_rope_scaling_kind), with the
    constants that kind uses.  attention_factor 0 means YaRN's own 0.1 ln(factor) + 1."""

    def __init__(self, rotary_dim: int = 128, theta: float = 10000.0, interleaved: bool = False,
                 scaling: Optional[str] = None, factor: float = 1.0, original_max_len: float = 0.0,
                 low_freq_factor: float = 1.0, high_freq_factor: float = 4.0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, attention_factor: float = 0.0):
        if scaling is not None and scaling not in _SCALING:
            raise ValueError(f"scaling must be None or one of {sorted(_SCALING)}")
        self.c = _RopeC()
        sc = None
        if scaling is not None:
            sc = ctypes.byref(_RopeScalingC(_SCALING[scaling], factor, original_max_len, low_freq_factor,
                                            high_freq_factor, beta_fast, beta_slow, attention_factor))
        _check(load_library().tsd_rope_init(ctypes.byref(self.c), int(rotary_dim), float(theta), int(bool(interleaved)),
                                            sc), "tsd_rope_init")
        self.rotary_dim, self.interleaved = int(rotary_dim), bool(interleaved)

    @property
    def turns(self):
        """Full turns per position of each pair, in units of 2^-64."""
        return [int(x) for x in self.c.turn[:self.rotary_dim // 2]]

    @property
    def mscale(self) -> float:
        return float(self.c.mscale)


def _rows(t, name, heads, dtype, device, tokens):
    """[T, heads, 128] rows whose heads are 128 apart; returns (pointer, elements from token to token)."""
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != 128 or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a [{tokens}, heads, 128] {dtype} tensor on {device}")
    if heads is not None and t.shape[1] != heads:
        raise ValueError(f"{name} must have {heads} heads")
    st = t.stride()
    if st[2] != 1 or (t.shape[1] > 1 and st[1] != 128):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (st[0] if tokens > 1 else int(t.shape[1]) * 128)


def rope_append(cache: KVCache, rope: RotaryEmbedding, q, k, v, q_indptr=None, max_tokens_per_seq: int = 1,
                positions=None, depth=None, out_q=None, status=None, stream=None):
    """Rotate a step's queries and keys and write its K and V rows into the cache (tsd_rope_append).

    q [T, Hq, 128], k, v [T, Hkv, 128], bf16 or fp32 (one type); tokens may be strided (slices of a fused
    projection).  New token j of sequence b goes to cache position seq_lens[b] - n_b + j; its angle is at
    `positions` (int32 [T]) if given, at seq_lens[b] - n_b + depth (int32 [T], as tree_mask returns) if
    given, else at its cache position.  Returns the rotated queries ([T, Hq, 128], contiguous; `out_q`
    may be q itself)."""
    import torch
    dev = cache.device
    with _Call(dev, stream) as call:
        T, Hq = int(q.shape[0]), int(q.shape[1])
        if q.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("q must be bfloat16 or float32")
        c = _QueriesC()
        c.q, q_stride = _rows(q, "q", None, q.dtype, dev, T)
        kp, k_stride = _rows(k, "k", cache.num_kv_heads, q.dtype, dev, T)
        vp, v_stride = _rows(v, "v", cache.num_kv_heads, q.dtype, dev, T)
        c.q_dtype = TSD_BF16 if q.dtype == torch.bfloat16 else TSD_F32
        c.num_q_heads, c.num_tokens = Hq, T
        c.q_indptr = _indptr(q_indptr, cache.batch, dev)
        c.max_tokens_per_seq = 1 if q_indptr is None else int(max_tokens_per_seq)
        c.causal, c.sm_scale = 1, 1.0
        if out_q is None:
            out_q = torch.empty((T, Hq, 128), dtype=q.dtype, device=dev)
        elif out_q.shape != q.shape or out_q.dtype != q.dtype or out_q.device != dev or not out_q.is_contiguous():
            raise ValueError("out_q must be a contiguous tensor of q's shape and type")
        _check(load_library().tsd_rope_append(
            ctypes.byref(cache.c_struct()), ctypes.byref(c), ctypes.byref(rope.c), q_stride, kp, k_stride, vp, v_stride,
            None if positions is None else _int32(positions, "positions", dev, T),
            None if depth is None else _int32(depth, "depth", dev, T), out_q.data_ptr(), _status_ptr(status, dev),
            call.ptr), "tsd_rope_append")
    return out_q


def tree_mask(parents, q_indptr=None, max_tokens_per_seq: int = 1, mask=None, depth=None, status=None, stream=None):
    """Ancestors of drafted tokens (tsd_tree_mask): parents int32 [T], each the index of an earlier draft of
    the same sequence or -1.  Returns (mask int32 [T, ceil(max_tokens_per_seq / 32)] of bits, depth
    int32 [T])."""
    import torch
    dev = parents.device
    if dev.type != "cuda":
        raise ValueError("parents must be on a CUDA device")
    with _Call(dev, stream) as call:
        T = int(parents.shape[0])
        pp = _int32(parents, "parents", dev, T)
        batch = T if q_indptr is None else int(q_indptr.shape[0]) - 1
        n = 1 if q_indptr is None else int(max_tokens_per_seq)
        W = (n + 31) // 32
        if mask is None:
            mask = torch.empty((T, W), dtype=torch.int32, device=dev)
        if depth is None:
            depth = torch.empty((T,), dtype=torch.int32, device=dev)
        _check(load_library().tsd_tree_mask(batch, _indptr(q_indptr, batch, dev), T, n, pp,
                                            _int32(mask, "mask", dev, T, W), _int32(depth, "depth", dev, T),
                                            _status_ptr(status, dev), call.ptr), "tsd_tree_mask")
    return mask, depth


def tree_decode(cache: KVCache, queries: Queries, mask=None, out=None, out_dtype=None, lse=True,
                workspace: Optional[Workspace] = None, status=None, stream=None):
    """Attention of drafted tokens over the cache and over the drafts their mask names (tsd_tree_decode).

    mask: int32 [T, ceil(max_tokens_per_seq / 32)], bit i of a row for draft i of the sequence, or None
    for a chain of drafts.  Returns (out [T, Hq, 128], lse [T, Hq] or None); a draft that sees nothing
    gets out 0 and lse -inf.  workspace: scratch to reuse; by default it is allocated per call."""
    import torch
    lib = load_library()
    dev = cache.device
    q = queries.q
    if q.device != dev or (queries.q_indptr is not None and queries.q_indptr.device != dev):
        raise ValueError("tree_decode takes device tensors only")
    with _Call(dev, stream) as call:
        _indptr(queries.q_indptr, cache.batch, dev)
        cs, qs = cache.c_struct(), queries.c_struct()
        T, Hq = int(q.shape[0]), int(q.shape[1])
        mp = None
        if mask is not None:
            mp = _int32(mask, "mask", dev, T, (qs.max_tokens_per_seq + 31) // 32)
        if out is None:
            out = torch.empty((T, Hq, 128), dtype=out_dtype or torch.bfloat16, device=dev)
        elif tuple(out.shape) != (T, Hq, 128) or out.device != dev or not out.is_contiguous():
            raise ValueError("out must be a contiguous [T, Hq, 128] tensor on the cache's device")
        elif out_dtype is not None and out_dtype != out.dtype:
            raise ValueError("out_dtype disagrees with out")
        if out.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("out must be bfloat16 or float32")
        if lse is True:
            lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        elif lse is None or lse is False:
            lse = None
        elif tuple(lse.shape) != (T, Hq) or lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous float32 [T, Hq] tensor on the cache's device")
        odt = TSD_BF16 if out.dtype == torch.bfloat16 else TSD_F32
        nbytes = lib.tsd_tree_decode_workspace_size(ctypes.byref(cs), ctypes.byref(qs), odt)
        ws, sp = _scratch(workspace, nbytes, ("tree_decode",) + _shape_key(cache, queries), dev, call, status)
        _check(lib.tsd_tree_decode(ctypes.byref(cs), ctypes.byref(qs), mp, out.data_ptr(), odt,
                                   None if lse is None else lse.data_ptr(), ws[0], nbytes, sp, call.ptr),
               "tsd_tree_decode")
    return out, lse


def _scratch(workspace, nbytes, key, dev, call, status):
    """Scratch of `nbytes` as (pointer, owner), and the status word to use.  A Workspace keeps its status
    word in its first 256 bytes; the scratch lies behind them."""
    import torch
    if workspace is None:
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        return (buf.data_ptr(), buf), _status_ptr(status, dev)
    buf = workspace.get(nbytes + 256, key, call.ptr)
    return (buf.data_ptr() + 256, buf), buf.data_ptr() if status is None else _status_ptr(status, dev)


class LayerCaches:
    """The layers of a model: KVCaches of one shape that share a page table and seq_lens, as the calls
    below take them.  Made once and kept; the calls also take a KVCache or a list of them."""

    def __init__(self, caches):
        caches = [caches] if isinstance(caches, KVCache) else list(caches)
        if not caches:
            raise ValueError("at least one cache")
        c0 = caches[0]
        for c in caches[1:]:
            if c.k.shape != c0.k.shape or c.device != c0.device or c.seq_lens.data_ptr() != c0.seq_lens.data_ptr() or \
                    int(c.max_seq_len) != int(c0.max_seq_len) or (c.page_table is None) != (c0.page_table is None) or \
                    (c.page_table is not None and c.page_table.data_ptr() != c0.page_table.data_ptr()):
                raise ValueError("the layers must share their page table, seq_lens and shapes")
        self.caches = caches
        self.c_layers = (_LayerC * len(caches))(*[_LayerC(c.k.data_ptr(), c.v.data_ptr()) for c in caches])

    @staticmethod
    def of(caches) -> "LayerCaches":
        return caches if isinstance(caches, LayerCaches) else LayerCaches(caches)


def _refs(refs, cache, dev):
    if cache.page_table is None:
        raise ValueError("refs go with a paged cache")
    return _int32(refs, "refs", dev, int(cache.k.shape[0]))


def cache_fork(caches, refs, src, dst, status=None, stream=None) -> None:
    """Start each empty sequence dst[i] as a copy of src[i] that shares its pages (tsd_cache_fork).

    refs: int32 [num_pages], how many page-table entries hold each page (0: free).  src, dst: int32 [n].
    The cache's page_table and seq_lens and refs are updated in place."""
    cache = LayerCaches.of(caches).caches[0]
    dev = cache.device
    with _Call(dev, stream) as call:
        n = int(src.shape[0])
        _check(load_library().tsd_cache_fork(ctypes.byref(cache.c_struct()), _refs(refs, cache, dev), n,
                                             _int32(src, "src", dev, n), _int32(dst, "dst", dev, n),
                                             _status_ptr(status, dev), call.ptr), "tsd_cache_fork")


def cache_resize(caches, refs, new_lens, workspace: Optional[Workspace] = None, status=None, stream=None) -> None:
    """Take and release pages so that sequence b has room for new_lens[b] tokens (tsd_cache_resize), and set
    seq_lens to new_lens.

    A growing sequence whose partly filled last page is shared gets a copy of it in every layer.  Pages are
    the lowest free ones at the start of the call, given out in order of sequence; where they do not
    suffice a sequence stays as it was (DEV_NO_PAGES).  The cache's page_table (-1 where a page was
    released), seq_lens and refs are updated in place."""
    lib = load_library()
    layers = LayerCaches.of(caches)
    cache = layers.caches[0]
    dev = cache.device
    with _Call(dev, stream) as call:
        rp = _refs(refs, cache, dev)
        np_ = _int32(new_lens, "new_lens", dev, cache.batch)
        cs = cache.c_struct()
        nbytes = lib.tsd_cache_resize_workspace_size(ctypes.byref(cs))
        ws, sp = _scratch(workspace, nbytes, ("cache_resize", cache.batch, int(cache.k.shape[0])), dev, call, status)
        _check(lib.tsd_cache_resize(ctypes.byref(cs), len(layers.caches), layers.c_layers, rp, np_, ws[0], nbytes, sp,
                                    call.ptr), "tsd_cache_resize")


def cache_compact(caches, keep, q_indptr=None, max_tokens_per_seq: int = 1, refs=None, out_lens=None, status=None,
                  stream=None):
    """Move the accepted drafts of every sequence to the front of its drafts, in all layers
    (tsd_cache_compact).

    keep: int32 [B, k_max], ascending indices of accepted drafts, then -1.  q_indptr: int32 [B + 1], the
    drafts of each sequence (None: one each).  refs: when given, a sequence whose rows to be written lie in
    a shared page is left as it was (DEV_SHARED_PAGE).  Returns the new lengths, int32 [B], to be passed to
    cache_resize; seq_lens itself is not changed."""
    import torch
    lib = load_library()
    layers = LayerCaches.of(caches)
    cache = layers.caches[0]
    dev = cache.device
    with _Call(dev, stream) as call:
        B = cache.batch
        if out_lens is None:
            out_lens = torch.empty((B,), dtype=torch.int32, device=dev)
        n = 1 if q_indptr is None else int(max_tokens_per_seq)
        kp = _int32(keep, "keep", dev, B, None)
        if int(keep.shape[1]) < 1:
            raise TsdError(TSD_ERR_INVALID_ARGUMENT, "keep must have room for one draft")
        _check(lib.tsd_cache_compact(ctypes.byref(cache.c_struct()), len(layers.caches), layers.c_layers,
                                     _indptr(q_indptr, B, dev), n * B, n, kp, int(keep.shape[1]),
                                     None if refs is None else _refs(refs, cache, dev),
                                     _int32(out_lens, "out_lens", dev, B), _status_ptr(status, dev), call.ptr),
               "tsd_cache_compact")
    return out_lens
