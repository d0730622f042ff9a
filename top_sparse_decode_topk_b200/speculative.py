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

A step without new tokens (T = 0) is allowed and does nothing.  All tensors are on the cache's device.  Nothing here
waits for the device, so every call can be captured into a CUDA graph.  The first call on a device, and the first
with a new workspace, makes the status word below, and is refused during a capture: make it before.

Outputs and scratch are allocated per call on the call's stream unless the caller passes them, so
calls on several streams and several captured graphs share nothing.  Device-detected problems set
bits in `status` (an int32 tensor), else in the workspace when one is passed, else in a word kept per
device; ``read_device_status`` reads the latter two.  `stream` defaults to the current stream; tensors
made on another stream have to be ready on it, as for every call of this package.  Two calls at once are fine where
they write different sequences; cache_fork and cache_resize write `refs`, so of those one at a time over a pool.  Trees
can be attended to densely only, and a LabelIndex does not follow rows written here: build it again.
"""

from __future__ import annotations

import ctypes
from typing import Optional

from . import (TSD_BF16, TSD_ERR_INVALID_ARGUMENT, TSD_F32, KVCache, Queries, TsdError, Workspace, _check, _LayerC,
               _QueriesC, _RopeC, _RopeScalingC, load_library)

_SCALING = {"linear": 1, "ntk": 2, "banded": 3, "yarn": 4}

_STATUS = {}   # device index -> the status word of calls without one of their own

# A step of one layer is a handful of calls, each a few microseconds on the GPU for a small batch, so what the
# calls do on the host is kept short: torch and the library are looked up once, and the device and stream are
# made current only where they are not.
torch = None
_LIB = None


def _ready():
    global torch, _LIB
    if torch is None:
        import torch as t
        _LIB = load_library()
        torch = t


def _elsewhere(dev, stream) -> bool:
    """Whether the call needs a guard: another device is current, or a stream was given."""
    if torch is None:
        _ready()
    return stream is not None or torch._C._cuda_getDevice() != dev.index


class _Guard:
    """Makes a device, and a stream on it, current."""

    def __init__(self, device, stream):
        self.guards = [torch.cuda.device(device)] + ([torch.cuda.stream(stream)] if stream is not None else [])

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _cuda(t, name):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device")
    return t.device


def _raw_stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _status_word(device):
    """A status word, cleared before any stream may use it."""
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError("the status word of this device or workspace does not exist yet: make a call before capturing")
    word = torch.zeros(64, dtype=torch.int32, device=device)
    torch.cuda.current_stream(device).synchronize()   # once: other streams may use it at once
    return word


def _status_ptr(status, device):
    if status is not None:
        if status.dtype != torch.int32 or status.device != device or status.numel() < 1:
            raise ValueError("status must be an int32 tensor on the cache's device")
        return status.data_ptr()
    word = _STATUS.get(device.index)
    if word is None:
        word = _STATUS.setdefault(device.index, _status_word(device))   # the first of several host threads' words
    return word.data_ptr()


def _int32(t, name, device, shape):
    """Pointer of a contiguous int32 tensor of the given shape on `device`."""
    if t.dtype is not torch.int32 or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _check_arrays(cache):
    """The kernels index k, v, seq_lens and page_table as dense arrays with a row for every sequence, and some write
    them.  A cache's fields may have been assigned since it was made, so k and v are looked at again too."""
    k, v, lens, table = cache.k, cache.v, cache.seq_lens, cache.page_table
    if k.dim() != 4 or k.shape != v.shape or k.shape[3] != 128 or k.dtype != v.dtype or str(k.dtype) != "torch.bfloat16" or \
            not k.is_contiguous() or not v.is_contiguous() or v.device != k.device or lens.device != k.device:
        raise ValueError("k and v must be contiguous bfloat16 tensors of one 4-d shape with head_dim 128, on one device")
    if lens.dim() < 1 or lens.numel() != lens.shape[0] or not lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous int32 [batch] tensor")
    if table is None:
        if cache.k.shape[0] < lens.shape[0]:
            raise ValueError("contiguous cache: k and v must have a row for every entry of seq_lens")
    elif table.device != cache.k.device or not table.is_contiguous() or table.shape[0] < lens.shape[0]:
        raise ValueError("page_table must be a contiguous tensor on the cache's device with a row for every entry of seq_lens")


def _check_written(cache):
    """For the calls that update page_table in place."""
    if cache.page_table is not None and cache.page_table is cache.__dict__.get("_table_copy"):
        raise ValueError("the page_table given was not contiguous, so the cache holds a copy, and an update would not "
                         "reach the original: give a contiguous table")


def _cache_struct(cache):
    """cache.c_struct(), reused while the cache holds the same tensors at the same addresses."""
    kept = cache.__dict__.get("_spec_struct")
    if kept is not None:
        k, v, lens, table, max_len, c = kept
        if k is cache.k and v is cache.v and lens is cache.seq_lens and table is cache.page_table and \
                max_len == cache.max_seq_len and c.k == k.data_ptr() and c.v == v.data_ptr() and \
                c.seq_lens == lens.data_ptr() and (table is None or c.page_table == table.data_ptr()):
            return c
    if cache.k.device.type != "cuda":
        raise ValueError("the cache must be on a CUDA device")
    _check_arrays(cache)
    c = cache.c_struct()
    cache.__dict__["_spec_struct"] = (cache.k, cache.v, cache.seq_lens, cache.page_table, cache.max_seq_len, c)
    return c


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


def _rows(t, name, shape, dtype, device):
    """[T, heads, 128] rows whose heads are 128 apart; returns (pointer, elements from token to token)."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be a {tuple(shape)} {dtype} tensor on {device}")
    a, b, c = t.stride()
    if c != 1 or (b != 128 and shape[1] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), a if shape[0] > 1 else shape[1] * 128


def rope_append(cache: KVCache, rope: RotaryEmbedding, q, k, v, q_indptr=None, max_tokens_per_seq: int = 1,
                positions=None, depth=None, out_q=None, status=None, stream=None):
    """Rotate a step's queries and keys and write its K and V rows into the cache (tsd_rope_append).

    q [T, Hq, 128], k, v [T, Hkv, 128], bf16 or fp32 (one type); tokens may be strided (slices of a fused
    projection).  New token j of sequence b goes to cache position seq_lens[b] - n_b + j; its angle is at
    `positions` (int32 [T]) if given, at seq_lens[b] - n_b + depth (int32 [T], as tree_mask returns) if
    given, else at its cache position.  Returns the rotated queries ([T, Hq, 128], contiguous; `out_q`
    may be q itself)."""
    dev = _cuda(cache.k, "the cache")
    if _elsewhere(dev, stream):
        with _Guard(dev, stream):
            return rope_append(cache, rope, q, k, v, q_indptr, max_tokens_per_seq, positions, depth, out_q, status)
    dtype = q.dtype
    if dtype is torch.bfloat16:
        code = TSD_BF16
    elif dtype is torch.float32:
        code = TSD_F32
    else:
        raise TypeError("q must be bfloat16 or float32")
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, 128]")
    T, Hq, _ = q.shape
    kv = (T, cache.k.shape[1], 128)
    qp, q_stride = _rows(q, "q", (T, Hq, 128), dtype, dev)
    kp, k_stride = _rows(k, "k", kv, dtype, dev)
    vp, v_stride = _rows(v, "v", kv, dtype, dev)
    cs = _cache_struct(cache)
    if q_indptr is None:
        ip, max_tokens_per_seq = None, 1
    else:
        ip = _int32(q_indptr, "q_indptr", dev, (cs.batch + 1,))
    c = _QueriesC(qp, code, Hq, T, ip, int(max_tokens_per_seq), 1, 1.0)
    if out_q is None:
        out_q = torch.empty((T, Hq, 128), dtype=dtype, device=dev)
    elif out_q.shape != q.shape or out_q.dtype is not dtype or out_q.device != dev or not out_q.is_contiguous():
        raise ValueError("out_q must be a contiguous tensor of q's shape and type")
    if T == 0:
        return out_q
    st = _LIB.tsd_rope_append(cs, c, rope.c, q_stride, kp, k_stride, vp, v_stride,
                              None if positions is None else _int32(positions, "positions", dev, (T,)),
                              None if depth is None else _int32(depth, "depth", dev, (T,)), out_q.data_ptr(),
                              _status_ptr(status, dev), _raw_stream(dev))
    if st:
        raise TsdError(st, "tsd_rope_append")
    return out_q


def tree_mask(parents, q_indptr=None, max_tokens_per_seq: int = 1, mask=None, depth=None, status=None, stream=None):
    """Ancestors of drafted tokens (tsd_tree_mask): parents int32 [T], each the index of an earlier draft of
    the same sequence or -1.  Returns (mask int32 [T, ceil(max_tokens_per_seq / 32)] of bits, depth
    int32 [T])."""
    dev = _cuda(parents, "parents")
    if _elsewhere(dev, stream):
        with _Guard(dev, stream):
            return tree_mask(parents, q_indptr, max_tokens_per_seq, mask, depth, status)
    T = parents.shape[0]
    pp = _int32(parents, "parents", dev, (T,))
    if q_indptr is None:
        batch, n, ip = T, 1, None
    else:
        batch, n = q_indptr.shape[0] - 1, int(max_tokens_per_seq)
        ip = _int32(q_indptr, "q_indptr", dev, (batch + 1,))
    W = (n + 31) // 32
    if mask is None:
        mask = torch.empty((T, W), dtype=torch.int32, device=dev)
    if depth is None:
        depth = torch.empty((T,), dtype=torch.int32, device=dev)
    if T == 0:
        return mask, depth
    st = _LIB.tsd_tree_mask(batch, ip, T, n, pp, _int32(mask, "mask", dev, (T, W)), _int32(depth, "depth", dev, (T,)),
                            _status_ptr(status, dev), _raw_stream(dev))
    if st:
        raise TsdError(st, "tsd_tree_mask")
    return mask, depth


def tree_decode(cache: KVCache, queries: Queries, mask=None, out=None, out_dtype=None, lse=True,
                workspace: Optional[Workspace] = None, status=None, stream=None):
    """Attention of drafted tokens over the cache and over the drafts their mask names (tsd_tree_decode).

    mask: int32 [T, ceil(max_tokens_per_seq / 32)], bit i of a row for draft i of the sequence, or None
    for a chain of drafts.  Returns (out [T, Hq, 128], lse [T, Hq] or None); a draft that sees nothing
    gets out 0 and lse -inf.  workspace: scratch to reuse; by default it is allocated per call."""
    dev = _cuda(cache.k, "the cache")
    if _elsewhere(dev, stream):
        with _Guard(dev, stream):
            return tree_decode(cache, queries, mask, out, out_dtype, lse, workspace, status)
    q = queries.q
    if q.device != dev:
        raise ValueError("tree_decode takes device tensors only")
    cs, qs = _cache_struct(cache), queries.c_struct()
    T, Hq, _ = q.shape
    if queries.q_indptr is not None:
        _int32(queries.q_indptr, "q_indptr", dev, (cs.batch + 1,))
    mp = None if mask is None else _int32(mask, "mask", dev, (T, (qs.max_tokens_per_seq + 31) // 32))
    if out is None:
        out = torch.empty((T, Hq, 128), dtype=out_dtype or torch.bfloat16, device=dev)
    elif out.shape != (T, Hq, 128) or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous [T, Hq, 128] tensor on the cache's device")
    elif out_dtype is not None and out_dtype != out.dtype:
        raise ValueError("out_dtype disagrees with out")
    if out.dtype is torch.bfloat16:
        code = TSD_BF16
    elif out.dtype is torch.float32:
        code = TSD_F32
    else:
        raise TypeError("out must be bfloat16 or float32")
    if lse is True:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    elif lse is None or lse is False:
        lse = None
    elif lse.shape != (T, Hq) or lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [T, Hq] tensor on the cache's device")
    if T == 0:
        return out, lse
    nbytes = _LIB.tsd_tree_decode_workspace_size(cs, qs, code)
    ws, keep, sp = _scratch(workspace, nbytes, dev, status)
    st = _LIB.tsd_tree_decode(cs, qs, mp, out.data_ptr(), code, None if lse is None else lse.data_ptr(), ws, nbytes, sp,
                              _raw_stream(dev))
    if st:
        raise TsdError(st, "tsd_tree_decode")
    return out, lse


def _scratch(workspace, nbytes, dev, status):
    """Scratch of `nbytes`: its pointer, its owner, and the status word to use."""
    if workspace is None:
        buf = torch.empty(nbytes if nbytes > 256 else 256, dtype=torch.uint8, device=dev)
        return buf.data_ptr(), buf, _status_ptr(status, dev)
    if workspace.spec_status is None:
        word = _status_word(dev)
        if workspace.spec_status is None:
            workspace.spec_status = word
    buf = workspace.spec_scratch(nbytes, dev)
    return buf.data_ptr(), buf, _status_ptr(workspace.spec_status if status is None else status, dev)


class LayerCaches:
    """The layers of a model: KVCaches of one shape that share a page table and seq_lens, as the calls
    below take them.  Made once and kept; the calls also take a KVCache or a list of them.  A cache whose k or v
    is replaced afterwards is looked at anew by the next call."""

    def __init__(self, caches):
        caches = [caches] if isinstance(caches, KVCache) else list(caches)
        if not caches:
            raise ValueError("at least one cache")
        self.caches = tuple(caches)
        self._bind()

    def _bind(self):
        caches, c0 = self.caches, self.caches[0]
        if len(caches) > 1:
            for c in caches:
                _check_written(c)   # each would have its own copy
        for c in caches:
            _check_arrays(c)
            if c.k.shape != c0.k.shape or c.device != c0.device or c.seq_lens.data_ptr() != c0.seq_lens.data_ptr() or \
                    int(c.max_seq_len) != int(c0.max_seq_len) or (c.page_table is None) != (c0.page_table is None) or \
                    (c.page_table is not None and c.page_table.data_ptr() != c0.page_table.data_ptr()):
                raise ValueError("the layers must share their page table, seq_lens and shapes")
        self._held = [(c, c.k, c.v) for c in caches]   # whose addresses these are
        self._c_layers = (_LayerC * len(caches))(*[_LayerC(c.k.data_ptr(), c.v.data_ptr()) for c in caches])

    @property
    def c_layers(self):
        for c, k, v in self._held:
            if c.k is not k or c.v is not v:
                self._bind()
                break
        return self._c_layers

    @staticmethod
    def of(caches) -> "LayerCaches":
        return caches if isinstance(caches, LayerCaches) else LayerCaches(caches)


def _refs(refs, cache, dev):
    if cache.page_table is None:
        raise ValueError("refs go with a paged cache")
    return _int32(refs, "refs", dev, (cache.k.shape[0],))


def cache_fork(caches, refs, src, dst, status=None, stream=None) -> None:
    """Start each empty sequence dst[i] as a copy of src[i] that shares its pages (tsd_cache_fork).

    refs: int32 [num_pages], how many page-table entries hold each page (0: free).  src, dst: int32 [n].
    The cache's page_table and seq_lens and refs are updated in place."""
    caches = LayerCaches.of(caches)
    cache = caches.caches[0]
    dev = _cuda(cache.k, "the cache")
    if _elsewhere(dev, stream):
        with _Guard(dev, stream):
            return cache_fork(caches, refs, src, dst, status)
    _check_written(cache)
    n = src.shape[0]
    st = _LIB.tsd_cache_fork(_cache_struct(cache), _refs(refs, cache, dev), n, _int32(src, "src", dev, (n,)),
                             _int32(dst, "dst", dev, (n,)), _status_ptr(status, dev), _raw_stream(dev))
    if st:
        raise TsdError(st, "tsd_cache_fork")


def cache_resize(caches, refs, new_lens, workspace: Optional[Workspace] = None, status=None, stream=None) -> None:
    """Take and release pages so that sequence b has room for new_lens[b] tokens (tsd_cache_resize), and set
    seq_lens to new_lens.

    A growing sequence whose partly filled last page is shared gets a copy of it in every layer.  Pages are
    the lowest free ones at the start of the call, given out in order of sequence; where they do not
    suffice a sequence stays as it was (DEV_NO_PAGES).  The cache's page_table (-1 where a page was
    released), seq_lens and refs are updated in place."""
    caches = LayerCaches.of(caches)
    cache = caches.caches[0]
    dev = _cuda(cache.k, "the cache")
    if _elsewhere(dev, stream):
        with _Guard(dev, stream):
            return cache_resize(caches, refs, new_lens, workspace, status)
    _check_written(cache)
    rp = _refs(refs, cache, dev)
    cs = _cache_struct(cache)
    lens = _int32(new_lens, "new_lens", dev, (cs.batch,))
    nbytes = _LIB.tsd_cache_resize_workspace_size(cs)
    ws, keep, sp = _scratch(workspace, nbytes, dev, status)
    layers = caches.c_layers
    st = _LIB.tsd_cache_resize(cs, len(layers), layers, rp, lens, ws, nbytes, sp, _raw_stream(dev))
    if st:
        raise TsdError(st, "tsd_cache_resize")


def cache_compact(caches, keep, q_indptr=None, max_tokens_per_seq: int = 1, refs=None, out_lens=None, status=None,
                  stream=None):
    """Move the accepted drafts of every sequence to the front of its drafts, in all layers
    (tsd_cache_compact).

    keep: int32 [B, k_max], ascending indices of accepted drafts, then -1.  q_indptr: int32 [B + 1], the
    drafts of each sequence (None: one each).  refs: when given, a sequence whose rows to be written lie in
    a shared page is left as it was (DEV_SHARED_PAGE).  Returns the new lengths, int32 [B], to be passed to
    cache_resize; seq_lens itself is not changed."""
    caches = LayerCaches.of(caches)
    cache = caches.caches[0]
    dev = _cuda(cache.k, "the cache")
    if _elsewhere(dev, stream):
        with _Guard(dev, stream):
            return cache_compact(caches, keep, q_indptr, max_tokens_per_seq, refs, out_lens, status)
    cs = _cache_struct(cache)
    B = cs.batch
    if out_lens is None:
        out_lens = torch.empty((B,), dtype=torch.int32, device=dev)
    if keep.dim() != 2:
        raise ValueError("keep must be [batch, k_max]")
    k_max = keep.shape[1]
    if k_max < 1:
        raise TsdError(TSD_ERR_INVALID_ARGUMENT, "keep must have room for one draft")
    kp = _int32(keep, "keep", dev, (B, k_max))
    if q_indptr is None:
        n, ip, T = 1, None, B
    else:   # only its gaps count: nothing here is indexed by token, so there is no number of tokens to keep within
        n, ip, T = int(max_tokens_per_seq), _int32(q_indptr, "q_indptr", dev, (B + 1,)), 0x7FFFFFFF
    layers = caches.c_layers
    st = _LIB.tsd_cache_compact(cs, len(layers), layers, ip, T, n, kp, k_max,
                                None if refs is None else _refs(refs, cache, dev),
                                _int32(out_lens, "out_lens", dev, (B,)), _status_ptr(status, dev), _raw_stream(dev))
    if st:
        raise TsdError(st, "tsd_cache_compact")
    return out_lens
