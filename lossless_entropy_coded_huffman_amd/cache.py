"""A paged cache of keys and values, through the C ABI (include/dfh.h):

* ``KVCache`` holds the pages, in 16 bits or quantised to 8 with a scale for each
  token and head; ``CacheBatch`` says which sequences a call is about;
* ``cache_write`` puts the keys and values of new tokens into the pages,
  ``cache_read`` gives them back;
* ``cached_attention`` is the attention of the new tokens over all that their
  sequences hold.

A step of several sequences, each with any number of new tokens (a prompt, a part of
one, a single token, none), is one batch: rows starts[s] .. starts[s + 1] - 1 of the
step's tensors are the new tokens of sequence s, the last ones of its lengths[s]
positions.  Streams, workspaces and captures are as in ``ops``: everything is enqueued
on ``stream`` (default: the current stream of the cache's device) and returns without
synchronising.  What the batch's tensors hold is read when the call runs, so a captured
step is replayed after they were changed in place.  Nothing here has a gradient:
inputs that require one are refused.
"""
from __future__ import annotations

import ctypes

import torch

from . import dfh
from .ops import _TYPES, _current_device, _launch, _no_gradient, _on, _p, _raw_stream, _workspace


class KVCache:
    """Pages of keys and values on the device (df_cache).

    k and v: [pages, kv_heads, page_size, head_dim], in dtype (bfloat16 or float16)
    with bits=16, int8 codes with bits=8, then with float32 k_scales and v_scales
    [pages, kv_heads, page_size]; all start as zeros.  page_size is a power of two from
    16 to 256, head_dim 32, 64, 128 or 256, kv_heads at most 256."""

    def __init__(self, pages: int, kv_heads: int, head_dim: int, *, page_size: int = 64, dtype=torch.bfloat16,
                 bits: int = 16, device=None):
        pages, kv_heads, head_dim, page_size, bits = (int(v) for v in (pages, kv_heads, head_dim, page_size, bits))
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("dtype must be bfloat16 or float16, got %s" % dtype)
        if bits not in (16, 8):
            raise ValueError("bits must be 16 or 8, got %d" % bits)
        if page_size < 16 or page_size > 256 or page_size & (page_size - 1):
            raise ValueError("page_size must be a power of two from 16 to 256, got %d" % page_size)
        if head_dim not in (32, 64, 128, 256):
            raise ValueError("head_dim must be 32, 64, 128 or 256, got %d" % head_dim)
        if not 1 <= kv_heads <= 256:
            raise ValueError("kv_heads must lie in 1 .. 256, got %d" % kv_heads)
        if not 1 <= pages <= 1 << 26:
            raise ValueError("pages must lie in 1 .. 2^26, got %d" % pages)
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise ValueError("a cache lies on the device, got %s" % device)
        shape = (pages, kv_heads, page_size, head_dim)
        kept = torch.int8 if bits == 8 else dtype
        self.k, self.v = (torch.zeros(shape, dtype=kept, device=device) for _ in range(2))
        self.k_scales, self.v_scales = (torch.zeros(shape[:3], dtype=torch.float32, device=device) if bits == 8 else None
                                        for _ in range(2))
        self.pages, self.kv_heads, self.head_dim, self.page_size = pages, kv_heads, head_dim, page_size
        self.dtype, self.bits, self.device = dtype, bits, self.k.device
        self.view = dfh.df_cache(_TYPES[dtype], bits, page_size, kv_heads, head_dim, pages, self.k.data_ptr(),
                                 self.v.data_ptr(), 0 if bits == 16 else self.k_scales.data_ptr(),
                                 0 if bits == 16 else self.v_scales.data_ptr())
        self._ref = ctypes.byref(self.view)

    def _tensors(self):
        return (self.k, self.v, self.k_scales, self.v_scales)


class CacheBatch:
    """The sequences of a step (df_cache_batch; the tensors are borrowed and kept
    alive), int32 on the cache's device:

    tables [seqs, width]: the pages of each sequence, position p in page
    tables[s, p // page_size]; lengths [seqs]: its positions, new tokens counted;
    starts [seqs + 1]: where its new tokens begin in the step's tensors, from 0 on,
    not falling.  max_new: the most new tokens of a sequence, where the program knows
    it; it only chooses kernels, any batch is computed right without or with a wrong one.

    A position before 0 or outside the table, and a page outside the pool, are tokens
    that are not there: not written, read back as zeros, not attended to.  Sequences may share
    pages that they read; a position that a step writes has one owner."""

    def __init__(self, tables: torch.Tensor, lengths: torch.Tensor, starts: torch.Tensor, *, max_new: int | None = None):
        if not tables.is_cuda or tables.dtype != torch.int32 or tables.dim() != 2 or tables.shape[1] < 1:
            raise ValueError("tables must be an int32 [seqs, width] tensor on the device")
        seqs, width = (int(n) for n in tables.shape)
        if seqs > 1 << 16 or width > 1 << 22:
            raise ValueError("tables must have at most 65536 rows of 2^22 pages, got %s" % (tuple(tables.shape),))
        for t, what, n in ((lengths, "lengths", seqs), (starts, "starts", seqs + 1)):
            _on(t, tables.device, what)
            if t.dtype != torch.int32 or tuple(t.shape) != (n,) or (n > 1 and t.stride(0) != 1):
                raise ValueError("%s must be a contiguous int32 tensor of %d elements" % (what, n))
        stride = tables.stride(0) if seqs > 1 else width
        if (width > 1 and tables.stride(1) != 1) or not width <= stride <= 1 << 30:
            raise ValueError("tables must have contiguous rows")
        if max_new is not None and int(max_new) < 0:
            raise ValueError("max_new must not be negative, got %d" % int(max_new))
        self.tables, self.lengths, self.starts = tables, lengths, starts
        self.seqs, self.width, self.device = seqs, width, tables.device
        self.max_new = None if max_new is None else int(max_new)
        self.view = dfh.df_cache_batch(seqs, width, stride, tables.data_ptr(), lengths.data_ptr(), starts.data_ptr(),
                                       min(self.max_new or 0, 1 << 24))
        self._ref = ctypes.byref(self.view)
        self._need = {}   # workspace bytes by shapes

    def _tensors(self):
        return (self.tables, self.lengths, self.starts)

    def positions(self, tokens: int) -> torch.Tensor:
        """int64 [tokens]: the position of each row of the step's tensors in its
        sequence, -1 for rows of no sequence; plain torch operations on the current
        stream."""
        return _positions(self.lengths, self.starts, int(tokens))


def _positions(lengths: torch.Tensor, starts: torch.Tensor, tokens: int) -> torch.Tensor:
    row = torch.arange(tokens, dtype=torch.int32, device=starts.device)
    if not len(lengths):
        return torch.full_like(row, -1, dtype=torch.int64)
    after = torch.searchsorted(starts[1:], row, right=True)
    seq = after.clamp(max=len(lengths) - 1)
    at = lengths[seq].long() - starts[1:][seq].long() + row
    return torch.where((row < starts[0]) | (row >= starts[-1]), -1, at).clamp(min=-1)


def _heads16(t: torch.Tensor) -> torch.Tensor:
    """t [tokens, heads, dim] with unit stride in dim, other strides that are multiples
    of 8 elements and at most 2^30, and a 16-byte aligned base: itself, or a copy."""
    a, b, one = t.stride()
    if one == 1 and (a | b) % 8 == 0 and a <= 1 << 30 and b <= 1 << 30 and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _enqueue(stream, dev, tensors, call):
    if stream is None and _current_device() == dev.index:
        return call(_raw_stream(dev.index))
    return _launch(stream, dev, tensors, call)


def _new_tokens(t: torch.Tensor, cache: KVCache, batch: CacheBatch, what: str, heads: int | None):
    _on(t, cache.device, what)
    if batch.device != cache.device:
        raise ValueError("the batch must lie on %s" % cache.device)
    if t.dtype != cache.dtype:
        raise TypeError("%s must be %s like the cache, got %s" % (what, cache.dtype, t.dtype))
    if t.dim() != 3 or t.shape[2] != cache.head_dim or (heads is not None and t.shape[1] != heads):
        raise ValueError("%s must be [tokens, %s, %d], got %s" % (what, "heads" if heads is None else heads, cache.head_dim,
                                                                  tuple(t.shape)))
    if t.shape[0] > 1 << 24:
        raise ValueError("%s has more than 2^24 tokens" % what)


def cache_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, batch: CacheBatch, stream=None) -> None:
    """The keys and values of the batch's new tokens, [tokens, kv_heads, head_dim] in the
    cache's dtype and any strides, into the cache's pages.  With 8 bits each token's
    head is kept as rint(127 x / max |x|) (ties to even) and the scale max |x| / 127;
    one that holds an infinity or NaN as codes 0 and the scale NaN.  Rows of no
    sequence are left out, and every other row of the pages stays as it was."""
    _no_gradient("cache_write", k, v)
    _new_tokens(k, cache, batch, "k", cache.kv_heads)
    _new_tokens(v, cache, batch, "v", cache.kv_heads)
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape, got %s and %s" % (tuple(k.shape), tuple(v.shape)))

    def call(handle):
        k2, v2 = _heads16(k), _heads16(v)
        st = dfh.lib().df_cache_write(cache._ref, batch._ref, k2.data_ptr(), k2.stride(0), k2.stride(1), v2.data_ptr(),
                                      v2.stride(0), v2.stride(1), k2.shape[0], handle)
        if st:
            dfh._check(st, "df_cache_write")

    _enqueue(stream, cache.device, (k, v) + cache._tensors() + batch._tensors(), call)


def cache_read(cache: KVCache, batch: CacheBatch, tokens: int, stream=None):
    """(k, v), [tokens, kv_heads, head_dim] in the cache's dtype: the rows that
    cache_write took for the same batch, as the cache holds them (codes times scale,
    rounded once).  starts that run over whole lengths give whole sequences.  Rows of
    no sequence are zeros."""
    tokens = int(tokens)
    if not 0 <= tokens <= 1 << 24:
        raise ValueError("tokens must lie in 0 .. 2^24, got %d" % tokens)
    if batch.device != cache.device:
        raise ValueError("the batch must lie on %s" % cache.device)

    def call(handle):
        k, v = (torch.empty((tokens, cache.kv_heads, cache.head_dim), dtype=cache.dtype, device=cache.device)
                for _ in range(2))
        st = dfh.lib().df_cache_read(cache._ref, batch._ref, k.data_ptr(), v.data_ptr(), tokens, handle)
        if st:
            dfh._check(st, "df_cache_read")
        return k, v

    return _enqueue(stream, cache.device, cache._tensors() + batch._tensors(), call)


def cached_attention(q: torch.Tensor, cache: KVCache, batch: CacheBatch, *, scale: float | None = None,
                     window: int | None = None, return_lse: bool = False, stream=None):
    """Attention of the batch's new tokens over the cache, into which their own keys and
    values are written already (cache_write with the same batch): for a token at
    position p

        out = sum_j softmax_j(scale q . k[j]) v[j]   over 0 <= j <= p, p - j < window

    q [tokens, heads, head_dim] in the cache's dtype and any strides, heads a multiple
    (up to 256) of the cache's kv_heads: head h reads key head h // (heads //
    kv_heads).  scale (positive; default head_dim ** -0.5); window: a positive count of
    positions, the token's own among them, or None for all.  Returns out like q,
    contiguous, and with return_lse the float32 [tokens, heads] logarithms of the
    rows' sums of exponentials.

    A row that sees no position (an empty sequence, a token before position 0) and a
    row of no sequence give 0, and -inf as logarithm.  What a position holds that a row
    does not see does not touch that row, infinities and NaN among it.  Sums are float32; weights
    are rounded to q's type before they multiply values, and float16 rounds 8-bit values
    as cache_read does."""
    _no_gradient("cached_attention", q)
    _new_tokens(q, cache, batch, "q", None)
    tokens, heads, dim = q.shape
    if heads < 1 or heads % cache.kv_heads or heads // cache.kv_heads > 256:
        raise ValueError("heads must be a multiple of kv_heads = %d, at most 256 times it, got %d"
                         % (cache.kv_heads, heads))
    if tokens * (heads // cache.kv_heads) > 1 << 30:
        raise ValueError("more than 2^30 rows a key head")
    scale = dim ** -0.5 if scale is None else float(scale)
    if not 0.0 < scale <= 3e38:
        raise ValueError("scale must be positive and finite, got %r" % (scale,))
    if window is not None and int(window) < 1:
        raise ValueError("window must be a positive count or None, got %r" % (window,))
    window = 0 if window is None else min(int(window), 1 << 40)
    dev = cache.device

    def call(handle):
        L = dfh.lib()
        q2 = _heads16(q)
        out = torch.empty((tokens, heads, dim), dtype=q.dtype, device=dev)
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=dev) if return_lse else None
        key = (cache.dtype, cache.kv_heads, cache.head_dim, cache.page_size, cache.bits, tokens, heads, window)
        need = batch._need.get(key)
        if need is None:
            need = L.df_cached_attention_workspace_bytes(cache._ref, batch._ref, tokens, heads, window)
            batch._need[key] = need
        ws = _workspace(need, dev) if need else None
        st = L.df_cached_attention(cache._ref, batch._ref, q2.data_ptr(), q2.stride(0), q2.stride(1), tokens, heads, scale,
                                   window, out.data_ptr(), _p(lse), _p(ws), need, handle)
        if st:
            dfh._check(st, "df_cached_attention")
        return (out, lse) if return_lse else out

    return _enqueue(stream, dev, (q,) + cache._tensors() + batch._tensors(), call)
