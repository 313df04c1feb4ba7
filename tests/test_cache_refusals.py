"""Refusals of the cache's C ABI, which come before anything is enqueued.  The pointers
are never read.  No GPU needed."""
import ctypes

import pytest
import torch

import lossless_entropy_coded_huffman_amd as dfh
from lossless_entropy_coded_huffman_amd import dfh as abi

P = 1 << 20          # an aligned address that nothing reads
ARG = -1


def cache(**kw):
    f = dict(type=0, bits=8, page_size=64, kv_heads=8, head_dim=128, pages=10, k=P, v=P, k_scales=P, v_scales=P)
    f.update(kw)
    return abi.df_cache(**f)


def batch(**kw):
    f = dict(seqs=3, width=4, table_stride=4, tables=P, lengths=P, starts=P, max_new=0)
    f.update(kw)
    return abi.df_cache_batch(**f)


def write(c, b, k=P, kt=1024, kh=128, v=P, vt=1024, vh=128, tokens=5):
    return dfh.lib().df_cache_write(ctypes.byref(c), ctypes.byref(b), k, kt, kh, v, vt, vh, tokens, None)


def read(c, b, k=P, v=P, tokens=5):
    return dfh.lib().df_cache_read(ctypes.byref(c), ctypes.byref(b), k, v, tokens, None)


BAD_CACHE = [dict(type=2), dict(type=-1), dict(bits=4), dict(bits=0), dict(page_size=8), dict(page_size=48),
             dict(page_size=512), dict(page_size=0), dict(kv_heads=0), dict(kv_heads=257), dict(head_dim=96),
             dict(head_dim=512), dict(pages=0), dict(pages=(1 << 26) + 1), dict(k=None), dict(v=None), dict(k=P + 8),
             dict(v=P + 4), dict(k_scales=None), dict(v_scales=None), dict(k_scales=P + 2), dict(v_scales=P + 1)]
BAD_BATCH = [dict(seqs=(1 << 16) + 1), dict(width=0), dict(width=(1 << 22) + 1, table_stride=1 << 23),
             dict(table_stride=3), dict(table_stride=(1 << 30) + 1), dict(tables=None), dict(lengths=None),
             dict(starts=None), dict(tables=P + 2), dict(lengths=P + 1), dict(starts=P + 3)]


@pytest.mark.parametrize("kw", BAD_CACHE)
def test_bad_cache(kw):
    assert write(cache(**kw), batch()) == read(cache(**kw), batch()) == ARG


@pytest.mark.parametrize("kw", BAD_BATCH)
def test_bad_batch(kw):
    assert write(cache(), batch(**kw)) == read(cache(), batch(**kw)) == ARG


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 2), dict(kt=1020), dict(kh=4),
                                dict(vt=12), dict(vh=130), dict(kt=(1 << 30) + 8), dict(vh=(1 << 30) + 8),
                                dict(tokens=(1 << 24) + 1)])
def test_bad_write(kw):
    assert write(cache(), batch(), **kw) == ARG


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 2), dict(tokens=(1 << 24) + 1)])
def test_bad_read(kw):
    assert read(cache(), batch(), **kw) == ARG


def test_nothing_to_do_enqueues_nothing():
    assert write(cache(), batch(), tokens=0, k=None, v=None) == 0
    assert write(cache(), batch(seqs=0, tables=None, lengths=None, starts=None)) == 0
    assert read(cache(), batch(), tokens=0, k=None, v=None) == 0


def test_host_tensors_are_refused():
    with pytest.raises(ValueError):
        dfh.KVCache(2, 1, 64, device="cpu")
    t = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dfh.CacheBatch(t, t[0, :1], t[0])


def attend(c, b, q=P, qt=4096, qh=128, tokens=5, heads=32, scale=0.1, window=0, out=P, lse=None, ws=P, nbytes=1 << 40):
    return dfh.lib().df_cached_attention(ctypes.byref(c), ctypes.byref(b), q, qt, qh, tokens, heads, scale, window, out,
                                         lse, ws, nbytes, None)


def space(c, b, tokens=5, heads=32, window=0):
    return dfh.lib().df_cached_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), tokens, heads, window)


@pytest.mark.parametrize("kw", BAD_CACHE)
def test_bad_cache_of_attention(kw):
    assert attend(cache(**kw), batch()) == ARG and space(cache(**kw), batch()) == 0


@pytest.mark.parametrize("kw", BAD_BATCH)
def test_bad_batch_of_attention(kw):
    assert attend(cache(), batch(**kw)) == ARG and space(cache(), batch(**kw)) == 0


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=P + 8), dict(qt=4100), dict(qh=4), dict(qt=(1 << 30) + 8), dict(out=None),
                                dict(out=P + 8), dict(lse=P + 2), dict(heads=0), dict(heads=12), dict(heads=8 * 257),
                                dict(tokens=(1 << 24) + 1), dict(tokens=1 << 23, heads=2048), dict(scale=0.0),
                                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
                                dict(ws=None), dict(ws=P + 16), dict(nbytes=100)])
def test_bad_attention(kw):
    # 4000 pages of 64: the keys are split, and a workspace is needed
    assert attend(cache(), batch(width=4000, table_stride=4000), **kw) == ARG


def test_attention_sizes():
    assert attend(cache(), batch(), tokens=0, q=None, out=None) == 0
    # partial sums take what the rows need, and never more than 256 MiB and a little for their statistics
    small = space(cache(), batch(seqs=1, width=16, table_stride=16, max_new=1), tokens=1)
    assert 0 < small <= 512 * 32 * 130 * 4 + 512
    for seqs, tokens, width in ((1, 1, 1 << 22), (64, 64, 4096), (65536, 65536, 100), (1, 16384, 1 << 16), (300, 40000, 2000)):
        assert space(cache(), batch(seqs=seqs, width=width, table_stride=width), tokens=tokens) <= 2 * (256 << 20) + 4096
