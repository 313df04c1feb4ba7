"""Refusals of the C ABI of products in 8-bit integers, which come before anything is
enqueued, and the sizes they ask for.  The pointers are never read.  No GPU needed."""
import ctypes

import pytest
import torch

import lossless_entropy_coded_huffman_amd as dfh
from lossless_entropy_coded_huffman_amd import dfh as abi

P = 1 << 20          # an aligned address that nothing reads
ARG = -1
BIG = 1 << 40


def matrix(**kw):
    f = dict(rows=16, cols=64, scale_type=0, scale_stride=1, zero_stride=1, codes=P, scales=P, zeros=P)
    f.update(kw)
    return abi.df_u8_matrix(**f)


def linear(w, ty=0, x=P, rows=2, xs=64, y=P, ws=P, nbytes=BIG):
    return dfh.lib().df_linear_u8(ctypes.byref(w), ty, x, rows, xs, y, ws, nbytes, None)


def by_codes(w, ty=0, x=P, scales=P, rows=2, xs=64, y=P, ws=P, nbytes=BIG):
    return dfh.lib().df_linear_u8_codes(ctypes.byref(w), ty, x, scales, rows, xs, y, ws, nbytes, None)


@pytest.mark.parametrize("kw", [dict(rows=0), dict(rows=(1 << 21) + 1), dict(cols=0), dict(cols=8), dict(cols=72),
                                dict(cols=65552), dict(scale_type=3), dict(scale_type=-1), dict(codes=None),
                                dict(codes=P + 8), dict(scales=None), dict(scales=P + 1),
                                dict(scale_type=2, scales=P + 2)])
def test_bad_matrix(kw):
    assert linear(matrix(**kw)) == by_codes(matrix(**kw)) == ARG
    assert dfh.lib().df_linear_u8_workspace_bytes(ctypes.byref(matrix(**kw)), 100, 0) == 0


@pytest.mark.parametrize("kw", [dict(ty=2), dict(ty=7), dict(x=None), dict(x=P + 8), dict(xs=56), dict(xs=68),
                                dict(xs=(1 << 21) + 16), dict(y=None), dict(y=P + 8), dict(rows=(1 << 24) + 1),
                                dict(rows=9, ws=None), dict(rows=9, nbytes=100), dict(rows=9, ws=P + 16)])
def test_bad_call(kw):
    assert linear(matrix(), **kw) == ARG
    assert by_codes(matrix(), **kw) == ARG


@pytest.mark.parametrize("kw", [dict(scales=None), dict(scales=P + 2), dict(xs=72)])
def test_bad_call_with_codes(kw):
    assert by_codes(matrix(), **kw) == ARG


@pytest.mark.parametrize("kw", [dict(type=2), dict(x=None), dict(x=P + 8), dict(rows=(1 << 24) + 1), dict(cols=0),
                                dict(cols=24), dict(cols=65552, stride=65552), dict(stride=56), dict(stride=68),
                                dict(stride=(1 << 21) + 8), dict(codes=None), dict(codes=P + 8), dict(scales=None),
                                dict(scales=P + 2)])
def test_bad_quantising(kw):
    a = dict(type=0, x=P, rows=3, cols=64, stride=64, codes=P, scales=P)
    a.update(kw)
    assert dfh.lib().df_quantize_rows(*a.values(), None) == ARG


def test_no_rows_enqueue_nothing():
    assert linear(matrix(), rows=0, x=None, y=None, ws=None, nbytes=0) == 0
    assert by_codes(matrix(), rows=0, x=None, scales=None, y=None, ws=None, nbytes=0) == 0
    assert dfh.lib().df_quantize_rows(0, None, 0, 64, 64, None, None, None) == 0


def test_sizes():
    def need(rows, cols, m, codes=0):
        return dfh.lib().df_linear_u8_workspace_bytes(ctypes.byref(matrix(rows=rows, cols=cols)), m, codes)
    assert need(4096, 14336, 4) == 0 and need(4096, 61440, 1) == 0
    assert need(4096, 65536, 1) >= 65536
    assert 2048 * 4096 <= need(14336, 4096, 2048) < 2 * 2048 * 4096
    assert need(14336, 4096, 2048, 1) <= need(14336, 4096, 2048) - 2048 * 4096


def test_host_tensors_are_refused():
    with pytest.raises(ValueError):
        dfh.U8Matrix(torch.zeros(16, 64, dtype=torch.uint8), torch.ones(16), cols=64)
    with pytest.raises(ValueError):
        dfh.quantize_rows(torch.zeros(2, 64, dtype=torch.bfloat16))
