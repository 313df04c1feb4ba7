"""Refusals of the operators' C ABI, which come before anything is enqueued, and
the sizes they ask for.  The pointers are never read.  No GPU needed."""
import ctypes

import pytest
import torch

import lossless_entropy_coded_huffman_amd as dfh
from lossless_entropy_coded_huffman_amd import dfh as abi

P = 1 << 20          # an aligned address that nothing reads
ARG = -1


def matrix(**kw):
    f = dict(rows=16, cols=64, group_size=32, scale_type=0, scale_stride=2, zero_stride=2, packed=P, scales=P, zeros=P)
    f.update(kw)
    return abi.df_u4_matrix(**f)


def linear(w, ty=0, x=P, rows=2, xs=64, y=P, ws=P, nbytes=1 << 40, fn="df_linear_u4"):
    return getattr(dfh.lib(), fn)(ctypes.byref(w), ty, x, rows, xs, y, ws, nbytes, None)


@pytest.mark.parametrize("kw", [dict(rows=0), dict(rows=(1 << 21) + 1), dict(cols=0), dict(cols=60),
                                dict(cols=(1 << 20) + 8), dict(group_size=0), dict(group_size=16), dict(group_size=48),
                                dict(scale_type=3), dict(scale_type=-1), dict(packed=None), dict(packed=P + 2),
                                dict(scales=None), dict(scales=P + 1), dict(scale_type=2, scales=P + 2)])
def test_bad_matrix(kw):
    for fn in ("df_linear_u4", "df_linear_u4_grad"):
        assert linear(matrix(**kw), fn=fn) == ARG


@pytest.mark.parametrize("kw", [dict(ty=2), dict(ty=7), dict(x=None), dict(x=P + 8), dict(xs=56), dict(xs=68),
                                dict(xs=(1 << 21) + 8), dict(y=None), dict(y=P + 8), dict(rows=(1 << 24) + 1),
                                dict(rows=513, ws=None), dict(rows=513, nbytes=100), dict(rows=513, ws=P + 16)])
def test_bad_linear_call(kw):
    assert linear(matrix(), **kw) == ARG


@pytest.mark.parametrize("kw", [dict(ty=2), dict(x=None), dict(x=P + 8), dict(xs=8), dict(xs=20), dict(y=None),
                                dict(y=P + 2), dict(ws=None), dict(nbytes=100), dict(ws=P + 16)])
def test_bad_linear_grad_call(kw):
    args = dict(xs=16)
    args.update(kw)
    assert linear(matrix(), fn="df_linear_u4_grad", **args) == ARG


def test_no_rows_enqueue_nothing():
    assert linear(matrix(), rows=0, x=None, y=None, ws=None, nbytes=0) == 0
    assert linear(matrix(), rows=0, x=None, y=None, ws=None, nbytes=0, fn="df_linear_u4_grad") == 0


def loss(**kw):
    f = dict(type=0, reduce=2, rows=4, vocab=100, hidden=64, x_stride=64, head_stride=64, x=P, head=P, labels=P,
             ignore_index=-100, index=None, teacher=None, teacher_type=0, top=0, index_stride=0, teacher_stride=0,
             temperature=1.0)
    f.update(kw)
    return abi.df_loss(**f)


DISTILL = dict(top=4, labels=None, index=P, teacher=P, index_stride=4, teacher_stride=4, temperature=2.0)
BAD_LOSS = [dict(type=2), dict(reduce=3), dict(rows=1 << 24), dict(vocab=0), dict(vocab=(1 << 21) + 1), dict(hidden=0),
            dict(hidden=60, x_stride=64), dict(hidden=(1 << 17) + 8, x_stride=1 << 18, head_stride=1 << 18),
            dict(x_stride=56), dict(x_stride=68), dict(head_stride=56), dict(head_stride=(1 << 21) + 8), dict(x=None),
            dict(x=P + 8), dict(head=None), dict(head=P + 2), dict(labels=None), dict(labels=P + 4),
            dict(temperature=2.0), dict(DISTILL, top=1025), dict(DISTILL, index=None), dict(DISTILL, index=P + 4),
            dict(DISTILL, teacher=None), dict(DISTILL, teacher_type=2, teacher=P + 2), dict(DISTILL, teacher_type=4),
            dict(DISTILL, temperature=0.0), dict(DISTILL, temperature=-1.0), dict(DISTILL, temperature=float("inf")), dict(DISTILL, temperature=5e-4), dict(DISTILL, temperature=2000.0),
            dict(DISTILL, temperature=float("nan"))]


@pytest.mark.parametrize("kw", BAD_LOSS)
def test_bad_loss(kw):
    L, d = dfh.lib(), loss(**kw)
    r = ctypes.byref(d)
    assert L.df_vocab_loss(r, P, P, P, 1 << 40, None) == ARG
    assert L.df_vocab_loss_grad(r, P, P, P, P, P, 1 << 40, None) == ARG
    assert L.df_loss_saved_bytes(r) == L.df_loss_workspace_bytes(r) == L.df_loss_grad_workspace_bytes(r, 1) == 0


@pytest.mark.parametrize("base", [{}, DISTILL])
def test_bad_loss_call(base):
    L, d = dfh.lib(), loss(**base)
    r = ctypes.byref(d)
    big = 1 << 40
    for a in ((None, P, P, big), (P, None, P, big), (P, P, None, big), (P, P, P, 16), (P, P, P + 16, big),
              (P, P + 2, P, big), (P + 2, P, P, big)):
        assert L.df_vocab_loss(r, *a, None) == ARG
    for a in ((None, P, P, P, P, big), (P, None, P, P, P, big), (P, P, None, None, P, big), (P, P, P + 8, P, P, big),
              (P, P, P, P + 8, P, big), (P, P, P, P, None, big), (P, P, P, P, P, 16), (P, P, P, P, P + 64, big)):
        assert L.df_vocab_loss_grad(r, *a, None) == ARG


def test_sizes():
    L = dfh.lib()
    w = matrix(rows=4096, cols=14336, group_size=128)
    assert L.df_linear_u4_workspace_bytes(ctypes.byref(w), 1) == 0
    assert 0 < L.df_linear_u4_workspace_bytes(ctypes.byref(w), 64) < 64 * 4096 * 4 * 64
    assert L.df_linear_u4_workspace_bytes(ctypes.byref(w), 2048) >= 0
    # the logits of a training step are never whole in the workspace
    d = loss(rows=4096, vocab=128256, hidden=4096, x_stride=4096, head_stride=4096)
    assert 0 < L.df_loss_workspace_bytes(ctypes.byref(d)) < 4096 * 128256 * 2 // 8
    assert 0 < L.df_loss_grad_workspace_bytes(ctypes.byref(d), 1) < 4096 * 128256 * 2
    assert L.df_loss_saved_bytes(ctypes.byref(d)) == 16 + 4096 * 3 * 4
    d = loss(**dict(DISTILL, rows=10))
    assert L.df_loss_saved_bytes(ctypes.byref(d)) == 16 + 10 * 6 * 4


def test_host_tensors_are_refused():
    # the binding has no CPU path
    with pytest.raises(ValueError):
        dfh.U4Matrix(torch.zeros(64, dtype=torch.uint8), torch.ones(2, 2), cols=64, group_size=32)
    with pytest.raises(ValueError):
        dfh.vocab_loss(torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(5, 64, dtype=torch.bfloat16),
                       torch.zeros(2, dtype=torch.int64))
