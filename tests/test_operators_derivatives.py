"""What the operators' derivatives do with a second differentiation and with
forward mode: the autograd functions over plain stand-ins for the kernels, so no
GPU is needed.  In every second derivative x is reached by another path too, as a
residual connection does: a node that autograd prunes cannot refuse."""
import gc
import weakref

import pytest
import torch
from torch.autograd import forward_ad

from lossless_entropy_coded_huffman_amd import ops


class Dense:
    """A weight matrix in place of a U4Matrix."""

    def __init__(self, weight):
        self.weight = weight

    def _tensors(self):
        return (self.weight, None)


@pytest.fixture
def dense(monkeypatch):
    g = torch.Generator().manual_seed(0)
    w = Dense(torch.randn(7, 5, generator=g, dtype=torch.float64))
    monkeypatch.setattr(ops, "_linear", lambda x, w, stream: x @ w.weight.t())
    monkeypatch.setattr(ops, "_linear_grad", lambda dy, w, stream: dy @ w.weight, raising=False)
    return w


def second(f, x0, v):
    x = x0.clone().requires_grad_()
    g, = torch.autograd.grad(f(x), x, create_graph=True)
    return torch.autograd.grad((g * v).sum(), x)[0]


def test_second_gradient_of_linear_u4(dense):
    g = torch.Generator().manual_seed(1)
    x, v = (torch.randn(3, 5, generator=g, dtype=torch.float64) for _ in range(2))
    got = second(lambda x: (x * x).sum() + ops.linear_u4(x, dense).pow(3).sum(), x, v)
    want = second(lambda x: (x * x).sum() + (x @ dense.weight.t()).pow(3).sum(), x, v)
    # a dozen float64 roundings of a sum of 35 terms
    assert float((got - want).abs().max()) <= 2.0 ** -40 * float(want.abs().max())
    y = x.clone().requires_grad_()
    assert torch.autograd.gradcheck(lambda x: ops.linear_u4(x, dense), y)
    assert torch.autograd.gradgradcheck(lambda x: ops.linear_u4(x, dense), y)


def test_linear_u4_grad_is_differentiable(dense):
    g = torch.Generator().manual_seed(2)
    dy = torch.randn(3, 7, generator=g, dtype=torch.float64).requires_grad_()
    assert torch.autograd.gradcheck(lambda d: ops.linear_u4_grad(d, dense), dy)
    assert not ops.linear_u4_grad(dy.detach(), dense).requires_grad


def test_changed_weights_are_refused_by_a_second_gradient(dense):
    x = torch.ones(2, 5, dtype=torch.float64, requires_grad=True)
    g, = torch.autograd.grad(ops.linear_u4(x, dense).pow(2).sum(), x, create_graph=True)
    dense.weight.mul_(2.0)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), x)


class Squares:
    """A loss call over [rows, hidden] states and a head: sum of (x head^T)^2, in
    place of a _Loss."""

    done = None

    def __init__(self, x, head):
        self.inputs = (x, head)

    def forward(self, stream):
        x, head = self.inputs
        return (x @ head.t()).pow(2).sum(), (torch.zeros(1),)

    def grads(self, kept, gout, want_x, want_head):
        x, head = (t.detach() for t in kept[:2])
        z = 2 * gout * (x @ head.t())
        return z @ head if want_x else None, z.t() @ x if want_head else None


@pytest.mark.parametrize("leaf", ["x", "head"])
def test_second_gradients_of_losses_are_refused(leaf):
    g = torch.Generator().manual_seed(3)
    x, head = (torch.randn(s, 5, generator=g, dtype=torch.float64) for s in (3, 7))
    x, head = x.requires_grad_(leaf == "x"), head.requires_grad_(leaf == "head")
    t = x if leaf == "x" else head
    loss = ops._run_loss(Squares(x, head), None)
    plain, = torch.autograd.grad((t * t).sum() + loss, t, retain_graph=True)
    # the first gradient stays what it is under create_graph
    first, = torch.autograd.grad((t * t).sum() + loss, t, create_graph=True)
    assert torch.equal(first, plain)
    want = (x @ head.t()) * 2
    want = (want @ head if leaf == "x" else want.t() @ x) + 2 * t
    assert float((first - want).abs().max()) <= 2.0 ** -44 * float(want.abs().max())
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first.sum(), t)


def test_forward_mode_is_refused(dense):
    # a tangent that no operator would carry on is not dropped
    x, dy, t = (torch.ones(3, n, dtype=torch.float64) for n in (5, 7, 5))
    head = torch.ones(7, 5, dtype=torch.float64)
    calls = [(lambda a: ops.linear_u4(a, dense), x, t), (lambda a: ops.linear_u4_grad(a, dense), dy, torch.ones_like(dy)),
             (lambda a: ops._run_loss(Squares(a, head), None), x, t),
             (lambda a: ops._run_loss(Squares(x, a), None), head, torch.ones_like(head))]
    for f, primal, tangent in calls:
        with forward_ad.dual_level():
            dual = forward_ad.make_dual(primal, tangent)
            for a in (dual, dual.detach().requires_grad_() * 1 + dual * 0):
                with pytest.raises(NotImplementedError):
                    f(a)
            f(primal)   # no tangent: as ever
            with torch.no_grad(), pytest.raises(NotImplementedError):
                f(dual)
        with pytest.raises(NotImplementedError):
            torch.func.jvp(f, (primal,), (tangent,))
    # forward over reverse, where only the gradient that comes in has a tangent
    for f in (lambda a: ops.linear_u4(a, dense), lambda a: ops._run_loss(Squares(a, head), None)):
        a = x.clone().requires_grad_()
        y = f(a)
        with forward_ad.dual_level():
            dual = forward_ad.make_dual(torch.ones_like(y).detach(), torch.ones_like(y).detach())
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(y, a, dual)


def test_a_loss_leaves_its_inputs_to_autograd():
    # with hooks that put what is saved elsewhere, nothing else holds the inputs
    g = torch.Generator().manual_seed(4)
    base, head = (torch.randn(s, 5, generator=g, dtype=torch.float64) for s in (3, 7))
    leaf = base.clone().requires_grad_()
    x = leaf * 2
    ref = weakref.ref(x)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.numpy(force=True).copy(), torch.from_numpy):
        loss = ops._run_loss(Squares(x, head), None)
    del x
    gc.collect()
    assert ref() is None
    got, = torch.autograd.grad(loss, leaf)
    assert torch.equal(got, 2 * ((2 * (2 * base @ head.t())) @ head))
