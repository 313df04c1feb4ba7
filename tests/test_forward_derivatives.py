"""Derivatives of a resident block beyond the first gradient: a gradient of a
gradient, forward mode and torch.func's transforms give what the block of plain
batched products gives.  No GPU needed."""
import contextlib

import pytest
import torch

from lossless_entropy_coded_huffman_amd import forward as fw

SHAPE = fw.BlockShape(hidden=32, heads=4, kv_heads=2, ffn=48)
E = 2.0 ** -24


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)
    return {name: torch.randn(r, c, generator=g) * 0.2 for name, r, c in SHAPE.matrices()}


def acts(seed, tokens=5):
    return torch.randn(tokens, SHAPE.hidden, generator=torch.Generator().manual_seed(seed))


def block(x, w):
    return fw.block_forward(x, w, SHAPE)


class PlainBmm:
    apply = staticmethod(torch.bmm)


def both(monkeypatch, f):
    """(f through the block, f through a block of torch.bmm)."""
    got = f()
    monkeypatch.setattr(fw, "_Bmm", PlainBmm)
    want = f()
    return got, want


def close(got, want):
    # the same products, summed in another order at most: a few thousand float32
    # roundings of values up to the largest
    assert float((got - want).abs().max()) <= 4096 * E * float(want.abs().max())


def test_gradient_of_a_gradient(monkeypatch):
    w, x0, v, u = weights(), acts(1), acts(2), acts(3)

    def hvp():
        x = x0.clone().requires_grad_()
        g, = torch.autograd.grad((block(x, w) * u).sum(), x, create_graph=True)
        return torch.autograd.grad((g * v).sum(), x)[0]

    got, want = both(monkeypatch, hvp)
    close(got, want)


def test_gradient_of_a_gradient_is_the_difference_quotient():
    # float32 inside the block: a step of 2^-8 leaves 2^-24 / 2^-8 of rounding and
    # 2^-16 of curvature, far under the 3% that a lost term would have to stay under
    w, x0, v, u = weights(), acts(1), acts(2), acts(3)

    def grad(x):
        x = x.clone().requires_grad_()
        return torch.autograd.grad((block(x, w) * u).sum(), x)[0]

    x = x0.clone().requires_grad_()
    g, = torch.autograd.grad((block(x, w) * u).sum(), x, create_graph=True)
    got, = torch.autograd.grad((g * v).sum(), x)
    h = 2.0 ** -8
    num = (grad(x0 + h * v) - grad(x0 - h * v)) / (2 * h)
    assert float((got - num).abs().max()) <= 0.03 * float(num.abs().max())


def test_forward_mode(monkeypatch):
    w, x0, v = weights(), acts(1), acts(2)
    got, want = both(monkeypatch, lambda: torch.func.jvp(lambda x: block(x, w), (x0,), (v,))[1])
    close(got, want)


def test_forward_over_reverse(monkeypatch):
    w, x0, v, u = weights(), acts(1), acts(2), acts(3)
    got, want = both(monkeypatch, lambda: torch.func.jvp(
        torch.func.grad(lambda x: (block(x, w) * u).sum()), (x0,), (v,))[1])
    close(got, want)


@pytest.mark.parametrize("transform", ["grad", "vmap", "vmap of grad", "grad of vmap"])
def test_transforms(monkeypatch, transform):
    w, u = weights(), acts(3)
    xs = torch.stack([acts(i) for i in range(3)])

    def one(x):
        return (block(x, w) * u).sum()

    f = {"grad": lambda: torch.func.grad(one)(xs[0]),
         "vmap": lambda: torch.func.vmap(lambda x: block(x, w))(xs),
         "vmap of grad": lambda: torch.func.vmap(torch.func.grad(one))(xs),
         "grad of vmap": lambda: torch.func.grad(lambda a: torch.func.vmap(one)(a).pow(2).sum())(xs)}[transform]
    got, want = both(monkeypatch, f)
    close(got, want)


class Cubes:
    """Blocks of x^3 in place of a QuantizedBlocks."""

    def _turn(self):
        return contextlib.nullcontext()

    def _run(self, i, x):
        return x.pow(3)


def test_second_gradient_of_quantised_blocks_is_refused():
    # x goes round the block too, as in a residual connection: a node that autograd
    # prunes cannot refuse
    x = torch.arange(1.0, 5.0).requires_grad_()

    def f():
        return (x * x).sum() + fw._QuantizedBlock.apply(x, Cubes(), 0).sum()

    plain, = torch.autograd.grad(f(), x)
    first, = torch.autograd.grad(f(), x, create_graph=True)
    assert torch.equal(first, plain) and torch.equal(plain, (2 * x + 3 * x * x).detach())
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first.sum(), x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_under_autocast(monkeypatch, dtype):
    # the products run in autocast's type, and so do their gradients
    w, u = {k: v.to(dtype) for k, v in weights().items()}, acts(3)

    def grad():
        x = acts(1).to(dtype).requires_grad_()
        with torch.autocast("cpu", dtype=torch.bfloat16):
            y = block(x, w)
        return torch.autograd.grad((y.float() * u).sum(), x)[0].float()

    got, want = both(monkeypatch, grad)
    # the same sums in 16 bits: a few dozen roundings of 2^-8 at most
    assert float((got - want).abs().max()) <= 64 * 2.0 ** -8 * float(want.abs().max())
