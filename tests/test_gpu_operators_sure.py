"""The logits that targets name are the ones under the log-sum, bit for bit: rows that
are sure of their label have loss and gradients of exactly zero, and distillation
from one entry is cross entropy."""
import pytest

import lossless_entropy_coded_huffman_amd as dfh
from test_gpu_operators import dev, head_and_x

pytestmark = pytest.mark.gpu
SIZES = [(1, 5, 72), (7, 3001, 1416), (40, 300, 4096), (300, 70, 136), (517, 1031, 200), (1100, 40, 2056)]


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def both(torch, x, head, labels, reduction, temp=1.0):
    """The loss by both calls, with gradients to x and head."""
    D = dev(torch)
    out = []
    for call in ("vocab", "distill"):
        xs, hs = x.to(D).requires_grad_(), head.to(D).requires_grad_()
        if call == "vocab":
            loss = dfh.vocab_loss(xs, hs, labels.to(D), reduction=reduction)
        else:
            teacher = torch.full((x.shape[0], 1), 3.0, device=D)
            loss = dfh.distill_loss(xs, hs, teacher, labels.to(D)[:, None], reduction=reduction)
        out.append((loss.detach(),) + torch.autograd.grad(loss.sum(), (xs, hs)))
    return out


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("m,v,h", SIZES)
def test_rows_that_are_sure(torch, m, v, h, dtype):
    dt = getattr(torch, dtype)
    g = torch.Generator().manual_seed(m)
    head = (torch.randn(v, h, generator=g) * (72 / h) ** 0.5).to(dt)
    labels = torch.randint(0, v, (m,), generator=g)
    x = (head[labels].float() * 8 * (torch.rand(m, 1, generator=g) + 1)).to(dt)
    z = x.double() @ head.double().t()
    top = z.gather(1, labels[:, None])
    gap = (top - z).scatter(1, labels[:, None], float("inf")).amin(1)
    assert float(gap.min()) > 110   # e^-110 is less than float32's smallest number
    for out in both(torch, x, head, labels, "none"):
        assert all(float(t.abs().max()) == 0.0 for t in out)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("m,v,h", SIZES)
def test_distillation_from_one_entry_is_cross_entropy(torch, m, v, h, dtype):
    dt = getattr(torch, dtype)
    x, head = head_and_x(torch, m, v, h, dt, seed=m + v)
    labels = torch.randint(0, v, (m,), generator=torch.Generator().manual_seed(v))
    a, b = both(torch, x, head, labels, "none")
    assert float(a[0].min()) > 0
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("temp", [0.5, 0.7, 3.0])
def test_sure_rows_at_other_temperatures(torch, temp):
    m, v, h = 60, 500, 264
    g = torch.Generator().manual_seed(2)
    head = (torch.randn(v, h, generator=g) * (72 / h) ** 0.5).to(torch.bfloat16)
    labels = torch.randint(0, v, (m,), generator=g)
    x = (head[labels].float() * 8 * temp).to(torch.bfloat16)
    z = x.double() @ head.double().t() / temp
    gap = (z.gather(1, labels[:, None]) - z).scatter(1, labels[:, None], float("inf")).amin(1)
    assert float(gap.min()) > 110
    D = dev(torch)
    xs, hs = x.to(D).requires_grad_(), head.to(D).requires_grad_()
    loss = dfh.distill_loss(xs, hs, torch.zeros(m, 1, device=D), labels.to(D)[:, None], temperature=temp, reduction="none")
    grads = torch.autograd.grad(loss.sum(), (xs, hs))
    assert all(float(t.abs().max()) == 0.0 for t in (loss.detach(), *grads))
