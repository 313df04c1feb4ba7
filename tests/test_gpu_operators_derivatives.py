"""Derivatives beyond the plain first gradient, on the GPU: a second gradient of
linear_u4 against float64, the refusals of the losses' and the blocks', and
gradients of tensors that autograd's hooks keep elsewhere."""
import pytest

import lossless_entropy_coded_huffman_amd as dfh
from lossless_entropy_coded_huffman_amd import forward as fw
from test_gpu_operators import E, dev, half_ulp, head_and_x, linear_bound, matrix, tiny, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("m", [3, 70, 530])
def test_second_gradient_of_linear_u4(torch, m, dtype):
    # f(x) = |linear(x)|^2 / 2, so H v = (v W^T) W; x goes round it too
    dt, D = getattr(torch, dtype), dev(torch)
    n, k = 72, 136
    w, w64, s64 = matrix(torch, n, k, 32, "fp32", seed=m)
    g = torch.Generator().manual_seed(m)
    v = torch.randn(m, k, generator=g).to(dt)
    x = torch.randn(m, k, generator=g).to(dt).to(D).requires_grad_()
    f = dfh.linear_u4(x, w).float().pow(2).sum() / 2 + (x.float() * 0).sum()
    dx, = torch.autograd.grad(f, x, create_graph=True)
    got, = torch.autograd.grad(dx, x, v.to(D))
    t = v.double() @ w64.t()
    u = half_ulp(torch, dt)
    et = linear_bound(torch, dt, v, w64, s64, m <= 512)   # of the inner product, in 16 bits
    ref, mag = t @ w64, t.abs() @ w64.abs()
    bound = (u * 1.01 + (n + 16) * E) * (mag + et @ w64.abs()) * (1 + u) + et @ w64.abs() + u * ref.abs() + tiny(torch, dt)
    within(got, ref, bound * (1 + u))


def test_second_gradients_that_are_refused(torch):
    D = dev(torch)
    x, head = head_and_x(torch, 5, 40, 64, torch.bfloat16, 1)
    x, head = x.to(D).requires_grad_(), head.to(D)
    labels = torch.zeros(5, dtype=torch.int64, device=D)
    shape = fw.BlockShape(hidden=64, heads=2, kv_heads=1, ffn=64)
    blocks = fw.QuantizedBlocks([fw.quantize_block(h, shape, 32) for h in fw.random_blocks(1, shape)], shape, D, 32)
    for f in (lambda: dfh.vocab_loss(x, head, labels), lambda: blocks.forward(x).float().sum()):
        g, = torch.autograd.grad(f() + (x * x).sum().float(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.float().sum(), x)


@pytest.mark.parametrize("call", ["vocab", "distill"])
def test_saved_tensors_on_the_host(torch, call):
    # x and head are laid out again for the kernels; what autograd keeps, copies
    # included, goes to the host and comes back, and nothing stays on the device
    D = dev(torch)
    m, v, h = 300, 1000, 512
    x, head = head_and_x(torch, m, v, h, torch.float16, 3)
    xt, ht = x.to(D).t().contiguous(), head.to(D).t().contiguous()
    g = torch.Generator().manual_seed(7)
    labels = torch.randint(0, v, (m,), generator=g).to(D)
    top, index = (t.to(D) for t in torch.randn(m, v, generator=g).topk(5, dim=1))

    def loss(a, b):
        if call == "vocab":
            return dfh.vocab_loss(a.t(), b.t(), labels)
        return dfh.distill_loss(a.t(), b.t(), top.t().contiguous().t(), index)

    xl, hl = xt.requires_grad_(), ht.requires_grad_()
    want = torch.autograd.grad(loss(xl, hl), (xl, hl))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    with torch.autograd.graph.save_on_cpu():
        kept = loss(xl * 1, hl * 1)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before < 2 * m * h   # less than x alone
    got = torch.autograd.grad(kept, (xl, hl))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_checkpointed_step(torch):
    # the forward call is made again in the backward pass, its tensors elsewhere
    from torch.utils.checkpoint import checkpoint
    D = dev(torch)
    w, _, _ = matrix(torch, 128, 256, 64, "bf16", seed=6)
    head = head_and_x(torch, 1, 900, 128, torch.bfloat16, 6)[1].to(D).t().contiguous().t()
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 50, 256, generator=g).to(torch.bfloat16).to(D)
    labels = torch.randint(0, 900, (50, 3), generator=g).to(D)

    def step(a, b):
        return dfh.vocab_loss(dfh.linear_u4(a.transpose(0, 1) * 2, w), b, labels)

    a, b = x.clone().requires_grad_(), head.clone().requires_grad_()
    want = torch.autograd.grad(step(a, b), (a, b))
    got = torch.autograd.grad(checkpoint(step, a, b, use_reentrant=False), (a, b))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("m", [40, 600])
def test_graph_of_a_float16_step_with_a_gradient_a_row(torch, m):
    # products with expanded weights in float16, and a loss whose rows have gradients
    # of their own: captured, replayed with other inputs and eager work between
    D = dev(torch)
    n, k, v = 129, 256, 1100
    w, _, _ = matrix(torch, n, k, 64, "fp32", seed=6)
    wy, _, _ = matrix(torch, 136, 136, 32, "fp32", seed=7)
    head = head_and_x(torch, 1, v, 136, torch.float16, 6)[1].to(D)
    x = torch.zeros(m, k, dtype=torch.float16, device=D)
    weight = torch.ones(m, device=D)
    labels = torch.zeros(m, dtype=torch.int64, device=D)

    def step():
        xl, hl = x.detach().requires_grad_(), head.detach().requires_grad_()
        h = torch.nn.functional.pad(dfh.linear_u4(xl, w), (0, 7))
        loss = dfh.vocab_loss(dfh.linear_u4(h, wy), hl, labels, reduction="none")
        return (loss.detach(),) + torch.autograd.grad(loss, (xl, hl), weight)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(4):
        g = torch.Generator().manual_seed(100 + r)
        x.copy_(torch.randn(m, k, generator=g).to(torch.float16))
        weight.copy_(64 * 10.0 ** (-4 * torch.rand(m, generator=g)))
        labels.copy_(torch.randint(0, v, (m,), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        assert all(bool(torch.isfinite(t.float()).all()) for t in want)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), r
