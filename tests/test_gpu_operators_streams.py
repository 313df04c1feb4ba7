"""Calls that are given a stream, with late work on it or on the current one: their
results and gradients are those of a call on the current stream."""
import numpy as np
import pytest

import lossless_entropy_coded_huffman_amd as dfh
from lossless_entropy_coded_huffman_amd import forward as fw
from lossless_entropy_coded_huffman_amd import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_gradient_of_a_loss_on_another_stream(torch, reduction):
    # the forward call runs on s and keeps its statistics there, and a copy of x
    # (which is not laid out for the kernels); its gradient runs on the current one
    g = torch.Generator().manual_seed(3)
    m, v, h = 300, 9001, 512
    head = (torch.randn(v, h, generator=g) * 0.1).to(torch.bfloat16).cuda().requires_grad_()
    x = torch.randn(h, m, generator=g).to(torch.bfloat16).cuda().requires_grad_()
    labels = torch.randint(0, v, (m,), generator=g).cuda()
    gout = torch.rand(m, generator=g).cuda() + 0.5 if reduction == "none" else torch.ones((), device="cuda")
    want = torch.autograd.grad(dfh.vocab_loss(x.t(), head, labels, reduction=reduction), (x, head), gout)
    s = torch.cuda.Stream()
    for _ in range(6):
        s.wait_stream(torch.cuda.current_stream())
        loss = dfh.vocab_loss(x.t(), head, labels, reduction=reduction, stream=s)
        got = torch.autograd.grad(loss, (x, head), gout)
        del loss
        with torch.cuda.stream(s):   # takes what the call's stream has to give
            torch.full((m * h,), 7.0, dtype=torch.bfloat16, device="cuda")
            torch.full((4 * m,), 7.0, device="cuda")
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("m", [3, 40, 700])
def test_product_of_a_transposed_batch_on_another_stream(torch, m):
    # x is ready on s and no view of rows, and the current stream is busy: the copy
    # that the call makes belongs to s
    g = torch.Generator().manual_seed(m)
    n, k = 96, 128
    packed = torch.randint(0, 256, (n * k // 2,), generator=g, dtype=torch.uint8).cuda()
    w = dfh.U4Matrix(packed, (torch.rand(n, 4, generator=g) + 0.5).cuda(), None, cols=k, group_size=32)
    x = torch.randn(2, m, k, generator=g).to(torch.bfloat16).cuda()
    dy = torch.randn(2, m, n, generator=g).to(torch.bfloat16).cuda()
    want = dfh.linear_u4(x.transpose(0, 1).contiguous(), w), dfh.linear_u4_grad(dy.transpose(0, 1).contiguous(), w)
    bx, bdy = torch.zeros_like(x), torch.zeros_like(dy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    with torch.cuda.stream(s):
        bx.copy_(x)
        bdy.copy_(dy)
    got = dfh.linear_u4(bx.transpose(0, 1), w, stream=s), dfh.linear_u4_grad(bdy.transpose(0, 1), w, stream=s)
    s.synchronize()
    torch.cuda.current_stream().synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("call", ["loss", "distill"])
def test_first_use_of_a_compressed_head_on_a_given_stream(torch, call):
    # the current stream is busy when a fresh head is used on s, and its gradient
    # follows without a wait of the caller's
    g = torch.Generator().manual_seed(5)
    m, v, h = 40, 3001, 256
    bits = synth.bf16_rne(np.random.default_rng(1).normal(0, 0.15, v * h).astype(np.float32))
    con = dfh.compress(dfh.KIND_BF16, bits)
    x = torch.randn(m, h, generator=g).to(torch.bfloat16).cuda()
    if call == "loss":
        args = (torch.randint(0, v, (m,), generator=g).cuda(),)
    else:
        args = tuple(t.cuda() for t in torch.randn(m, v, generator=g).topk(8, dim=1))

    def step(stream):
        head = fw.CompressedHead(con, v, h, torch.device("cuda:0"))
        head.scratch.fill_(float("nan"))
        leaf = x.clone().requires_grad_()
        torch.cuda.synchronize()
        if stream is not None:
            torch.cuda._sleep(20_000_000)
        loss = getattr(head, call)(leaf, *args, stream=stream)
        grad, = torch.autograd.grad(loss, leaf)
        torch.cuda.synchronize()
        return loss.detach(), grad

    want, got = step(None), step(torch.cuda.Stream())
    assert torch.isfinite(want[0]) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("m", [3, 300])
def test_gradient_of_a_product_on_another_stream(torch, m):
    # the weights come late on s; the gradient on the current stream is ordered behind
    # the call on s, which read them
    g = torch.Generator().manual_seed(m)
    n, k = 96, 128
    packed = torch.randint(0, 256, (n * k // 2,), generator=g, dtype=torch.uint8).cuda()
    late = torch.zeros_like(packed)
    w = dfh.U4Matrix(late, (torch.rand(n, 4, generator=g) + 0.5).cuda(), None, cols=k, group_size=32)
    x = torch.randn(m, k, generator=g).to(torch.bfloat16).cuda().requires_grad_()
    dy = torch.randn(m, n, generator=g).to(torch.bfloat16).cuda()
    want = dfh.linear_u4_grad(dy, dfh.U4Matrix(packed, w.scales, None, cols=k, group_size=32))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(packed)
    y = dfh.linear_u4(x, w, stream=s)
    got, = torch.autograd.grad(y, x, dy)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_saved_tensors_on_the_host_after_a_call_on_another_stream(torch):
    # the call on s is late; what it keeps goes to the host behind it
    g = torch.Generator().manual_seed(9)
    m, v, h = 300, 2001, 256
    head = (torch.randn(v, h, generator=g) * 0.1).to(torch.bfloat16).cuda().requires_grad_()
    x = torch.randn(h, m, generator=g).to(torch.bfloat16).cuda().requires_grad_()
    labels = torch.randint(0, v, (m,), generator=g).cuda()
    want = torch.autograd.grad(dfh.vocab_loss(x.t(), head, labels), (x, head))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    with torch.autograd.graph.save_on_cpu():
        loss = dfh.vocab_loss(x.t(), head, labels, stream=s)
    got = torch.autograd.grad(loss, (x, head))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
