"""Operators on inputs whose strides the kernels do not take as they are: the same
results as from contiguous copies."""
import pytest

import lossless_entropy_coded_huffman_amd as dfh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def u4(torch, rows, cols, group, seed=0):
    g = torch.Generator().manual_seed(seed)
    packed = torch.randint(0, 256, (rows * cols // 2,), generator=g, dtype=torch.uint8).cuda()
    scales = (torch.rand(rows, cols // group, generator=g) * 0.02 + 0.01).to(torch.bfloat16).cuda()
    return dfh.U4Matrix(packed, scales, None, cols=cols, group_size=group)


def far(torch, rows, cols, step, seed):
    """[rows, cols] with rows `step` elements apart."""
    buf = torch.zeros((rows - 1) * step + cols, dtype=torch.bfloat16, device="cuda")
    t = buf.as_strided((rows, cols), (step, 1))
    t.copy_(torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)))
    return t


@pytest.mark.parametrize("rows", [2, 9])
def test_last_tokens_of_long_prompts(torch, rows):
    # hidden[:, -1] of [rows, tokens, hidden]: rows further apart than 2^21 elements
    w = u4(torch, 128, 256, 64)
    x, dy = far(torch, rows, 256, (1 << 21) + 256, 1), far(torch, rows, 128, (1 << 21) + 128, 2)
    assert torch.equal(dfh.linear_u4(x, w), dfh.linear_u4(x.contiguous(), w))
    assert torch.equal(dfh.linear_u4_grad(dy, w), dfh.linear_u4_grad(dy.contiguous(), w))
    odd = u4(torch, 127, 256, 64)
    assert torch.equal(dfh.linear_u4_grad(dy[:, :127], odd), dfh.linear_u4_grad(dy[:, :127].contiguous(), odd))
    head = torch.randn(500, 256, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    labels = torch.arange(rows, device="cuda")
    assert torch.equal(dfh.vocab_loss(x, head, labels), dfh.vocab_loss(x.contiguous(), head, labels))


def test_one_row_of_any_stride(torch):
    g = torch.Generator().manual_seed(5)
    for n in (128, 127):
        w = u4(torch, n, 256, 64)
        x = torch.randn(256, 1, generator=g).to(torch.bfloat16).cuda()
        dy = torch.randn(n, 1, generator=g).to(torch.bfloat16).cuda()
        assert x.t().stride() == (1, 1) and dy.t().stride() == (1, 1)
        assert torch.equal(dfh.linear_u4(x.t(), w), dfh.linear_u4(x.view(1, 256), w))
        assert torch.equal(dfh.linear_u4_grad(dy.t(), w), dfh.linear_u4_grad(dy.view(1, n), w))
    head = torch.randn(500, 256, generator=g).to(torch.bfloat16).cuda()
    label = torch.tensor([7], device="cuda")
    assert torch.equal(dfh.vocab_loss(x.t(), head, label), dfh.vocab_loss(x.view(1, 256), head, label))
