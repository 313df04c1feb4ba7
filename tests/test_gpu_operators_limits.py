"""Calls within the stated limits whose launches would hold 2^32 threads or more."""
import pytest

import lossless_entropy_coded_huffman_amd as dfh
from test_gpu_operators import E, dev, half_ulp, matrix, tiny, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield torch
    torch.cuda.empty_cache()


def test_distillation_of_many_entries(torch):
    # 2^26 entries, one wave each
    D = dev(torch)
    rows, top, v, h = 1 << 16, 1024, 1500, 8
    g = torch.Generator(device=D).manual_seed(1)
    x = torch.randn(rows, h, generator=g, device=D).to(torch.bfloat16)
    head = torch.randn(v, h, generator=g, device=D).to(torch.bfloat16)
    teacher = (torch.randn(rows, top, generator=g, device=D) * 2).to(torch.bfloat16)
    index = torch.randint(0, v, (rows, top), generator=g, device=D)
    got = dfh.distill_loss(x, head, teacher, index, reduction="none").double()
    for lo in (0, rows // 2, rows - 512):
        s = slice(lo, lo + 512)
        z = x[s].double() @ head.double().t()
        logq, logt = torch.log_softmax(z, 1), torch.log_softmax(teacher[s].double(), 1)
        ref = (logt.exp() * (logt - logq.gather(1, index[s]))).sum(1)
        # a logit is off by (h + 8) e sum |x| |head|, in the log-sum and in the mean of
        # the targets; float32 steps of the terms, and sums of up to 1500 of them
        dz = ((h + 8) * E * (x[s].double().abs() @ head.double().abs().t())).amax(1)
        bound = 2 * dz + (top + 16) * E * (logt.exp() * (logt.abs() + logq.gather(1, index[s]).abs())).sum(1) + v * E
        assert bool(((got[s] - ref).abs() <= bound).all())


def test_gradient_of_the_most_rows(torch):
    # 2^24 rows of an odd number of outputs, which are padded for the product
    D = dev(torch)
    m, n, k = 1 << 24, 9, 8
    w, w64, _ = matrix(torch, n, k, 32, "fp32", seed=1)
    g = torch.Generator(device=D).manual_seed(2)
    dy = torch.randn(m, n, generator=g, device=D, dtype=torch.float16)
    dx = dfh.linear_u4_grad(dy, w)
    u = half_ulp(torch, torch.float16)
    for lo in (0, m // 2 - 100, m - 1000):
        d = dy[lo: lo + 1000].double().cpu()
        ref = d @ w64
        bound = (u * 1.01 + (n + 16) * E) * (d.abs() @ w64.abs()) * (1 + u) + u * ref.abs() + tiny(torch, torch.float16)
        within(dx[lo: lo + 1000], ref, bound)


def test_loss_of_very_many_tiles(torch):
    # 2^21 rows of 2^18 logits: 2^23 tiles of 256 x 256, more than a launch holds
    D = dev(torch)
    m, v, h = 1 << 21, 1 << 18, 8
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 70 GB for the statistics of the tiles")
    g = torch.Generator(device=D).manual_seed(3)
    x = torch.randn(m, h, generator=g, device=D).to(torch.bfloat16)
    head = torch.randn(v, h, generator=g, device=D).to(torch.bfloat16)
    labels = torch.randint(0, v, (m,), generator=g, device=D)
    got = dfh.vocab_loss(x, head, labels, reduction="none").double()
    for lo in (0, m // 2 - 50, m - 100):   # the halves of the launch, and its ends
        s = slice(lo, lo + 100)
        z = x[s].double() @ head.double().t()
        ref = torch.logsumexp(z, 1) - z.gather(1, labels[s][:, None])[:, 0]
        dz = ((h + 8) * E * (x[s].double().abs() @ head.double().abs().t())).amax(1)
        # 2^18 exponentials in sums of at most 64, then 4096 parts in a tree of 32 and 256
        assert bool(((got[s] - ref).abs() <= 2 * dz + 512 * E * (1 + ref.abs())).all())
