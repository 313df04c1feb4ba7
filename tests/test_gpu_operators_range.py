"""Scales of any size that float32 holds: products with FP16 operands on both sides
of the row counts where the kernel changes, and their gradients, against float64.
The bounds are those of test_gpu_operators, where a weight that is held in 16 bits is
off by 2^-31 of the largest scale (of its row; in a gradient of the matrix) if that
is more than half a step of its own."""
import pytest

import lossless_entropy_coded_huffman_amd as dfh
from test_gpu_operators import E, dev, few_rows, half_ulp, linear_bound, tiny, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def weights(torch, n, k, group, s, zeros, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8)
    z = torch.randint(0, 16, s.shape, generator=g, dtype=torch.uint8) if zeros else None
    d = dev(torch)
    w = dfh.U4Matrix((q[:, 0::2] | (q[:, 1::2] << 4)).reshape(-1).to(d), s.to(d).expand(n, -1),
                     None if z is None else z.to(d).expand(n, -1), cols=k, group_size=group)
    idx = torch.arange(k) // group
    s64 = s.double().expand(n, -1)[:, idx]
    z64 = z.double().expand(n, -1)[:, idx] if zeros else 8.0
    return w, (q.double() - z64) * s64, s64.abs()


SIZES = [(3, 70, 200, 32), (70, 70, 200, 32), (530, 70, 200, 32), (530, 259, 4104, 128), (193, 4200, 4104, 4104),
         (530, 70, 40, 32)]


@pytest.mark.parametrize("size,act", [(1e-9, 6e4), (1e-7, 1e4), (1e-6, 1e3), (1e4, 2.0 ** -8), (3e6, 2.0 ** -16)])
@pytest.mark.parametrize("m,n,k,group", SIZES)
def test_scales_out_of_fp16s_range(torch, m, n, k, group, size, act):
    dt, D = torch.float16, dev(torch)
    g = torch.Generator().manual_seed(m + n)
    s = (torch.rand(n if n % 2 == 0 else 1, (k + group - 1) // group, generator=g) + 0.5) * size
    w, w64, s64 = weights(torch, n, k, group, s, n % 2 == 1, m)
    x = (torch.randn(m, k, generator=g) * act / k ** 0.5).to(dt)
    few = few_rows(m, n, k)
    peak = s64.amax(1)[None, :] * (0 if few else 2.0 ** -31)
    bound = linear_bound(torch, dt, x, w64, s64, few) + x.double().abs().sum(1, keepdim=True) * peak * 1.01
    y = dfh.linear_u4(x.to(D), w)
    ref = x.double() @ w64.t()
    assert float(ref.abs().max()) < 6e4 and float(ref.abs().max()) > 2.0 ** -20
    within(y, ref, bound)
    dy = (torch.randn(m, n, generator=g) * act / n ** 0.5).to(dt)
    ref, u = dy.double() @ w64, half_ulp(torch, dt)
    bound = (u * 1.01 + (n + 16) * E) * (dy.double().abs() @ w64.abs()) * (1 + u) + u * ref.abs() + tiny(torch, dt)
    within(dfh.linear_u4_grad(dy.to(D), w), ref,
           bound + dy.double().abs().sum(1, keepdim=True) * s64.max() * 2.0 ** -31 * 1.01)


@pytest.mark.parametrize("m,n,k,group", [(3, 70, 200, 32), (530, 70, 200, 32), (193, 4200, 4104, 128)])
def test_scales_of_all_sizes_in_one_matrix(torch, m, n, k, group):
    # a row's results depend on that row's scales alone, however large another's are
    dt, D = torch.float16, dev(torch)
    g = torch.Generator().manual_seed(n)
    s = 10.0 ** (torch.rand(n, 1, generator=g) * 10 - 9) * (torch.rand(n, (k + group - 1) // group, generator=g) + 0.5)
    s[5] = 0.0
    w, w64, s64 = weights(torch, n, k, group, s, True, m)
    x = torch.randn(m, k, generator=g).to(dt)
    few = few_rows(m, n, k)
    peak = s64.amax(1)[None, :] * (0 if few else 2.0 ** -31)
    bound = linear_bound(torch, dt, x, w64, s64, few) + x.double().abs().sum(1, keepdim=True) * peak * 1.01
    within(dfh.linear_u4(x.to(D), w), x.double() @ w64.t(), bound)
    dy = torch.randn(m, n, generator=g).to(dt)
    ref, u = dy.double() @ w64, half_ulp(torch, dt)
    bound = (u * 1.01 + (n + 16) * E) * (dy.double().abs() @ w64.abs()) * (1 + u) + u * ref.abs() + tiny(torch, dt)
    within(dfh.linear_u4_grad(dy.to(D), w), ref,
           bound + dy.double().abs().sum(1, keepdim=True) * s64.max() * 2.0 ** -31 * 1.01)


def test_one_infinite_scale(torch):
    # the group it stands for is infinite (NaN where q = z); other rows are as ever
    D = dev(torch)
    for m in (3, 530):
        n, k = 40, 64
        s = torch.full((n, 2), 0.01)
        s[7, 1] = float("inf")
        w, w64, _ = weights(torch, n, k, 32, s, False, 1)
        x = torch.ones(m, k, dtype=torch.float16)
        y = dfh.linear_u4(x.to(D), w).double().cpu()
        assert not torch.isfinite(y[:, 7]).any()
        s[7, 1] = 0.01
        w2, _, _ = weights(torch, n, k, 32, s, False, 1)
        keep = [i for i in range(n) if i != 7]
        assert torch.equal(y[:, keep], dfh.linear_u4(x.to(D), w2).double().cpu()[:, keep])


@pytest.mark.parametrize("m", [1, 4, 40, 200])
@pytest.mark.parametrize("k,group,zeros", [(512, 128, True), (512, 32, True), (200, 64, False), (1416, 1416, True)])
def test_a_large_input_at_a_zero_weight(torch, m, k, group, zeros):
    # BF16: every sum of x (16 + q), x and (16 + z) x is a whole number under 2^24, so
    # float32 has it exactly, and a large input whose weight is zero leaves no trace
    D, n = dev(torch), 40
    g = torch.Generator().manual_seed(k)
    s = torch.full((n, (k + group - 1) // group), 0.5)
    w, w64, _ = weights(torch, n, k, group, s, zeros, k)
    x = torch.randint(-2, 3, (m, k), generator=g).to(torch.bfloat16)
    big = 3 * 2.0 ** 17
    # a column of zero weights: codes equal to the zero points there
    q = torch.stack((w.packed & 15, w.packed >> 4), -1).view(n, k).cpu()
    zp = w.zeros.cpu().expand(n, -1) if zeros else torch.full((n, s.shape[1]), 8, dtype=torch.uint8)
    col = 77
    q[:, col] = zp[:, col // group]
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).reshape(-1).to(D)
    w = dfh.U4Matrix(packed, w.scales, w.zeros, cols=k, group_size=group)
    w64[:, col] = 0.0
    x[:, col] = big
    assert float((x.double().abs().sum(1) * 31).max()) < 2.0 ** 24
    ref = (x.double() @ w64.t()).to(torch.bfloat16)
    assert float(ref.abs().max()) > 0
    assert torch.equal(dfh.linear_u4(x.to(D), w).cpu(), ref)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("m,v,h", [(64, 300, 64), (300, 2049, 136)])
def test_rows_with_gradients_of_all_sizes(torch, m, v, h, dtype):
    # reduction "none": dhead of an entry that only rows of small gradients name keeps
    # its bits beside rows whose gradient is 10^7 times as large
    dt, D = getattr(torch, dtype), dev(torch)
    g = torch.Generator().manual_seed(m)
    x = torch.randn(m, h, generator=g).to(dt)
    head = (torch.randn(v, h, generator=g) * (40 / h ** 0.5)).to(dt)   # sure of one entry each
    labels = torch.randperm(v, generator=g)[:m]
    gout = 1024 * 10.0 ** (torch.rand(m, generator=g) * -7)
    labels[3] = -100
    x[3] = float("inf")
    hs = head.to(D).requires_grad_()
    loss = dfh.vocab_loss(x.to(D), hs, labels.to(D), reduction="none")
    dh, = torch.autograd.grad(loss, hs, gout.to(D))
    valid = labels >= 0
    xz = x.double().masked_fill(~valid[:, None], 0.0)
    z = xz @ head.double().t()
    q = torch.softmax(z, 1)
    t = torch.zeros_like(q).scatter(1, labels.clamp(min=0)[:, None], 1.0)
    d = q - t
    u, gw = half_ulp(torch, dt), gout.double() * valid
    # p is off by twice its logits' error and float32 steps of the exponent, then rounded
    # to 16 bits (FP16 times 2^15), and x times a row's gradient is rounded as well
    dz = ((h + 8) * E * (xz.abs() @ head.double().abs().t())).amax(1)
    lse, zt = torch.logsumexp(z, 1).abs(), z.abs().amax(1)
    ed = (2 * dz[:, None] + 8 * E * (lse[:, None] + zt[:, None] + 4)) * q * 1.01 + 4 * E * t
    ed = (ed * (1 + u) + u * d.abs() + (2.0 ** -40 if dt == torch.float16 else 2.0 ** -134)) * (1 + u) + u * d.abs()
    ref = (d * gw[:, None]).t() @ xz
    floor = 2.0 ** -39 * (gw[:, None] * xz.abs()).max() * 1.01 * (d.abs() + ed).sum(0)[:, None]
    bound = ((ed + (m + 64) * E * d.abs()) * gw[:, None]).t() @ xz.abs() * (1 + 8 * E) + floor
    within(dh, ref, bound * (1 + u) + (u + 8 * E) * ref.abs() + tiny(torch, dt))


@pytest.mark.parametrize("m", [1, 4, 17, 60, 200])
@pytest.mark.parametrize("n,k,group", [(40, 200, 32), (259, 1416, 1416), (70, 4104, 128)])
def test_every_row_ends_in_an_infinity(torch, m, n, k, group):
    # BF16: inf times a weight of either sign, NaN at a zero weight, whatever the place
    D = dev(torch)
    g = torch.Generator().manual_seed(k)
    s = torch.rand(n, (k + group - 1) // group, generator=g) + 0.5
    w, w64, _ = weights(torch, n, k, group, s, True, k)
    x = torch.randn(m, k, generator=g).to(torch.bfloat16)
    for at in (k - 1, 0, 45):
        xi = x.clone()
        xi[:, at] = float("inf")
        xi[m // 2, at] = -float("inf")
        ref = xi.double() @ w64.t()
        got = dfh.linear_u4(xi.to(D), w).double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(got.nan_to_num(0.5), ref.nan_to_num(0.5))
    # a sum that is finite where the products with 16 + q are not
    xi = x.clone()
    xi[:, 45] = 2.0 ** 126
    q = torch.stack((w.packed & 15, w.packed >> 4), -1).view(n, k).cpu()
    q[:, 45] = w.zeros.cpu().expand(n, -1)[:, 45 // group]
    w64[:, 45] = 0.0
    w2 = dfh.U4Matrix((q[:, 0::2] | (q[:, 1::2] << 4)).reshape(-1).to(D), w.scales, w.zeros, cols=k, group_size=group)
    ref = xi.double() @ w64.t()
    bound = k * E * (xi.double().masked_fill(xi == 2.0 ** 126, 0.0).abs() @ w64.abs().t())
    within(dfh.linear_u4(xi.to(D), w2), ref, bound + 2.0 ** -8 * ref.abs() * 1.01)
