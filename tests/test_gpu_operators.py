"""Products with uint4 weights, vocabulary cross entropy and distillation on
the GPU, against plain implementations in float64.

Tolerances.  u is half a unit in the last place of the call's 16-bit type,
e = 2^-24 that of float32.  A float32 sum of n terms is off by at most n e times
the sum of the terms' magnitudes; a value that is rounded to 16 bits by u times
its magnitude (plus half the smallest subnormal).  Each test adds these up for
the roundings that the operator documents, with the magnitudes taken from the
float64 computation.
"""
import math

import numpy as np
import pytest

import lossless_entropy_coded_huffman_amd as dfh
from lossless_entropy_coded_huffman_amd import synth

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def dev(torch):
    return torch.device("cuda:0")


def half_ulp(torch, dt):
    return torch.finfo(dt).eps / 2


def tiny(torch, dt):
    """Half the smallest subnormal of a 16-bit type."""
    return 2.0 ** -25 if dt == torch.float16 else 2.0 ** -134


def within(got, ref, bound):
    got = got.double().cpu()
    err = (got - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), "worst %g over its bound %g at %s (of %d bad)" % (
        float(err[bad][0]), float(bound[bad][0]), bad.nonzero()[0].tolist(), int(bad.sum()))


# ------------------------------------------------------------- uint4 products
def matrix(torch, n, k, group, scale="bf16", zeros=True, seed=0, broadcast=False):
    """(U4Matrix on the GPU, its weights in float64)."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8)
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).reshape(-1)
    ng = (k + group - 1) // group
    sdt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[scale]
    r = 1 if broadcast else n
    s = ((torch.rand(r, ng, generator=g) + 0.5) * 0.02 * torch.where(torch.rand(r, ng, generator=g) < 0.1, -1.0, 1.0)).to(sdt)
    z = torch.randint(0, 16, (r, ng), generator=g, dtype=torch.uint8) if zeros else None
    d = dev(torch)
    sd = s.to(d).expand(n, ng)
    zd = z.to(d).expand(n, ng) if zeros else None
    w = dfh.U4Matrix(packed.to(d), sd, zd, cols=k, group_size=group)
    idx = torch.arange(k) // group
    zz = z.double() if zeros else torch.full((r, ng), 8.0, dtype=torch.float64)
    return w, ((q.double() - zz.expand(n, ng)[:, idx]) * s.double().expand(n, ng)[:, idx]), s.double().abs().expand(n, ng)[:, idx]


def few_rows(m, n, k):
    """Rows whose products take the integers as they are (include/dfh.h)."""
    return m <= 192 or (m <= 384 and n * k <= 1 << 24) or (m <= 512 and n * k <= 1 << 22)


def linear_bound(torch, dt, x, w64, s64, few):
    """Bound on |y - ref|: few rows scale the sums of integers, more round every
    weight."""
    u, k = half_ulp(torch, dt), x.shape[1]
    xa = x.double().abs()
    mag = xa @ w64.abs().t()
    ref = (x.double() @ w64.t()).abs()
    if few:
        # a group's sums of x (bias + q) and (bias + z) x in float32, scaled: bias
        # 128 in BF16, none in FP16; 128 terms a sum, then the blocks and waves
        mag = xa @ (s64 * (286.0 if dt == torch.bfloat16 else 16.0)).t()
        acc = (128 + k / 128 + 16) * E * mag
        return acc * (1 + u) + u * ref + tiny(torch, dt)
    # every weight rounded twice (its float32 product and the 16-bit value)
    return (u * 1.01 + (k + 16) * E) * mag * (1 + u) + u * ref + tiny(torch, dt)


FEW = [(1, 16, 64, 32), (4, 4100, 8712, 96), (1, 70, 9000, 128), (3, 33000, 520, 32), (1, 37, 16384, 160), (6, 2048, 2048, 64), (48, 1000, 3080, 32), (1, 17, 4096, 128), (1, 300, 1416, 1416), (2, 1024, 256, 64), (16, 33, 8, 32), (16, 130, 520, 96),
       (17, 64, 1024, 128), (128, 260, 1032, 128), (200, 129, 640, 64), (256, 65, 2080, 416), (300, 2304, 2048, 64), (32, 47, 136, 32), (33, 200, 2048, 256), (64, 31, 4104, 128), (5, 1, 24, 64)]
MANY = [(65, 64, 64, 32), (100, 130, 520, 96), (257, 64, 72, 72), (513, 70, 136, 32), (193, 4200, 4104, 128), (400, 2304, 2048, 64), (333, 257, 1416, 32), (256, 512, 256, 128), (129, 1, 8, 32),
        (640, 1031, 72, 72), (1500, 2304, 192, 64), (2049, 6400, 64, 64)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("m,n,k,group", FEW + MANY)
def test_linear_u4(torch, m, n, k, group, dtype):
    dt = getattr(torch, dtype)
    scale = ["bf16", "fp16", "fp32"][(m + n) % 3]
    w, w64, s64 = matrix(torch, n, k, group, scale, zeros=n % 2 == 0, seed=m + n, broadcast=(m + n + k) % 5 == 0)
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(k)).to(dt)
    y = dfh.linear_u4(x.to(dev(torch)), w)
    assert y.dtype == dt and y.shape == (m, n)
    within(y, x.double() @ w64.t(), linear_bound(torch, dt, x, w64, s64, few_rows(m, n, k)))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("m,n,k,group", [(1, 16, 64, 32), (3, 5, 8, 8), (17, 131, 1416, 1416), (64, 256, 512, 128),
                                         (333, 257, 136, 32), (70, 2304, 192, 64), (2049, 72, 6400, 128)])
def test_linear_u4_gradient(torch, m, n, k, group, dtype):
    dt = getattr(torch, dtype)
    w, w64, _ = matrix(torch, n, k, group, "fp32", zeros=m % 2 == 1, seed=m)
    dy = torch.randn(m, n, generator=torch.Generator().manual_seed(n)).to(dt)
    x = torch.randn(m, k).to(dt).to(dev(torch)).requires_grad_()
    dx, = torch.autograd.grad(dfh.linear_u4(x, w), x, dy.to(dev(torch)))
    ref = dy.double() @ w64
    u = half_ulp(torch, dt)
    bound = (u * 1.01 + (n + 16) * E) * (dy.double().abs() @ w64.abs()) * (1 + u) + u * ref.abs() + tiny(torch, dt)
    within(dx, ref, bound)
    # the same call without autograd gives the same bits
    assert torch.equal(dfh.linear_u4_grad(dy.to(dev(torch)), w), dx)


def test_linear_u4_gradient_is_the_difference_quotient(torch):
    # y is linear in x: y(x + d) - y(x) = d W^T, and <dy, d W^T> = <dx, d>
    w, w64, s64 = matrix(torch, 96, 128, 32, "fp32", seed=5)
    g = torch.Generator().manual_seed(1)
    x, d, dy = (torch.randint(-4, 5, s, generator=g).to(torch.bfloat16) for s in ((4, 128), (4, 128), (4, 96)))
    D = dev(torch)
    y0, y1 = dfh.linear_u4(x.to(D), w).double().cpu(), dfh.linear_u4((x + d).to(D), w).double().cpu()
    dx = dfh.linear_u4_grad(dy.to(D), w).double().cpu()
    u = half_ulp(torch, torch.bfloat16)
    lhs, rhs = (dy.double() * (y1 - y0)).sum(), (dx * d.double()).sum()
    b = (dy.double().abs() * (linear_bound(torch, torch.bfloat16, x + d, w64, s64, True)
                              + linear_bound(torch, torch.bfloat16, x, w64, s64, True))).sum()
    b = b + (d.double().abs() * (2.02 * u * (dy.double().abs() @ w64.abs()) + u * dx.abs())).sum()
    assert abs(float(lhs - rhs)) <= float(b)


@pytest.mark.parametrize("m", [3, 80, 530])
def test_linear_u4_strides_and_shapes(torch, m):
    D = dev(torch)
    w, w64, _ = matrix(torch, 40, 72, 32, "bf16", seed=2)
    base = torch.randn(m, 200, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(D)
    want = dfh.linear_u4(base[:, 8:80].contiguous(), w)
    for view in (base[:, 8:80], base[:, 8:80].t().contiguous().t(), base.clone()[:, 8:80]):
        assert torch.equal(dfh.linear_u4(view, w), want)
    odd = torch.empty(m * 72 + 3, dtype=torch.bfloat16, device=D)[3:].view(m, 72)   # not 16-byte aligned
    odd.copy_(base[:, 8:80])
    assert torch.equal(dfh.linear_u4(odd, w), want)
    assert torch.equal(dfh.linear_u4(base[:, 8:80].reshape(1, m, 72), w), want.view(1, m, 40))
    assert torch.equal(dfh.linear_u4(base[0, 8:80], w), dfh.linear_u4(base[:1, 8:80], w)[0])
    empty = dfh.linear_u4(base[:0, 8:80], w)
    assert empty.shape == (0, 40)
    assert dfh.linear_u4_grad(empty, w).shape == (0, 72)
    dy = torch.randn(m, 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(D)
    a = dfh.linear_u4_grad(dy[:, 5:45], w)
    assert torch.equal(a, dfh.linear_u4_grad(dy[:, 5:45].contiguous(), w))


def test_linear_u4_unaligned_weights(torch):
    # a layer that starts inside a larger buffer, 4-byte aligned only, and rows
    # whose length is no multiple of 32
    D = dev(torch)
    for k in (64, 72):
        w, w64, s64 = matrix(torch, 50, k, 32, "fp32", seed=k)
        buf = torch.zeros(w.packed.numel() + 4, dtype=torch.uint8, device=D)
        buf[4:] = w.packed
        w2 = dfh.U4Matrix(buf[4:], w.scales, w.zeros, cols=k, group_size=32)
        for m in (1, 20, 50, 90, 520):
            x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).to(torch.float16).to(D)
            assert torch.equal(dfh.linear_u4(x, w2), dfh.linear_u4(x, w))
            dy = torch.randn(m, 50, generator=torch.Generator().manual_seed(m)).to(torch.float16).to(D)
            assert torch.equal(dfh.linear_u4_grad(dy, w2), dfh.linear_u4_grad(dy, w))


@pytest.mark.parametrize("m", [1, 40, 270, 530])
def test_linear_u4_infinities_and_nan(torch, m):
    # inf in one element of one row: that row's results are inf * weight or, where
    # the weight is zero, NaN; NaN in another row; the rows between are untouched
    D = dev(torch)
    w, w64, _ = matrix(torch, 48, 96, 32, "fp32", zeros=True, seed=9)
    for dt in (torch.bfloat16, torch.float16):
        x = torch.ones(m, 96, dtype=dt)
        clean = dfh.linear_u4(x.to(D), w)
        x[0, 5] = float("inf")
        if m > 2:
            x[2, 7] = float("nan")
        got = dfh.linear_u4(x.to(D), w).float().cpu()
        wr = w64 if m <= 512 else w64.to(dt).double()
        ref = (x.double()[0] * wr).sum(dim=1)     # inf * 0 is NaN
        assert torch.equal(torch.isnan(got[0]), torch.isnan(ref))
        ok = ~torch.isnan(ref)
        assert torch.equal(got[0][ok].double(), ref[ok])
        if m > 2:
            assert torch.isnan(got[2]).all()
            rest = [i for i in range(m) if i not in (0, 2)]
            assert torch.equal(got[rest], clean.float().cpu()[rest])
    # the largest finite values do not overflow on the way
    x = torch.zeros(m, 96, dtype=torch.bfloat16)
    x[:, 3] = 3e38
    ref = x.double() @ w64.t()
    got = dfh.linear_u4(x.to(D), w).double().cpu()
    assert ((got - ref).abs() <= 2.02 * 2.0 ** -8 * ref.abs()).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_linear_u4_any_zero_point(torch, dtype):
    # zero points are bytes: 0 to 255, not only those of the quantiser
    dt, D = getattr(torch, dtype), dev(torch)
    g = torch.Generator().manual_seed(3)
    n, k, grp = 70, 200, 32
    q = torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8)
    z = torch.randint(0, 256, (n, 7), generator=g, dtype=torch.uint8)
    z[0], z[1] = 0, 255
    s = torch.rand(n, 7, generator=g) * 0.01 + 0.01
    w = dfh.U4Matrix((q[:, 0::2] | (q[:, 1::2] << 4)).reshape(-1).to(D), s.to(D), z.to(D), cols=k, group_size=grp)
    idx = torch.arange(k) // grp
    w64, s64 = (q.double() - z.double()[:, idx]) * s.double()[:, idx], s.double()[:, idx]
    for m in (2, 30, 600):
        x = torch.randn(m, k, generator=g).to(dt)
        few = m <= 512
        # the sums are of x (128 + q) and (128 + z) x in BF16, of x (q - z) in FP16
        mag = x.double().abs() @ (s64 * 526).t()
        u = half_ulp(torch, dt)
        ref = x.double() @ w64.t()
        bound = (128 + k / 128 + 16) * E * mag * (1 + u) + u * ref.abs() + tiny(torch, dt) if few else \
            (u * 1.01 + (k + 16) * E) * (x.double().abs() @ w64.abs().t()) * (1 + u) + u * ref.abs() + tiny(torch, dt)
        within(dfh.linear_u4(x.to(D), w), ref, bound)


def test_linear_u4_rows_behind_the_last_are_left(torch):
    # columns and rows past the end of y in a larger buffer keep their bytes
    D = dev(torch)
    for m, n in ((3, 19), (70, 130), (600, 70)):
        w, _, _ = matrix(torch, n, 64, 32, "fp32", seed=n)
        x = torch.randn(m, 64).to(torch.bfloat16).to(D)
        buf = torch.full((m * n + 64,), 7.0, dtype=torch.bfloat16, device=D)
        L = dfh.lib()
        need = L.df_linear_u4_workspace_bytes(w._ref, m)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=D)
        assert L.df_linear_u4(w._ref, 0, x.data_ptr(), m, 64, buf.data_ptr(), ws.data_ptr(), need,
                              torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(buf[: m * n].view(m, n), dfh.linear_u4(x, w))
        assert bool((buf[m * n:] == 7.0).all())


def test_linear_u4_from_a_decoded_container(torch):
    # the codec's own path: quantise, Huffman code, decode on the GPU, multiply
    D = dev(torch)
    n, k = 96, 256
    q = synth.quantize_u4(np.random.default_rng(0).normal(0, 0.02, n * k).astype(np.float32), True)
    packed = synth.pack_u4(q)
    dc = dfh.to_device(dfh.compress(dfh.KIND_U4, packed), D)
    out = dc.empty_output()
    dfh.df_decompress(dc, out)
    s = torch.rand(n, 2, generator=torch.Generator().manual_seed(0)) + 0.5
    w = dfh.U4Matrix(out, s.to(D), None, cols=k, group_size=128)
    w64 = (torch.from_numpy(q.reshape(n, k)).double() - 8) * s.double().repeat_interleave(128, 1)
    x = torch.randn(9, k, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    within(dfh.linear_u4(x.to(D), w), x.double() @ w64.t(),
           linear_bound(torch, torch.bfloat16, x, w64, s.double().repeat_interleave(128, 1), True))


# ---------------------------------------------------------------------- losses
def head_and_x(torch, m, v, h, dt, seed, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, h, generator=g).to(dt)
    head = (torch.randn(v, h, generator=g) * (spread / math.sqrt(h))).to(dt)
    return x, head


def plain_loss(torch, x, head, valid, t, idx, temp, reduction):
    """Float64: (per row loss, q, target matrix, count)."""
    z = (x.double().masked_fill(~valid[:, None], 0.0) @ head.double().t()) / temp
    logq = torch.log_softmax(z, dim=1)
    per = torch.where(t > 0, t * (t.clamp(min=1e-300).log() - logq.gather(1, idx)), 0.0).sum(1) * temp * temp
    tm = torch.zeros_like(z).scatter_add_(1, idx, t)
    return torch.where(valid, per, 0.0), logq.exp(), tm


def check_loss(torch, loss, dx, dhead, x, head, valid, t, idx, temp, reduction, gout, extra_scale_rounding):
    dt = x.dtype
    u, h = half_ulp(torch, dt), x.shape[1]
    per, q, tm = plain_loss(torch, x, head, valid, t, idx, temp, reduction)
    xz = x.double().masked_fill(~valid[:, None], 0.0)
    n = int(valid.sum())
    # a logit is off by h e sum |x| |head|; the log-sum and each target logit by
    # that, plus float32 steps of values up to |lse| (2^3 of them)
    dz = (h + 8) * E * (xz.abs() @ head.double().abs().t()) / temp
    dzm = dz.amax(dim=1)
    lse = torch.logsumexp(xz @ head.double().t() / temp, dim=1).abs()
    zt = (xz @ head.double().t() / temp).abs().amax(dim=1)
    b = temp * temp * (2 * dzm + 8 * E * (lse + zt + 4)) * valid
    if reduction == "none":
        within(loss, per, b + 2 * E * per.abs())
        g = gout.double() * valid
    else:
        tot, div = per.sum(), (max(n, 1) if reduction == "mean" else 1)
        within(loss.reshape(1), (tot / div).reshape(1), (b.sum() / div + 4 * E * tot / div).reshape(1) + 1e-45)
        g = gout.double().reshape(1).expand(x.shape[0]) / div * valid
    if dx is None and dhead is None:
        return
    g = g * temp
    # dz = p - t is off by p times (twice the logits' error, and float32 steps of the
    # exponent) before it is rounded to 16 bits; FP16 stores it times 2^15
    d = (q - tm)
    ed = (2 * dzm[:, None] + 8 * E * (lse[:, None] + zt[:, None] + 4)) * q * 1.01 + 4 * E * tm
    sub = 2.0 ** -40 if dt == torch.float16 else 2.0 ** -134
    ed = ed * (1 + u) + u * d.abs() + sub
    v = head.shape[0]
    if dx is not None:
        ref = (d * g[:, None]) @ head.double()
        bound = (ed + (v + 64) * E * d.abs()) @ head.double().abs() * g.abs()[:, None] * (1 + 4 * E)
        within(dx, ref, bound * (1 + u) + (u + 4 * E) * ref.abs() + tiny(torch, dt))
    if dhead is not None:
        ew = ed * (1 + u) + (u * d.abs() + sub if extra_scale_rounding else 0.0)
        ref = (d * g[:, None]).t() @ xz
        gm = g.abs().max()
        bound = (((ew + (x.shape[0] + 64) * E * d.abs()) * g.abs()[:, None]
                  + (sub * gm if extra_scale_rounding else 0.0) * valid[:, None]).t() @ xz.abs()) * (1 + 8 * E)
        within(dhead, ref, bound * (1 + u) + (u + 8 * E) * ref.abs() + tiny(torch, dt))


LOSS_SHAPES = [(1, 5, 8), (4, 1, 16), (2, 2, 8), (3, 64, 72), (17, 1000, 128), (64, 257, 264), (65, 2049, 64), (130, 517, 520),
               (300, 4100, 136), (1100, 3001, 64), (261, 60003, 72), (513, 33000, 64)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("m,v,h", LOSS_SHAPES)
def test_vocab_loss(torch, m, v, h, reduction, dtype):
    dt, D = getattr(torch, dtype), dev(torch)
    x, head = head_and_x(torch, m, v, h, dt, seed=m + v)
    g = torch.Generator().manual_seed(m)
    labels = torch.randint(0, v, (m,), generator=g)
    if m > 1:
        labels[torch.rand(m, generator=g) < 0.3] = -100
    valid = labels != -100
    x[~valid] = float("nan")      # what ignored rows hold does not matter
    xs, hs = x.to(D).requires_grad_(), head.to(D).requires_grad_()
    loss = dfh.vocab_loss(xs, hs, labels.to(D), reduction=reduction)
    gout = (torch.rand(m, generator=g) - 0.3) if reduction == "none" else torch.tensor(0.75)
    dx, dh = torch.autograd.grad(loss, (xs, hs), gout.to(D))
    check_loss(torch, loss.detach(), dx, dh, x, head, valid, valid.double()[:, None], labels.clamp(min=0)[:, None], 1.0,
               reduction, gout, reduction == "none")
    # one gradient alone gives the same bits, and so does a second call
    l2 = dfh.vocab_loss(xs, hs.detach(), labels.to(D), reduction=reduction)
    assert torch.equal(l2.detach(), loss.detach())
    assert torch.equal(torch.autograd.grad(l2, xs, gout.to(D))[0], dx)
    l3 = dfh.vocab_loss(xs.detach(), hs, labels.to(D), reduction=reduction)
    assert torch.equal(torch.autograd.grad(l3, hs, gout.to(D))[0], dh)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("reduction", ["none", "mean"])
@pytest.mark.parametrize("top,temp", [(1, 1.0), (7, 2.0), (64, 1.0), (200, 0.5)])
@pytest.mark.parametrize("m,v,h", [(1, 300, 8), (20, 1000, 128), (130, 517, 264), (300, 4100, 64)])
def test_distill_loss(torch, m, v, h, top, temp, reduction, dtype):
    dt, D = getattr(torch, dtype), dev(torch)
    x, head = head_and_x(torch, m, v, h, dt, seed=m + top)
    g = torch.Generator().manual_seed(m + v)
    teacher, index = (torch.randn(m, v, generator=g) * 2).topk(top, dim=1)
    tdt = [torch.float32, torch.bfloat16, torch.float16][(m + top) % 3]
    teacher = teacher.to(tdt)
    if m > 1:
        index[3:5] = -1                                           # rows without entries
        index[torch.rand(m, top, generator=g) < 0.2] = v + 5      # padding inside rows
        if top > 4:
            index[6, 2] = index[6, 0] = index[6, 1] = 11          # the same index three times
            teacher[7, 1] = -float("inf")                         # an entry of no weight
    there = (index >= 0) & (index < v)
    valid = there.any(1)
    x[~valid] = float("inf")
    t = torch.softmax((teacher.double() / temp).masked_fill(~there, -math.inf), dim=1)
    t = torch.where(valid[:, None], t, 0.0)
    idx = torch.where(there, index, 0)
    xs, hs = x.to(D).requires_grad_(), head.to(D).requires_grad_()
    loss = dfh.distill_loss(xs, hs, teacher.to(D), index.to(D), temperature=temp, reduction=reduction)
    gout = (torch.rand(m, generator=g) + 0.5) if reduction == "none" else torch.tensor(1.5)
    dx, dh = torch.autograd.grad(loss, (xs, hs), gout.to(D))
    check_loss(torch, loss.detach(), dx, dh, x, head, valid, t, idx, temp, reduction, gout, reduction == "none")


def test_distill_of_the_student_itself_is_zero(torch):
    # teacher = the student's own logits over the whole vocabulary: loss 0, gradient 0
    D = dev(torch)
    x, head = head_and_x(torch, 12, 96, 64, torch.bfloat16, 3)
    z = (x.double() @ head.double().t())
    index = torch.arange(96).expand(12, 96)
    xs = x.to(D).requires_grad_()
    loss = dfh.distill_loss(xs, head.to(D), z.float().to(D), index.contiguous().to(D), reduction="none")
    dx, = torch.autograd.grad(loss.sum(), xs)
    # p and t agree to the float32 error of a logit (at most 64 e sum |x| |head|) and 16 e
    b = (64 + 16) * E * (x.double().abs() @ head.double().abs().t()).amax() + 64 * E
    assert float(loss.detach().abs().max()) <= float(b)
    assert float(dx.abs().max()) <= float(4 * b * head.double().abs().sum(0).max())


def test_loss_edges(torch):
    D = dev(torch)
    x, head = head_and_x(torch, 6, 50, 64, torch.bfloat16, 1)
    xs, hs = x.to(D).requires_grad_(), head.to(D).requires_grad_()
    none = torch.full((6,), -100, device=D)
    for red, shape in (("none", (6,)), ("sum", ()), ("mean", ())):
        loss = dfh.vocab_loss(xs, hs, none, reduction=red)       # nothing to learn from
        assert loss.shape == shape and float(loss.detach().abs().sum()) == 0.0
        gr = torch.autograd.grad(loss.sum(), (xs, hs))
        assert all(float(t.abs().sum()) == 0.0 for t in gr)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=D).requires_grad_()   # no rows at all
    for red in ("none", "sum", "mean"):
        loss = dfh.vocab_loss(e, hs, torch.empty(0, dtype=torch.int64, device=D), reduction=red)
        assert float(loss.detach().sum()) == 0.0
        dx, dh = torch.autograd.grad(loss.sum(), (e, hs))
        assert dx.shape == (0, 64) and float(dh.abs().sum()) == 0.0
    # labels outside the vocabulary: NaN in their row, no gradient from it, others kept
    good = torch.tensor([1, 49, 0, 7, 9, 30], device=D)
    bad = good.clone()
    bad[1], bad[3] = 50, -1
    lg = dfh.vocab_loss(xs, hs, good, reduction="none")
    lb = dfh.vocab_loss(xs, hs, bad, reduction="none")
    keep = [0, 2, 4, 5]
    assert torch.isnan(lb[[1, 3]]).all() and torch.equal(lb[keep], lg[keep])
    dg = torch.autograd.grad(lg, xs, torch.ones(6, device=D))[0]
    db = torch.autograd.grad(lb, xs, torch.ones(6, device=D))[0]
    assert torch.equal(db[keep], dg[keep]) and float(db[[1, 3]].abs().sum()) == 0.0
    # another ignore_index, in reach of the vocabulary
    li = dfh.vocab_loss(xs, hs, good, ignore_index=7, reduction="none")
    assert float(li.detach()[3]) == 0.0 and torch.equal(li[keep], lg[keep])
    # vocabulary entries that are shut off by a huge negative bias direction: -inf logits
    hx = head.clone()
    hx[10:20] = -float("inf")
    xp = x.abs() + 0.1
    li = dfh.vocab_loss(xp.to(D), hx.to(D), good, reduction="none")
    rest = torch.cat([head[:10], head[20:]])
    lab = torch.tensor([1, 39, 0, 7, 9, 20])
    ref = dfh.vocab_loss(xp.to(D), rest.to(D), lab.to(D), reduction="none")
    # a different tile cut of the same terms: float32 sums of 40 terms
    assert float((li - ref).abs().max()) <= 64 * E * float(ref.abs().max() + 8)


def test_loss_strides_and_shapes(torch):
    D = dev(torch)
    x, head = head_and_x(torch, 24, 77, 64, torch.float16, 2)
    labels = torch.randint(0, 77, (24,), generator=torch.Generator().manual_seed(0)).to(D)
    want = dfh.vocab_loss(x.to(D), head.to(D), labels, reduction="none")
    wide = torch.zeros(24, 200, dtype=torch.float16, device=D)
    wide[:, 16:80] = x.to(D)
    hw = torch.zeros(77, 72, dtype=torch.float16, device=D)
    hw[:, :64] = head.to(D)
    ht = head.to(D).t().contiguous().t()
    assert torch.equal(dfh.vocab_loss(wide[:, 16:80], hw[:, :64], labels, reduction="none"), want)
    assert torch.equal(dfh.vocab_loss(wide[:, 16:80], ht, labels, reduction="none"), want)
    got = dfh.vocab_loss(x.to(D).view(4, 6, 64), head.to(D), labels.view(4, 6), reduction="none")
    assert got.shape == (4, 6) and torch.equal(got.view(-1), want)
    one = dfh.vocab_loss(x.to(D)[0], head.to(D), labels[0], reduction="none")
    assert one.shape == () and torch.equal(one, dfh.vocab_loss(x.to(D)[:1], head.to(D), labels[:1], reduction="none")[0])
    # gradients have the inputs' shapes, and go through strided inputs
    leaf = wide.clone().requires_grad_()
    hleaf = ht.clone().requires_grad_()
    loss = dfh.vocab_loss(leaf[:, 16:80], hleaf, labels)
    dl, dh = torch.autograd.grad(loss, (leaf, hleaf))
    xs, hs = x.to(D).requires_grad_(), head.to(D).requires_grad_()
    dx, dh2 = torch.autograd.grad(dfh.vocab_loss(xs, hs, labels), (xs, hs))
    assert torch.equal(dl[:, 16:80], dx) and torch.equal(dh, dh2) and float(dl[:, :16].abs().sum()) == 0.0
    # an expanded gradient of the loss
    l = dfh.vocab_loss(xs, hs, labels, reduction="none")
    a = torch.autograd.grad(l.sum(), xs, retain_graph=True)[0]
    b = torch.autograd.grad(l, xs, torch.ones(24, device=D))[0]
    assert torch.equal(a, b)


def test_loss_gradient_matches_differences(torch):
    # central differences of the float64 loss at the call's own inputs
    D = dev(torch)
    x, head = head_and_x(torch, 4, 40, 16, torch.bfloat16, 8)
    labels = torch.tensor([3, -100, 39, 0])
    xs, hs = x.to(D).requires_grad_(), head.to(D).requires_grad_()
    dx, dh = torch.autograd.grad(dfh.vocab_loss(xs, hs, labels.to(D)), (xs, hs))

    def f(xx, hh):
        z = torch.log_softmax(xx @ hh.t(), dim=1)
        return -(z[0, 3] + z[2, 39] + z[3, 0]) / 3

    x64, h64, step = x.double(), head.double(), 1e-5
    g = torch.Generator().manual_seed(0)
    u = 2.0 ** -8
    for _ in range(20):
        dirx = torch.randn(4, 16, generator=g, dtype=torch.float64)
        dirh = torch.randn(40, 16, generator=g, dtype=torch.float64)
        num = (f(x64 + step * dirx, h64 + step * dirh) - f(x64 - step * dirx, h64 - step * dirh)) / (2 * step)
        got = (dx.double().cpu() * dirx).sum() + (dh.double().cpu() * dirh).sum()
        # dz rounded once, each gradient rounded once: at most 2 u of the summed magnitudes
        z = torch.softmax(x64 @ h64.t(), 1)
        t = torch.zeros_like(z)
        t[0, 3] = t[2, 39] = t[3, 0] = 1
        d = (z - t).abs() * torch.tensor([1, 0, 1, 1.0], dtype=torch.float64)[:, None] / 3
        mag = ((d @ h64.abs()) * dirx.abs()).sum() + ((d.t() @ x64.abs()) * dirh.abs()).sum()
        assert abs(float(num - got)) <= float(2.05 * u * mag) + 1e-8


# ----------------------------------------------------- streams, graphs, chains
def test_other_stream_and_two_calls_at_once(torch):
    D = dev(torch)
    w, _, _ = matrix(torch, 512, 256, 64, "bf16", seed=4)
    x, head = head_and_x(torch, 200, 3000, 64, torch.bfloat16, 4)
    x, head = x.to(D), head.to(D)
    labels = torch.randint(0, 3000, (200,), generator=torch.Generator().manual_seed(1)).to(D)
    xa = torch.randn(200, 256, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(D)
    want = dfh.linear_u4(xa, w), dfh.vocab_loss(x, head, labels, reduction="none")
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(8):
        outs.append((dfh.linear_u4(xa, w, stream=s1), dfh.vocab_loss(x, head, labels, reduction="none", stream=s2)))
        outs.append((dfh.linear_u4(xa, w, stream=s2.cuda_stream),
                     dfh.vocab_loss(x, head, labels, reduction="none", stream=s1)))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_graph_of_a_training_step(torch):
    """linear_u4 -> vocab_loss and its gradients, captured and replayed with
    other inputs and with eager work of the program between the replays."""
    D = dev(torch)
    n, k, v = 128, 256, 1500
    w, _, _ = matrix(torch, n, k, 64, "bf16", seed=6)
    head = head_and_x(torch, 1, v, n, torch.bfloat16, 6)[1].to(D)
    for m in (5, 150):
        x = torch.zeros(m, k, dtype=torch.bfloat16, device=D)
        labels = torch.zeros(m, dtype=torch.int64, device=D)

        def step():
            xl, hl = x.detach().requires_grad_(), head.detach().requires_grad_()
            loss = dfh.vocab_loss(dfh.linear_u4(xl, w), hl, labels)
            return (loss.detach(),) + torch.autograd.grad(loss, (xl, hl))

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
            x.copy_(torch.randn(m, k, generator=g).to(torch.bfloat16))
            labels.copy_(torch.randint(0, v, (m,), generator=g))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (m, r)


def test_input_changed_before_the_gradient_is_refused(torch):
    D = dev(torch)
    x, head = head_and_x(torch, 8, 50, 64, torch.bfloat16, 1)
    xs, hs = x.to(D).requires_grad_(), head.to(D)
    labels = torch.zeros(8, dtype=torch.int64, device=D)
    loss = dfh.vocab_loss(xs, hs, labels)
    labels.fill_(1)
    with pytest.raises(RuntimeError):
        loss.backward()


def test_refusals_on_the_device(torch):
    D = dev(torch)
    w, _, _ = matrix(torch, 16, 64, 32)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device=D)
    for bad in (torch.zeros(2, 63, dtype=torch.bfloat16, device=D), torch.zeros(2, 64, device=D), x.cpu()):
        with pytest.raises((ValueError, TypeError)):
            dfh.linear_u4(bad, w)
    p, s, z = w.packed, w.scales, w.zeros
    for kw in (dict(cols=60), dict(cols=64, group_size=48), dict(cols=64, group_size=0), dict(cols=128, group_size=64)):
        with pytest.raises(ValueError):
            dfh.U4Matrix(p, s, z, **kw)
    with pytest.raises(ValueError):
        dfh.U4Matrix(p[:-1], s, z, cols=64, group_size=32)
    with pytest.raises(ValueError):
        dfh.U4Matrix(p, s, z[:, :1], cols=64, group_size=32)
    with pytest.raises(ValueError):
        dfh.U4Matrix(p, s.float().requires_grad_(), z, cols=64, group_size=32)
    with pytest.raises(TypeError):
        dfh.U4Matrix(p, s.double(), z, cols=64, group_size=32)
    head = torch.zeros(10, 64, dtype=torch.bfloat16, device=D)
    lab = torch.zeros(2, dtype=torch.int64, device=D)
    for args in ((x, head, lab.int()), (x, head, lab[:1]), (x, head.half(), lab), (x.float(), head.float(), lab),
                 (x, head[:, :60], lab), (x[:, :60], head[:, :60], lab), (x.cpu(), head, lab), (x, head, lab.cpu())):
        with pytest.raises((ValueError, TypeError)):
            dfh.vocab_loss(*args)
    with pytest.raises(ValueError):
        dfh.vocab_loss(x, head, lab, reduction="average")
    t, i = torch.zeros(2, 4, device=D), torch.zeros(2, 4, dtype=torch.int64, device=D)
    for a, b, temp in ((t, i[:, :3], 1.0), (t, i.int(), 1.0), (t, i, 0.0), (t, i, 1e-4), (t, i, 1e4), (t, i, float("inf")), (t, i, float("nan")),
                       (t.double(), i, 1.0), (t[:, :0], i[:, :0], 1.0)):
        with pytest.raises((ValueError, TypeError)):
            dfh.distill_loss(x, head, a, b, temperature=temp)


def test_gradients_of_gradients_are_refused(torch):
    # first order under create_graph works, the second raises
    D = dev(torch)
    w, _, _ = matrix(torch, 24, 64, 32, "fp32", seed=1)
    x, head = head_and_x(torch, 5, 40, 24, torch.bfloat16, 1)
    a = torch.randn(5, 64).to(torch.bfloat16).to(D).requires_grad_()
    h = dfh.linear_u4(a, w)
    loss = dfh.vocab_loss(h, head.to(D), torch.zeros(5, dtype=torch.int64, device=D))
    plain, = torch.autograd.grad(loss, a, retain_graph=True)
    g, = torch.autograd.grad(loss, a, create_graph=True)
    assert torch.equal(g, plain)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.float().sum(), a)


def test_strided_targets(torch):
    # columns of wider tensors, rows expanded over the batch, labels with a stride
    D = dev(torch)
    x, head = head_and_x(torch, 10, 90, 64, torch.float16, 6)
    x, head = x.to(D), head.to(D)
    g = torch.Generator().manual_seed(4)
    t, i = (torch.randn(10, 90, generator=g) * 2).topk(6, dim=1)
    t, i = t.to(D), i.to(D)
    want = dfh.distill_loss(x, head, t, i, reduction="none")
    tw, iw = torch.zeros(10, 20, device=D), torch.zeros(10, 13, dtype=torch.int64, device=D)
    tw[:, 3:9], iw[:, 5:11] = t, i
    assert torch.equal(dfh.distill_loss(x, head, tw[:, 3:9], iw[:, 5:11], reduction="none"), want)
    assert torch.equal(dfh.distill_loss(x, head, t.t().contiguous().t(), i.t().contiguous().t(), reduction="none"), want)
    e = dfh.distill_loss(x, head, t[:1].expand(10, 6), i[:1].expand(10, 6), reduction="none")
    assert torch.equal(e, dfh.distill_loss(x, head, t[:1].repeat(10, 1), i[:1].repeat(10, 1), reduction="none"))
    lab = torch.randint(0, 90, (10, 3), generator=g).to(D)
    assert torch.equal(dfh.vocab_loss(x, head, lab[:, 1], reduction="none"),
                       dfh.vocab_loss(x, head, lab[:, 1].contiguous(), reduction="none"))


def test_loss_in_pieces_of_the_vocabulary(torch):
    # a vocabulary of several pieces (16384 rows: 4096 entries each), the target in
    # each piece, against one call per half of the rows (pieces twice as long)
    D = dev(torch)
    m, v, h = 16384, 9000, 64
    g = torch.Generator().manual_seed(12)
    x = torch.randn(m, h, generator=g).to(torch.bfloat16).to(D)
    head = (torch.randn(v, h, generator=g) * 0.3).to(torch.bfloat16).to(D).requires_grad_()
    labels = torch.randint(0, v, (m,), generator=g).to(D)
    xs = x.clone().requires_grad_()
    loss = dfh.vocab_loss(xs, head, labels, reduction="sum")
    dx, dh = torch.autograd.grad(loss, (xs, head))
    parts = []
    for lo in (0, m // 2):
        xp = x[lo: lo + m // 2].clone().requires_grad_()
        lp = dfh.vocab_loss(xp, head, labels[lo: lo + m // 2], reduction="sum")
        parts.append((lp.detach(),) + torch.autograd.grad(lp, (xp, head)))
    # a float64 run of the whole on the GPU
    z = x.double() @ head.detach().double().t()
    p = torch.softmax(z, 1)
    ref = torch.nn.functional.cross_entropy(z, labels, reduction="sum")
    p[torch.arange(m, device=D), labels] -= 1
    assert abs(float(loss.detach()) - float(ref)) <= float(ref) * 64 * E * 8
    u = 2.0 ** -8
    a = p.abs()
    bx = ((u + 1e-4) * a @ head.detach().double().abs()) + u * 1.1 * (p @ head.detach().double()).abs()
    bh = ((u + 1e-4) * a.t() @ x.double().abs()) + u * 1.1 * (p.t() @ x.double()).abs()
    assert bool(((dx.double() - p @ head.detach().double()).abs() <= bx).all())
    assert bool(((dh.double() - p.t() @ x.double()).abs() <= bh).all())
    assert abs(float(parts[0][0] + parts[1][0]) - float(ref)) <= float(ref) * 64 * E * 8
    assert bool(((torch.cat([parts[0][1], parts[1][1]]).double() - p @ head.detach().double()).abs() <= bx).all())
