"""Products in 8-bit integers on the GPU, against the definition in float64, where
every sum of code products is exact.

Tolerances.  Codes have to be equal: of two 16-bit floats, 127 x / top is half way
between two integers or at least 2^-19 of itself away from there, which float64 and
the kernels both tell apart.  A scale top / 127 is rounded once, to e = 2^-24 of
itself (or half of float32's smallest subnormal).  An output is a sum converted to
float32, times two scales of which one was rounded (four roundings of e; 5 e covers
their products), rounded once to its type.
"""
import numpy as np
import pytest

import lossless_entropy_coded_huffman_amd as dfh

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def types(torch):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def quantised(torch, x):
    """Codes and scales of finite rows in float64."""
    x = x.cpu().double()
    top = x.abs().amax(dim=-1, keepdim=True)
    codes = torch.round(127 * x / torch.where(top > 0, top, 1.0))
    return codes, (top / 127).squeeze(-1)


def matrix(torch, n, k, scale="fp32", zeros=True, broadcast=False, seed=0, codes=None):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (n, k), generator=g, dtype=torch.uint8) if codes is None else codes
    r = 1 if broadcast else n
    s = ((torch.rand(r, generator=g) + 0.5) * 1e-3 * torch.where(torch.rand(r, generator=g) < 0.1, -1.0, 1.0)) \
        .to(types(torch)[scale])
    z = torch.randint(0, 256, (r,), generator=g, dtype=torch.uint8) if zeros else None
    w = dfh.U8Matrix(q.cuda(), s.cuda().expand(n), z.cuda().expand(n) if zeros else None, cols=k)
    zz = z.double().expand(n) if zeros else torch.full((n,), 128.0, dtype=torch.float64)
    return w, q.double() - zz[:, None], s.double().expand(n)


def check(torch, got, codes, xs, w64, s):
    ref = (codes @ w64.t()) * xs.reshape(-1, 1) * s
    u = torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -134
    bound = ref.abs() * ((1 + 5 * E) * (1 + u) - 1) + tiny
    err = (got.double().cpu().reshape(ref.shape) - ref).abs()
    assert bool((err <= bound).all()), "off by %g of the bound" % float((err / bound).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 37, 48), (2, 129, 1024), (3, 64, 1040), (4, 1000, 2064), (1, 8195, 96),
                                   (4, 8200, 528), (1, 17, 61440), (2, 33, 32768), (5, 31, 16), (7, 513, 4096),
                                   (16, 64, 1040), (33, 100, 160), (65, 200, 2048), (64, 1024, 14336), (130, 257, 272),
                                   (300, 511, 1424), (517, 2047, 1040)])
def test_product(torch, m, n, k, dtype):
    w, w64, s = matrix(torch, n, k, scale="fp32" if m % 2 else dtype, zeros=(m + n) % 3 > 0, broadcast=n % 2 == 0, seed=m)
    g = torch.Generator().manual_seed(k)
    x = (torch.randn(m, k, generator=g) * torch.rand(m, 1, generator=g) * 4).to(types(torch)[dtype])
    codes, xs = quantised(torch, x)
    check(torch, dfh.linear_u8(x.cuda(), w), codes, xs, w64, s)
    c, sc = dfh.quantize_rows(x.cuda())
    assert torch.equal(c.cpu().double(), codes)
    assert bool(((sc.cpu().double() - xs).abs() <= xs * E).all())
    check(torch, dfh.linear_u8(c, w, scales=sc, dtype=types(torch)[dtype]), codes, xs, w64, s)


@pytest.mark.parametrize("m", [1, 4, 9, 300])
@pytest.mark.parametrize("x_code,w_code,zero", [(127, 255, 0), (-127, 255, 0), (127, 0, 255), (-128, 0, 255), (-128, 255, 0)])
def test_largest_sums(torch, m, x_code, w_code, zero):
    # 65536 terms of the largest size: one more bit would not fit
    n, k = 24, 65536
    q = torch.full((n, k), w_code, dtype=torch.uint8)
    one = torch.ones(n)
    w = dfh.U8Matrix(q.cuda(), one.cuda(), torch.full((n,), zero, dtype=torch.uint8).cuda(), cols=k)
    c = torch.full((m, k), x_code, dtype=torch.int8)
    y = dfh.linear_u8(c.cuda(), w, scales=torch.full((m,), 2.0 ** -20).cuda(), dtype=torch.bfloat16)
    ref = float(k * x_code * (w_code - zero)) * 2.0 ** -20
    assert bool((y.double().cpu() - ref).abs().le(abs(ref) * (2.0 ** -8 + 5 * E)).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("k", [64, 4096, 9008])
def test_codes_of_hard_rows(torch, k, dtype):
    dt = types(torch)[dtype]
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(12, k, generator=g)
    x = rows.to(dt)
    top = torch.finfo(dt).max
    x[0] = 0                                                     # nothing
    x[1] = (torch.randint(-1, 2, (k,), generator=g) * 0.5).to(dt)  # ties: half of the largest
    x[1, 0] = 1
    x[2] = (torch.rand(k, generator=g).double() * 2 - 1).mul(top).to(dt)   # the type's largest
    x[2, -1] = top
    x[3] = (x[3].float() * torch.finfo(dt).tiny).to(dt)            # subnormals
    x[4] = 0
    x[4, k // 2] = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps   # the smallest
    x[5] = torch.randint(-127, 128, (k,), generator=g).to(dt)      # multiples of a 254th
    x[5, 3] = 127
    x[6] = (torch.randint(-254, 255, (k,), generator=g).float() / 2).to(dt)
    x[6, k - 1] = -127
    c, s = dfh.quantize_rows(x.cuda())
    codes, xs = quantised(torch, x)
    assert torch.equal(c.cpu().double(), codes)
    assert bool(((s.cpu().double() - xs).abs() <= xs * E + 2.0 ** -150).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_codes_at_every_exponent(torch, dtype):
    # rows whose largest value has each exponent that the type has, subnormals' too
    dt = types(torch)[dtype]
    low, high = (-24, 15) if dtype == "fp16" else (-133, 127)
    e = torch.arange(low, high + 1, dtype=torch.float64)
    g = torch.Generator().manual_seed(8)
    part = torch.rand(len(e), 96, generator=g).double() * 2 - 1
    part[:, 5] = 1
    x = (part * torch.exp2(e)[:, None]).to(dt)
    codes, xs = quantised(torch, x)
    c, sc = dfh.quantize_rows(x.cuda())
    assert torch.equal(c.cpu().double(), codes)
    assert bool(((sc.cpu().double() - xs).abs() <= xs * E + 2.0 ** -150).all())
    # few rows are quantised by the product itself
    w = dfh.U8Matrix(torch.full((96, 96), 128, dtype=torch.uint8).cuda() + torch.eye(96, dtype=torch.uint8).cuda(),
                     torch.ones(96).cuda(), None, cols=96)
    for i in range(0, len(e), 4):
        y = dfh.linear_u8(x[i:i + 4].cuda(), w)
        tiny = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134
        ref = codes[i:i + 4] * xs[i:i + 4, None]
        u = torch.finfo(dt).eps / 2
        near = ref.abs() * ((1 + 5 * E) * (1 + u) - 1) + tiny + 127 * 2.0 ** -150
        assert bool(((y.double().cpu() - ref).abs() <= near).all())


@pytest.mark.parametrize("m", [1, 3, 40])
def test_rows_that_are_not_finite(torch, m):
    # each spoils its own row alone
    n, k = 70, 2064
    w, w64, s = matrix(torch, n, k)
    for dt in (torch.bfloat16, torch.float16):
        for bad in (float("nan"), float("inf"), -float("inf")):
            x = torch.randn(m, k, generator=torch.Generator().manual_seed(1)).to(dt)
            x[m - 1, k - 5] = bad
            y = dfh.linear_u8(x.cuda(), w)
            assert bool(y[m - 1].isnan().all())
            c, sc = dfh.quantize_rows(x.cuda())
            assert not c[m - 1].any() and bool(sc[m - 1].isnan())
            if m > 1:
                codes, xs = quantised(torch, x[:-1])
                check(torch, y[:-1], codes, xs, w64, s)


@pytest.mark.parametrize("m", [1, 3, 130])
def test_layouts(torch, m):
    n, k = 96, 528
    w, w64, s = matrix(torch, n, k)
    g = torch.Generator().manual_seed(m)
    base = torch.randn(m, 2, k + 24, generator=g).to(torch.bfloat16)
    whole = base.cuda()
    plain = base[:, 1, :k].contiguous().cuda()
    want = dfh.linear_u8(plain, w)
    codes, scales = dfh.quantize_rows(plain)
    views = [whole[:, 1, :k], whole[:, 1, 3: 3 + k][:, :], whole.transpose(0, 1)[1][:, :k]]
    views[1] = torch.cat([plain.new_zeros(m, 3), plain], 1)[:, 3:]             # 2-byte aligned
    views.append(plain.t().contiguous().t())                                    # columns apart
    for v in views:
        assert torch.equal(dfh.linear_u8(v, w), want)
        c, sc = dfh.quantize_rows(v)
        assert torch.equal(c, codes) and torch.equal(sc, scales)
    assert torch.equal(dfh.linear_u8(plain.view(1, m, 1, k), w).view(m, n), want)
    assert torch.equal(dfh.linear_u8(plain[0], w), want[0]) or m > 4            # another kernel for one row
    odd = torch.cat([codes.new_zeros(m, 5), codes], 1)[:, 5:]
    twice = torch.stack([scales, scales], 1)[:, 0]
    for c in (codes, odd, codes.t().contiguous().t()):
        assert torch.equal(dfh.linear_u8(c, w, scales=twice), want)
    assert dfh.linear_u8(plain[:0], w).shape == (0, n)
    assert dfh.quantize_rows(plain[:0])[0].shape == (0, k)


def test_many_rows(torch):
    # more rows than a launch's grid is cut for, in both kernels that take a row at a time
    m, n, k = 70001, 24, 2080
    w, w64, s = matrix(torch, n, k)
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(0)).to(torch.float16)
    y = dfh.linear_u8(x.cuda(), w)
    for part in (slice(0, 100), slice(65500, 65600), slice(m - 100, m)):
        codes, xs = quantised(torch, x[part])
        check(torch, y[part], codes, xs, w64, s)


def test_scales_of_any_size(torch):
    # x's scale times the weights' leaves float32's range, the outputs do not
    m, n, k = 3, 40, 256
    for rows in (m, 40):
        w, w64, _ = matrix(torch, n, k, zeros=False)
        g = torch.Generator().manual_seed(2)
        x = (torch.randn(rows, k, generator=g) * 1e36).to(torch.bfloat16)
        s = torch.full((n,), 1e-38)
        w = dfh.U8Matrix(w.codes, s.cuda(), None, cols=k)
        codes, xs = quantised(torch, x)
        check(torch, dfh.linear_u8(x.cuda(), w), codes, xs, w64, s.double())


@pytest.mark.parametrize("m", [2, 50, 700])
def test_on_a_stream_and_captured(torch, m):
    n, k = 300, 1040
    w, _, _ = matrix(torch, n, k)
    g = torch.Generator().manual_seed(m)
    xs = [torch.randn(m, k, generator=g).to(torch.bfloat16).cuda() for _ in range(3)]
    want = [dfh.linear_u8(x, w) for x in xs]
    s = torch.cuda.Stream()
    late = torch.zeros_like(xs[0]).t().contiguous().t()        # laid out anew, on the call's stream
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    with torch.cuda.stream(s):
        late.copy_(xs[0])
    got = dfh.linear_u8(late, w, stream=s)
    codes = dfh.quantize_rows(late, stream=s)
    both = dfh.linear_u8(codes[0], w, scales=codes[1], stream=s)
    s.synchronize()
    assert torch.equal(got, want[0]) and torch.equal(both, want[0])
    torch.cuda.synchronize()
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = dfh.linear_u8(x, w)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        dfh.linear_u8(xs[0], w)
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])


def test_a_container_s_codes(torch):
    # quantised as the codec's uint8 layers are, compressed, decoded and multiplied
    n, k = 256, 512
    rng = np.random.default_rng(0)
    wt = rng.normal(0, 0.02, (n, k)).astype(np.float32)
    s = np.abs(wt).max() / 127
    q = (np.rint(wt / s) + 128).astype(np.uint8)
    dc = dfh.to_device(dfh.compress(dfh.KIND_U8, q.reshape(-1)), torch.device("cuda:0"))
    out = dc.empty_output()
    dfh.df_decompress(dc, out)
    w = dfh.U8Matrix(out, torch.tensor([s]).cuda().expand(n), None, cols=k)
    x = torch.randn(6, k, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    codes, xs = quantised(torch, x)
    check(torch, dfh.linear_u8(x.cuda(), w), codes, xs, torch.from_numpy(q.astype(np.float64) - 128),
          torch.full((n,), float(np.float32(s)), dtype=torch.float64))


def test_refused_calls(torch):
    n, k = 32, 64
    w, _, _ = matrix(torch, n, k)
    q, s = w.codes, w.scales
    x = torch.zeros(3, k, dtype=torch.bfloat16, device="cuda")
    codes, scales = dfh.quantize_rows(x)
    with pytest.raises(RuntimeError):
        dfh.linear_u8(x.clone().requires_grad_(), w)
    with pytest.raises(RuntimeError):
        dfh.quantize_rows(x.clone().requires_grad_())
    with torch.no_grad():
        dfh.linear_u8(x.clone().requires_grad_(), w)
    for a in (x.float(), codes):
        with pytest.raises(TypeError):
            dfh.linear_u8(a, w)
    with pytest.raises(TypeError):
        dfh.linear_u8(x, w, scales=scales)
    with pytest.raises(TypeError):
        dfh.linear_u8(x, w, dtype=torch.float16)
    with pytest.raises(TypeError):
        dfh.linear_u8(codes, w, scales=scales, dtype=torch.float32)
    for a in (x[:, :48], x.cpu()):
        with pytest.raises(ValueError):
            dfh.linear_u8(a, w)
    for sc in (scales[:2], scales.double(), scales.cpu()):
        with pytest.raises(ValueError):
            dfh.linear_u8(codes, w, scales=sc)
    for a in (x[:, :40], x.cpu(), x.new_zeros(())):
        with pytest.raises(ValueError):
            dfh.quantize_rows(a)
    with pytest.raises(TypeError):
        dfh.quantize_rows(x.float())
    for bad in (dict(codes=q[: n // 2]), dict(cols=40), dict(cols=1 << 17), dict(codes=q.view(torch.int8)),
                dict(scales=s.view(n // 2, 2)), dict(zeros=torch.zeros(n, device="cuda")), dict(codes=q.cpu()),
                dict(scales=s.cpu()), dict(zeros=torch.zeros(n - 1, dtype=torch.uint8, device="cuda")),
                dict(codes=q.view(-1)[1:], cols=16)):
        a = dict(codes=q, scales=s, zeros=None, cols=k)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            dfh.U8Matrix(a["codes"], a["scales"], a["zeros"], cols=a["cols"])
    with pytest.raises(TypeError):
        dfh.U8Matrix(q, s.double(), None, cols=k)
