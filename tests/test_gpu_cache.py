"""The paged cache on the GPU: what is written and read back, against the definition.

Codes have to be equal, and so has everything kept in 16 bits.  A scale is rounded once
from max |x| / 127, to 2^-24 of itself (or half of float32's smallest subnormal).  A
value read back is a code times that scale in float32 (rounded once more, exact in
float64 here), rounded to the cache's type: what float32 and the type give for the
stored code and scale, bit for bit.
"""
import random

import pytest

import lossless_entropy_coded_huffman_amd as dfh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def types(torch):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}


def batch_of(torch, new, lengths, page, *, width=None, spare=3, seed=0, shuffle=True, max_new=None):
    """(CacheBatch, tables as lists, pages in the pool) with pages of their own for every
    sequence, anywhere in the pool."""
    used = [(t + page - 1) // page for t in lengths]
    width = width or max([1] + used)
    order = list(range(sum(used) + spare))
    if shuffle:
        random.Random(seed).shuffle(order)
    tables, at = [], 0
    for u in used:
        tables.append(order[at: at + u] + [(1 << 30)] * (width - u))
        at += u
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    t = torch.tensor(tables, dtype=torch.int32).reshape(len(new), width)
    b = dfh.CacheBatch(t.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                       torch.tensor(starts, dtype=torch.int32).cuda(), max_new=max_new)
    return b, tables, len(order)


def places(tables, new, lengths, page):
    """(page, row) of every new token, None where there is none."""
    out = []
    for table, n, length in zip(tables, new, lengths):
        for p in range(length - n, length):
            out.append((table[p // page], p % page) if 0 <= p and p // page < len(table) else None)
    return out


def quantised(torch, x):
    x = x.cpu().double()
    top = x.abs().amax(dim=-1, keepdim=True)
    return torch.round(127 * x / torch.where(top > 0, top, 1.0)).to(torch.int8), (top / 127).squeeze(-1)


def check_written(torch, cache, k, v, where, fill):
    """Every row of the pool: written ones by the definition, others as they were."""
    for name, x in (("k", k), ("v", v)):
        got = getattr(cache, name).cpu()
        want = torch.full_like(got, fill)
        if cache.bits == 8:
            scales = getattr(cache, name + "_scales").cpu().double()
            wants = torch.full_like(scales, fill)
            codes, s = quantised(torch, x)
        else:
            codes = x.cpu()
        for i, at in enumerate(where):
            if at is not None:
                want[at[0], :, at[1]] = codes[i]
                if cache.bits == 8:
                    wants[at[0], :, at[1]] = s[i]
        assert torch.equal(got, want)
        if cache.bits == 8:
            assert bool(((scales - wants).abs() <= wants.abs() * 2.0 ** -24 + 2.0 ** -150).all())


def filled(torch, cache, value):
    for t in cache._tensors():
        if t is not None:
            t.fill_(value)
    return cache


CASES = [
    # kv_heads, head_dim, page, new, lengths
    (1, 32, 16, [1], [1]),
    (8, 128, 64, [1, 1, 1], [1, 64, 65]),
    (8, 128, 64, [1] * 70, [1 + 7 * i for i in range(70)]),
    (3, 64, 16, [0, 5, 0, 0, 17, 1, 0], [9, 5, 0, 40, 33, 16, 1]),
    (2, 256, 32, [33, 100], [33, 131]),
    (5, 32, 256, [300, 0, 2], [300, 17, 514]),
    (1, 128, 128, [1000], [1001]),
    (256, 32, 16, [3, 2], [3, 20]),
]


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_write_and_read(torch, case, dtype, bits):
    kv, dim, page, new, lengths = CASES[case]
    dt = types(torch)[dtype]
    b, tables, pages = batch_of(torch, new, lengths, page, seed=case)
    cache = filled(torch, dfh.KVCache(pages, kv, dim, page_size=page, dtype=dt, bits=bits), 77)
    g = torch.Generator().manual_seed(case)
    n = sum(new)
    k, v = ((torch.randn(n, kv, dim, generator=g) * 10 ** torch.randn(n, kv, 1, generator=g)).to(dt).cuda() for _ in range(2))
    dfh.cache_write(k, v, cache, b)
    check_written(torch, cache, k, v, places(tables, new, lengths, page), 77)
    rk, rv = dfh.cache_read(cache, b, n)
    if bits == 16:
        assert torch.equal(rk, k) and torch.equal(rv, v)
        return
    for got, name in ((rk, "k"), (rv, "v")):
        at = [w for w in places(tables, new, lengths, page)]
        p, r = (torch.tensor([w[i] for w in at], device="cuda") for i in (0, 1))
        codes, s = getattr(cache, name)[p, :, r], getattr(cache, name + "_scales")[p, :, r]
        assert torch.equal(got, (codes.float() * s[..., None]).to(dt))


@pytest.mark.parametrize("bits", [8, 16])
def test_tokens_that_are_not_there(torch, bits):
    # new tokens before position 0, outside the table, on pages outside the pool, and
    # rows before the first and behind the last sequence: nothing is touched for them
    page, kv, dim = 16, 2, 64
    tables = torch.tensor([[0, 1], [-1, 2], [3, 1 << 30], [4, 5], [6, 7]], dtype=torch.int32)
    lengths = [3, 20, 20, 40, 20]
    starts = [2, 7, 27, 37, 47, 49]
    cache = filled(torch, dfh.KVCache(8, kv, dim, page_size=page, bits=bits), 55)
    b = dfh.CacheBatch(tables.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                       torch.tensor(starts, dtype=torch.int32).cuda())
    n = 60
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(n, kv, dim, generator=g).to(torch.bfloat16) for _ in range(2))
    where = [None] * n
    for s in range(5):
        for r in range(starts[s], starts[s + 1]):
            p = lengths[s] - starts[s + 1] + r
            if 0 <= p < 32 and 0 <= int(tables[s, p // page]) < 8:
                where[r] = (int(tables[s, p // page]), p % page)
    k[[0, 1, 50, 59]] = float("nan")
    dfh.cache_write(k.cuda(), v.cuda(), cache, b)
    check_written(torch, cache, torch.nan_to_num(k), v, where, 55)
    rk, rv = dfh.cache_read(cache, b, n)
    gone = torch.tensor([w is None for w in where])
    assert not rk.cpu()[gone].any() and not rv.cpu()[gone].any()
    assert rk.cpu()[~gone].any(dim=2).all()
    if bits == 16:
        assert torch.equal(rv.cpu()[~gone], v[~gone])


@pytest.mark.parametrize("begin", [1, 3, 70])
def test_rows_before_the_first_sequence(torch, begin):
    # the first tokens share a wave with rows of no sequence
    page, kv, dim, new, lengths = 16, 1, 32, [2, 0, 9], [2, 5, 30]
    b, tables, pages = batch_of(torch, new, lengths, page)
    b = dfh.CacheBatch(b.tables, b.lengths, b.starts + begin)
    cache = filled(torch, dfh.KVCache(pages, kv, dim, page_size=page), 7)
    n = begin + sum(new) + 2
    k = torch.randn(n, kv, dim, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    dfh.cache_write(k.cuda(), -k.cuda(), cache, b)
    where = [None] * begin + places(tables, new, lengths, page) + [None] * 2
    check_written(torch, cache, k, -k, where, 7)
    back = dfh.cache_read(cache, b, n)[0].cpu()
    assert torch.equal(back[begin: -2], k[begin: -2]) and not back[:begin].any() and not back[-2:].any()


def test_no_sequences_and_no_tokens(torch):
    cache = filled(torch, dfh.KVCache(2, 1, 32, page_size=16), 1)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    b = dfh.CacheBatch(none.view(0, 1), none, torch.zeros(1, dtype=torch.int32, device="cuda"))
    x = torch.ones(3, 1, 32, dtype=torch.bfloat16, device="cuda") * 2
    dfh.cache_write(x, x, cache, b)
    assert bool((cache.k == 1).all())
    assert not any(t.any() for t in dfh.cache_read(cache, b, 3))
    b2, _, _ = batch_of(torch, [0, 0], [5, 0], 16, spare=2)
    dfh.cache_write(x[:0], x[:0], cache, b2)
    assert dfh.cache_read(cache, b2, 0)[0].shape == (0, 1, 32)
    assert bool((cache.k == 1).all())


def test_vectors_that_are_not_finite(torch):
    kv, dim, page = 2, 128, 16
    for dt in (torch.bfloat16, torch.float16):
        b, tables, pages = batch_of(torch, [6], [6], page)
        cache = dfh.KVCache(pages, kv, dim, page_size=page, dtype=dt, bits=8)
        x = torch.randn(6, kv, dim, generator=torch.Generator().manual_seed(0)).to(dt)
        x[0, 0, 5], x[1, 1, 127], x[2, 0, 0] = float("nan"), float("inf"), -float("inf")
        x[3] = 0
        bad = torch.zeros(6, kv, dtype=torch.bool)
        bad[0, 0] = bad[1, 1] = bad[2, 0] = True
        dfh.cache_write(x.cuda(), x.cuda(), cache, b)
        for t in dfh.cache_read(cache, b, 6):
            t = t.cpu()
            assert bool(t[bad].isnan().all()) and bool(t[~bad].isfinite().all()) and not t[3].any()
        page0 = tables[0][0]
        assert not cache.k[page0, 0, 0].any() and bool(cache.k_scales[page0, 0, 0].isnan())


@pytest.mark.parametrize("bits", [8, 16])
def test_layouts_and_streams(torch, bits):
    kv, dim, page, new, lengths = 4, 64, 32, [7, 0, 40], [50, 3, 40]
    n = sum(new)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(n, kv, dim, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    b, tables, pages = batch_of(torch, new, lengths, page)
    want = dfh.KVCache(pages, kv, dim, page_size=page, bits=bits)
    dfh.cache_write(k, v, want, b)
    both = torch.cat([k, v], dim=2)                                 # one tensor of both
    forms = [(both[..., :dim], both[..., dim:]),
             (k.transpose(0, 1).contiguous().transpose(0, 1), v.transpose(1, 2).contiguous().transpose(1, 2)),
             (torch.cat([k.new_zeros(n, kv, 1), k], 2)[..., 1:], v)]
    for fk, fv in forms:
        cache = dfh.KVCache(pages, kv, dim, page_size=page, bits=bits)
        dfh.cache_write(fk, fv, cache, b)
        assert torch.equal(cache.k, want.k) and torch.equal(cache.v, want.v)
    # a table that is part of a wider one
    wide = torch.full((3, 9), 1 << 30, dtype=torch.int32)
    wide[:, 2: 2 + b.width] = b.tables.cpu()
    cache = dfh.KVCache(pages, kv, dim, page_size=page, bits=bits)
    dfh.cache_write(k, v, cache, dfh.CacheBatch(wide.cuda()[:, 2: 2 + b.width], b.lengths, b.starts))
    assert torch.equal(cache.k, want.k) and torch.equal(cache.v, want.v)
    # another stream, with late work on the current one
    s = torch.cuda.Stream()
    late = torch.zeros(n, dim, kv, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    cache = dfh.KVCache(pages, kv, dim, page_size=page, bits=bits)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    with torch.cuda.stream(s):
        late.copy_(k)
    dfh.cache_write(late, v, cache, b, stream=s)
    got = dfh.cache_read(cache, b, n, stream=s)
    s.synchronize()
    assert torch.equal(cache.k, want.k) and torch.equal(got[0], dfh.cache_read(want, b, n)[0])
    torch.cuda.synchronize()


def test_captured_steps(torch):
    # one graph writes a token at whatever position the batch's tensors then name
    kv, dim, page = 2, 128, 16
    tables = torch.tensor([[3, 1], [0, 2]], dtype=torch.int32).cuda()
    lengths = torch.tensor([1, 9], dtype=torch.int32).cuda()
    b = dfh.CacheBatch(tables, lengths, torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), max_new=1)
    cache = dfh.KVCache(4, kv, dim, page_size=page, bits=8)
    eager = dfh.KVCache(4, kv, dim, page_size=page, bits=8)
    x = torch.randn(24, 2, kv, dim, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    k = x[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dfh.cache_write(k, k, cache, b)
        back = dfh.cache_read(cache, b, 2)
    for i in range(24):
        lengths.copy_(torch.tensor([1 + i, 9 + i], dtype=torch.int32))
        k.copy_(x[i])
        graph.replay()
        dfh.cache_write(x[i], x[i], eager, b)
        assert torch.equal(cache.k, eager.k) and torch.equal(cache.v_scales, eager.v_scales)
        assert torch.equal(back[0], dfh.cache_read(eager, b, 2)[0])


def test_a_pool_beyond_32_bits(torch):
    # rows whose byte and element offsets pass 2^32
    kv, dim, page = 8, 128, 256
    pages = 17000                                      # 4.46e9 elements
    cache = dfh.KVCache(pages, kv, dim, page_size=page, bits=8)
    tables = torch.tensor([[pages - 1, 16384, 5]], dtype=torch.int32).cuda()
    b = dfh.CacheBatch(tables, torch.tensor([600], dtype=torch.int32).cuda(), torch.tensor([0, 600], dtype=torch.int32).cuda())
    x = torch.randn(600, kv, dim, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    dfh.cache_write(x.cuda(), x.cuda(), cache, b)
    codes, _ = quantised(torch, x)
    for i, p in enumerate((pages - 1, 16384, 5)):
        part = codes[256 * i: 256 * (i + 1)]
        assert torch.equal(cache.k[p, :, : len(part)].cpu(), part.transpose(0, 1))
        assert torch.equal(cache.v[p, :, : len(part)].cpu(), part.transpose(0, 1))
    got = dfh.cache_read(cache, b, 600)[0].cpu()
    scales = torch.cat([cache.k_scales[p] for p in (pages - 1, 16384, 5)], 1)[:, :600].t().cpu()
    assert torch.equal(got, (codes.float() * scales[..., None]).to(torch.bfloat16))
    assert int(cache.k.view(-1).view(torch.int64).ne(0).sum()) <= 600 * kv * dim // 8


def test_many_sequences(torch):
    # 5000 sequences, many without a new token: found by three rounds of search
    kv, dim, page = 1, 32, 16
    rng = random.Random(4)
    new = [rng.choice([0, 0, 1, 2, 19]) for _ in range(5000)]
    lengths = [n + rng.randrange(20) for n in new]
    b, tables, pages = batch_of(torch, new, lengths, page, seed=5)
    cache = filled(torch, dfh.KVCache(pages, kv, dim, page_size=page), 3)
    n = sum(new)
    k = torch.randn(n, kv, dim, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    dfh.cache_write(k.cuda(), -k.cuda(), cache, b)
    check_written(torch, cache, k, -k, places(tables, new, lengths, page), 3)
    assert torch.equal(dfh.cache_read(cache, b, n)[0].cpu(), k)


def test_refused_calls(torch):
    b, _, pages = batch_of(torch, [2], [5], 16)
    cache = dfh.KVCache(pages, 2, 64, page_size=16)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError):
        dfh.cache_write(x.clone().requires_grad_(), x, cache, b)
    for k, v in ((x[:1], x), (x[:, :1], x[:, :1]), (x[..., :32], x[..., :32]), (x[0], x[0]), (x.cpu(), x)):
        with pytest.raises(ValueError):
            dfh.cache_write(k, v, cache, b)
    for k in (x.half(), x.float()):
        with pytest.raises(TypeError):
            dfh.cache_write(k, k, cache, b)
    for n in (-1, (1 << 24) + 1):
        with pytest.raises(ValueError):
            dfh.cache_read(cache, b, n)
    t, lengths, s = b.tables, b.lengths, b.starts
    for a in ((t.long(), lengths, s), (t, lengths.long(), s), (t, lengths, s[:1]), (t[0], lengths, s), (t.cpu(), lengths, s),
              (t, lengths.cpu(), s), (t[:, :0], lengths, s), (t, lengths, torch.zeros(4, dtype=torch.int32, device="cuda")[::2])):
        with pytest.raises(ValueError):
            dfh.CacheBatch(*a)
    with pytest.raises(ValueError):
        dfh.CacheBatch(t, lengths, s, max_new=-1)
    for kw in (dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(bits=4), dict(head_dim=96),
               dict(kv_heads=0), dict(kv_heads=257), dict(pages=0), dict(device="cpu")):
        a = dict(pages=2, kv_heads=1, head_dim=64)
        a.update(kw)
        with pytest.raises(ValueError):
            dfh.KVCache(**a)
    with pytest.raises(TypeError):
        dfh.KVCache(2, 1, 64, dtype=torch.float32)
