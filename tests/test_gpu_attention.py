"""Attention over the paged cache on the GPU, against the definition in float64.

Tolerances.  e = 2^-24; u is half a step of the call's 16-bit type.  A score is a
float32 sum of D products, off by at most (D + 4) e scale sum |q k| with its scales; an
exponential by that, by the rounding of its argument (2 e |z - max|) and by 4 e of
its own, and every further tile or part multiplies by factors that are off by a few e:
with n keys (n + 8) e covers these and the sums.  Together r[j], relative.  Weights (times the
values' scales, with 8 bits) are rounded to the type (u, and half of float16's smallest
subnormal), and so is the output.  So with w the exact weights
    |out - ref| <= sum w |v| (r + u) + |ref| sum w r + u |ref| + subnormals,
where the magnitudes come from the float64 computation; half as much again covers
products of these terms.  The pool is full of NaN but for the live positions of the
batch, so nothing that a row does not see may touch it.
"""
import math
import random

import pytest

import lossless_entropy_coded_huffman_amd as dfh
from test_gpu_cache import batch_of, types

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def spoiled(torch, cache):
    """All of the pool NaN (8 bits: its scales)."""
    if cache.bits == 8:
        cache.k.fill_(100)
        cache.v.fill_(100)
        cache.k_scales.fill_(math.nan)
        cache.v_scales.fill_(math.nan)
    else:
        cache.k.fill_(math.nan)
        cache.v.fill_(math.nan)
    return cache


def filled(torch, cache, tables, lengths, seed=0, size=1.0):
    """Random live positions; the whole keys and values of each sequence in float64."""
    g = torch.Generator().manual_seed(seed)
    page, out = cache.page_size, []
    for table, n in zip(tables, lengths):
        kv = []
        for name in ("k", "v"):
            x = torch.randn(n, cache.kv_heads, cache.head_dim, generator=g) * size
            p = torch.tensor([table[i // page] for i in range(n)], dtype=torch.long, device="cuda")
            r = torch.arange(n, device="cuda") % page
            if cache.bits == 8:
                codes = (x * 40).round().clamp(-127, 127).to(torch.int8)
                scales = (torch.rand(n, cache.kv_heads, generator=g) + 0.5) * size / 40
                getattr(cache, name)[p, :, r] = codes.cuda()
                getattr(cache, name + "_scales")[p, :, r] = scales.cuda()
                kv.append((codes.double() * scales.double()[..., None]).cuda())
            else:
                x = x.to(cache.dtype)
                getattr(cache, name)[p, :, r] = x.cuda()
                kv.append(x.double().cuda())
        out.append(kv)
    return out


def check(torch, got, lse, q, kvs, new, lengths, scale, window, bits, rows=None):
    """Every new token's output and log-sum (rows: of these tokens alone)."""
    t, dt = 0, q.dtype
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -134
    heads = q.shape[1]
    got, lse = got.double(), lse.double()
    for (k, v), n, length in zip(kvs, new, lengths):
        rep = heads // k.shape[1] if k.numel() else 1
        pos = torch.arange(length - n, length, device="cuda")
        keep = pos >= 0
        assert not got[t: t + n][~keep].any() and bool((lse[t: t + n][~keep] == -math.inf).all())
        for h in range(heads):
            if length == 0:
                break
            ts = torch.arange(t, t + n, device="cuda")[keep]
            ps = pos[keep]
            if rows is not None:
                sel = torch.isin(ts, rows)
                ts, ps = ts[sel], ps[sel]
            if not ts.numel():
                continue
            kk, vv, qq = k[:, h // rep], v[:, h // rep], q[ts, h].double()
            j = torch.arange(length, device="cuda")
            seen = (j[None] <= ps[:, None]) & (ps[:, None] - j[None] < (window or 1 << 40))
            z = ((qq @ kk.t()) * scale).masked_fill(~seen, -math.inf)
            m = z.amax(1, keepdim=True)
            p = (z - m).exp()
            total = p.sum(1, keepdim=True)
            w = p / total
            ref = w @ vv
            a = (qq.abs() @ kk.abs().t()) * scale
            r = (k.shape[2] + 4) * E * a + (2 * (m - z).masked_fill(~seen, 0.0) + length + 12) * E
            spread = (w * r).sum(1, keepdim=True)
            small = tiny / total * (seen.double() @ vv.abs()) if dt == torch.float16 else 0.0
            bound = 1.5 * ((w * (r + u)) @ vv.abs() + ref.abs() * spread + u * ref.abs() + small) + tiny
            err = (got[ts, h] - ref).abs()
            assert bool((err <= bound).all()), "head %d: %g of the bound" % (h, float((err / bound).max()))
            full = (m + total.log())[:, 0]
            lb = 1.5 * ((w * r).sum(1) + (length + 8) * E + 4 * E * full.abs())
            assert bool(((lse[ts, h] - full).abs() <= lb).all())
        t += n


CASES = [
    # kv, group, dim, page, new, lengths, window, hint
    (1, 1, 32, 16, [1], [1], None, 1),
    (2, 4, 128, 64, [1], [2000], None, 1),
    (8, 4, 128, 64, [1] * 7, [1, 31, 32, 33, 64, 500, 4097], None, 1),
    (2, 7, 64, 16, [1, 0, 1, 1], [17, 90, 0, 1000], None, 1),
    (1, 32, 128, 32, [1, 1], [700, 95], None, 1),
    (3, 3, 64, 128, [4, 1, 9, 10], [4, 300, 9, 1000], None, None),
    (2, 4, 128, 16, [8, 8], [500, 8], None, 8),
    (2, 2, 256, 64, [1, 16, 3], [129, 16, 333], None, None),
    (2, 2, 256, 16, [65, 130], [129, 130], None, None),
    (1, 1, 128, 64, [300], [300], None, None),
    (2, 4, 128, 64, [33, 1, 200], [97, 700, 200], None, None),
    (2, 8, 64, 16, [100, 0, 1, 257, 4], [100, 50, 3, 513, 4], None, None),
    (1, 40, 64, 32, [1, 5], [77, 70], None, None),
    (1, 256, 32, 16, [1, 2], [40, 33], None, None),
    (2, 3, 32, 256, [1, 90, 3], [1000, 90, 3], None, None),
    (2, 4, 128, 64, [1, 1, 1], [10, 200, 3000], 100, 1),
    (2, 4, 64, 16, [7, 150, 1], [500, 333, 64], 33, None),
    (1, 4, 128, 32, [200], [900], 1, None),
    (1, 2, 256, 128, [100, 1], [700, 300], 64, None),
    (2, 1, 128, 64, [5, 3, 2], [2, 0, 7], None, None),                 # tokens before position 0
    (1, 1, 64, 16, [200, 50], [150, 0], 20, None),
    (1, 4, 128, 64, [1, 1], [9000, 5], None, 1),                       # split over many workgroups
    (1, 4, 64, 64, [64], [6000], None, None),                           # a short chunk of a long prompt
    (2, 4, 128, 64, [60, 1, 20], [700, 700, 20], None, 1),             # a wrong hint
    (2, 4, 64, 32, [60, 9, 20], [700, 700, 20], None, 9),
    (4, 2, 64, 16, [2] * 70, [2 + 13 * i for i in range(70)], None, 2),
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(torch, case, dtype, bits):
    kv, group, dim, page, new, lengths, window, hint = CASES[case]
    dt = types(torch)[dtype]
    b, tables, pages = batch_of(torch, new, lengths, page, seed=case, max_new=hint)
    cache = spoiled(torch, dfh.KVCache(pages, kv, dim, page_size=page, dtype=dt, bits=bits))
    kvs = filled(torch, cache, tables, lengths, seed=case)
    q = torch.randn(sum(new), kv * group, dim, generator=torch.Generator().manual_seed(99)).to(dt).cuda()
    got, lse = dfh.cached_attention(q, cache, b, window=window, return_lse=True)
    check(torch, got, lse, q, kvs, new, lengths, dim ** -0.5, window, bits)
    assert torch.equal(dfh.cached_attention(q, cache, b, window=window), got)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("scale,size", [(1.0, 1.0), (0.01, 3.0), (0.7, 12.0)])
def test_scores_of_any_size(torch, scale, size, bits):
    # nearly even weights, and ones where a single key has all
    new, lengths = [1, 70, 3], [800, 300, 40]
    for dt in (torch.bfloat16, torch.float16):
        b, tables, pages = batch_of(torch, new, lengths, 32)
        cache = spoiled(torch, dfh.KVCache(pages, 2, 64, page_size=32, dtype=dt, bits=bits))
        kvs = filled(torch, cache, tables, lengths, size=size)
        q = (torch.randn(sum(new), 6, 64, generator=torch.Generator().manual_seed(1)) * size).to(dt).cuda()
        got, lse = dfh.cached_attention(q, cache, b, scale=scale, return_lse=True)
        check(torch, got, lse, q, kvs, new, lengths, scale, None, bits)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new,lengths", [([1, 2], [300, 77]), ([90, 60], [300, 60])])
def test_scales_that_differ_widely(torch, new, lengths, dtype):
    # 8 bits: tokens' scales from the smallest to the largest that the type has values for,
    # growing, falling and mixed along the sequence
    dt = types(torch)[dtype]
    lo, hi = (-14, 15) if dtype == "fp16" else (-60, 60)
    for order in ("up", "down", "mixed"):
        b, tables, pages = batch_of(torch, new, lengths, 16)
        cache = spoiled(torch, dfh.KVCache(pages, 1, 64, page_size=16, dtype=dt, bits=8))
        kvs = filled(torch, cache, tables, lengths)
        for i, (table, n) in enumerate(zip(tables, lengths)):
            e = torch.linspace(lo, hi, n).round()
            e = e.flip(0) if order == "down" else e[torch.randperm(n, generator=torch.Generator().manual_seed(i))] if order == "mixed" else e
            f = (2.0 ** e.double()) / 127
            p = torch.tensor([table[j // 16] for j in range(n)], device="cuda")
            r = torch.arange(n, device="cuda") % 16
            cache.v_scales[p, 0, r] = f.float().cuda()
            kvs[i][1] = cache.v[p, 0, r].double()[:, None] * f.float().double().cuda()[:, None, None]
        q = torch.randn(sum(new), 3, 64, generator=torch.Generator().manual_seed(1)).to(dt).cuda()
        got, lse = dfh.cached_attention(q, cache, b, return_lse=True)
        check(torch, got, lse, q, kvs, new, lengths, 0.125, None, 8)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [[3], [100]])
def test_queries_of_any_size(torch, new, dtype):
    # 8 bits: rows of q from the type's smallest to its largest, and elements of one row far apart
    dt, length = types(torch)[dtype], 200
    b, tables, pages = batch_of(torch, new, [length], 16)
    cache = spoiled(torch, dfh.KVCache(pages, 1, 128, page_size=16, dtype=dt, bits=8))
    kvs = filled(torch, cache, tables, [length])
    n = new[0]
    g = torch.Generator().manual_seed(2)
    for size in ((-24.0, -10.0, 0.0, 10.0) if dtype == "fp16" else (-130.0, -60.0, 0.0, 60.0, 110.0)):
        q = torch.randn(n, 2, 128, generator=g).double() * 2.0 ** size
        q = q.clamp(-torch.finfo(dt).max, torch.finfo(dt).max).to(dt).cuda()
        # scores of ordinary size, as far as the scale's type reaches
        scale = min(max(2.0 ** -size / 12, 2.0 ** -120), 2.0 ** 120)
        got, lse = dfh.cached_attention(q, cache, b, scale=scale, return_lse=True)
        check(torch, got, lse, q, kvs, new, [length], scale, None, 8)
    q = (torch.randn(n, 2, 128, generator=g) * 2.0 ** torch.randint(-12, 1, (n, 2, 128), generator=g)).to(dt).cuda()
    got, lse = dfh.cached_attention(q, cache, b, return_lse=True)
    check(torch, got, lse, q, kvs, new, [length], 128 ** -0.5, None, 8)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("new", [[2], [150], [9]])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_not_seen_does_not_touch(torch, new, bad, bits):
    # each position's key and value is spoiled in turn: rows before it, and those whose
    # window it has left, keep their bits; rows that see it become what the definition says
    kv, group, dim, page, window = 1, 3, 64, 16, 40
    n, length = new[0], 160
    for dt in (torch.bfloat16, torch.float16):
        b, tables, pages = batch_of(torch, new, [length], page)
        cache = spoiled(torch, dfh.KVCache(pages, kv, dim, page_size=page, dtype=dt, bits=bits))
        filled(torch, cache, tables, [length])
        q = torch.randn(n, kv * group, dim, generator=torch.Generator().manual_seed(1)).to(dt).cuda()
        clean = {w: dfh.cached_attention(q, cache, b, window=w) for w in (None, window)}
        for at in (length - n - 1 if n < length else 0, length - n, length - n // 2, length - 1, 100):
            for names in (("k",), ("v",), ("k", "v")):
                saved = [t.clone() for t in cache._tensors() if t is not None]
                for name in names:
                    if bits == 8:
                        getattr(cache, name + "_scales")[tables[0][at // page], 0, at % page] = bad
                    else:
                        getattr(cache, name)[tables[0][at // page], 0, at % page, 5] = bad
                for w in (None, window):
                    got = dfh.cached_attention(q, cache, b, window=w)
                    pos = torch.arange(length - n, length, device="cuda")
                    sees = (pos >= at) & (pos - at < (w or 1 << 30))
                    # another tile of the same keys may sum in another order, not here
                    assert torch.equal(got[~sees], clean[w][~sees])
                    if "v" in names:
                        assert not got[sees][..., 5].isfinite().any()
                for t, old in zip([t for t in cache._tensors() if t is not None], saved):
                    t.copy_(old)


def test_a_row_of_q_that_is_not_finite(torch):
    for new, lengths in (([1, 1], [50, 60]), ([100], [300])):
        b, tables, pages = batch_of(torch, new, lengths, 16)
        cache = spoiled(torch, dfh.KVCache(pages, 1, 64, page_size=16))
        filled(torch, cache, tables, lengths)
        q = torch.randn(sum(new), 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
        clean = dfh.cached_attention(q, cache, b)
        for bad in (math.nan, math.inf):
            q2 = q.clone()
            q2[0, 1, 7] = bad
            got = dfh.cached_attention(q2, cache, b)
            assert bool(got[0, 1].isnan().all())
            got[0, 1] = clean[0, 1]
            assert torch.equal(got, clean)


@pytest.mark.parametrize("bits", [16, 8])
def test_positions_and_rows_that_are_not_there(torch, bits):
    # pages outside the pool, positions outside the table, rows of no sequence
    page, kv, group, dim = 16, 2, 4, 64
    tables = torch.tensor([[0, 1, 2], [3, -1, 4], [5, 6, 1 << 30], [7, 8, 9]], dtype=torch.int32)
    lengths, starts = [40, 48, 48, 70], [3, 4, 24, 25, 60]
    cache = spoiled(torch, dfh.KVCache(11, kv, dim, page_size=page, bits=bits))
    lists = [[0, 1, 2], [3, 10, 4], [5, 6], [7, 8, 9]]        # page 10: in no table
    kvs = filled(torch, cache, lists, [40, 48, 32, 48])
    n = 66
    q = torch.randn(n, kv * group, dim, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    ref_of = {}
    for s, gone in ((1, list(range(16, 32))), (2, list(range(32, 48))), (3, list(range(48, 70))), (0, [])):
        k, v = kvs[s]
        there = [i for i in range(lengths[s]) if i not in gone]
        ref_of[s] = (k, v, there)
    for hint in (1, None):
        b = dfh.CacheBatch(tables.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                           torch.tensor(starts, dtype=torch.int32).cuda(), max_new=hint)
        got, lse = dfh.cached_attention(q, cache, b, return_lse=True)
        none = [0, 1, 2] + list(range(60, n))
        assert not got[none].any() and bool((lse[none] == -math.inf).all())
        for s in range(4):
            k, v, there = ref_of[s]
            for t in range(starts[s], starts[s + 1]):
                p = lengths[s] - starts[s + 1] + t
                j = [i for i in there if i <= p]
                for h in (0, 3, 7):
                    z = (k[j][:, h // group] @ q[t, h].double()) * dim ** -0.5
                    w = z.softmax(0)
                    vv = v[j][:, h // group]
                    ref = w @ vv
                    # every weight and the output are rounded; the rest is far smaller
                    assert bool(((got[t, h].double() - ref).abs() <= (2.0 ** -8 + 1e-4) * (w @ vv.abs()) + 2.0 ** -8 * ref.abs()).all())


@pytest.mark.parametrize("new", [[1, 1], [90, 3]])
def test_layouts_streams_and_shared_pages(torch, new):
    kv, group, dim, page, lengths = 2, 4, 128, 32, [200, 150]
    b, tables, pages = batch_of(torch, new, lengths, page)
    cache = spoiled(torch, dfh.KVCache(pages, kv, dim, page_size=page))
    filled(torch, cache, tables, lengths)
    n = sum(new)
    q = torch.randn(n, kv * group, dim, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    want = dfh.cached_attention(q, cache, b)
    wide = torch.zeros(n, 2 * kv * group, dim + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, ::2, :dim] = q
    for f in (wide[:, ::2, :dim], q.transpose(0, 1).contiguous().transpose(0, 1), q.transpose(1, 2).contiguous().transpose(1, 2),
              torch.cat([q.new_zeros(n, kv * group, 1), q], 2)[..., 1:]):
        assert torch.equal(dfh.cached_attention(f, cache, b), want)
    one = q[:1, :1].expand(n, kv * group, dim)              # one vector for all
    assert torch.equal(dfh.cached_attention(one, cache, b), dfh.cached_attention(one.contiguous(), cache, b))
    # a sequence that reads another's first pages
    t2 = b.tables.clone()
    t2[1, :4] = t2[0, :4]
    b2 = dfh.CacheBatch(t2, b.lengths, b.starts)
    own = dfh.KVCache(pages, kv, dim, page_size=page)
    for name in ("k", "v"):
        getattr(own, name).copy_(getattr(cache, name))
        for i in range(4):
            getattr(own, name)[tables[1][i]] = getattr(cache, name)[tables[0][i]]
    assert torch.equal(dfh.cached_attention(q, cache, b2), dfh.cached_attention(q, own, b))
    # another stream, late input
    s = torch.cuda.Stream()
    late = torch.zeros(n, dim, kv * group, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    with torch.cuda.stream(s):
        late.copy_(q)
    got, lse = dfh.cached_attention(late, cache, b, return_lse=True, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    empty = dfh.cached_attention(q[:0], cache, dfh.CacheBatch(b.tables, b.lengths, torch.zeros_like(b.starts)))
    assert empty.shape == (0, kv * group, dim)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    b0 = dfh.CacheBatch(none.view(0, 1), none, torch.zeros(1, dtype=torch.int32, device="cuda"))
    got, lse = dfh.cached_attention(q, cache, b0, return_lse=True)
    assert not got.any() and bool((lse == -math.inf).all())


def test_decoding_from_one_graph(torch):
    # a captured step (write, attend) is replayed as the sequences grow; a second graph has a
    # workspace of its own and runs between
    kv, group, dim, page = 2, 4, 128, 16
    steps, start = 40, [1, 30]
    tables = torch.tensor([[3, 1, 8, 9, 11], [0, 2, 5, 7, 10]], dtype=torch.int32).cuda()
    lengths = torch.tensor(start, dtype=torch.int32).cuda()
    b = dfh.CacheBatch(tables, lengths, torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), max_new=1)
    g = torch.Generator().manual_seed(0)
    kvq = [torch.randn(steps, 2, h, dim, generator=g).to(torch.bfloat16).cuda() for h in (kv, kv, kv * group)]
    for bits in (8, 16):
        cache, eager = (dfh.KVCache(12, kv, dim, page_size=page, bits=bits) for _ in range(2))
        k, v, q = (t[0].clone() for t in kvq)
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                dfh.cache_write(k, v, cache, b)
                out = dfh.cached_attention(q, cache, b)
            graphs.append((graph, out))
        for i in range(steps):
            lengths.copy_(torch.tensor([start[0] + i, start[1] + i], dtype=torch.int32))
            for t, src in zip((k, v, q), kvq):
                t.copy_(src[i])
            for graph, _ in graphs:
                graph.replay()
            dfh.cache_write(kvq[0][i], kvq[1][i], eager, b)
            want = dfh.cached_attention(kvq[2][i], eager, b)
            torch.cuda.synchronize()
            assert all(torch.equal(out, want) for _, out in graphs)


@pytest.mark.parametrize("bits", [16, 8])
def test_a_prompt_in_chunks_is_the_prompt_at_once(torch, bits):
    # the same keys are seen in the same tiles: each token's sums are those of the whole
    # prompt, up to their order
    kv, group, dim, page, n = 2, 2, 64, 32, 450
    g = torch.Generator().manual_seed(5)
    k, v, q = (torch.randn(n, h, dim, generator=g).to(torch.float16).cuda() for h in (kv, kv, kv * group))
    b, tables, pages = batch_of(torch, [n], [n], page)
    cache = dfh.KVCache(pages, kv, dim, page_size=page, dtype=torch.float16, bits=bits)
    dfh.cache_write(k, v, cache, b)
    whole = dfh.cached_attention(q, cache, b)
    parts, at = [], 0
    again = dfh.KVCache(pages, kv, dim, page_size=page, dtype=torch.float16, bits=bits)
    for c in (1, 100, 7, 200, 64, 78):
        p = dfh.CacheBatch(b.tables, torch.tensor([at + c], dtype=torch.int32).cuda(), torch.tensor([0, c], dtype=torch.int32).cuda())
        dfh.cache_write(k[at: at + c], v[at: at + c], again, p)
        parts.append(dfh.cached_attention(q[at: at + c], again, p))
        at += c
    assert at == n and torch.equal(again.k, cache.k)
    rk, rv = (t.double() for t in dfh.cache_read(cache, b, n))
    kvs = [(rk, rv)]
    if bits == 16:
        for out in (whole, torch.cat(parts)):
            lse = dfh.cached_attention(q, cache, b, return_lse=True)[1]
            check(torch, out, lse, q, kvs, [n], [n], dim ** -0.5, None, bits)
    # two sides, each off by at most its weights' and output's roundings (values are at most 5)
    assert float((torch.cat(parts).double() - whole.double()).abs().max()) <= 2 * 5 * 4 * 2.0 ** -11


def test_a_pool_beyond_32_bits(torch):
    kv, dim, page, group = 8, 128, 256, 4
    pages = 9000                                       # 2.4e9 elements, 4.7e9 bytes
    cache = dfh.KVCache(pages, kv, dim, page_size=page, bits=16)
    lists = [[pages - 1, 8999 - 1, 4097], [8192, 5, 8195]]
    lengths = [600, 520]
    kvs = filled(torch, cache, lists, lengths)
    for new in ([1, 1], [70, 2]):
        t = torch.tensor(lists, dtype=torch.int32).cuda()
        starts = torch.tensor([0, new[0], sum(new)], dtype=torch.int32).cuda()
        b = dfh.CacheBatch(t, torch.tensor(lengths, dtype=torch.int32).cuda(), starts)
        q = torch.randn(sum(new), kv * group, dim, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
        got, lse = dfh.cached_attention(q, cache, b, return_lse=True)
        check(torch, got, lse, q, kvs, new, lengths, dim ** -0.5, None, 16)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("some", [1, 60])
def test_many_sequences(torch, some, bits):
    # more than are split, with padding before and behind, beside a prompt
    page, kv, group, dim, seqs = 16, 2, 4, 64, 700
    new = [i % 3 if i != 400 else some for i in range(seqs)]
    lengths = [n + 7 * i % 50 for i, n in enumerate(new)]
    b, tables, pages = batch_of(torch, new, lengths, page, seed=5)
    cache = spoiled(torch, dfh.KVCache(pages, kv, dim, page_size=page, bits=bits))
    kvs = filled(torch, cache, tables, lengths, seed=5)
    before, behind, n = 5, 9, sum(new)
    q = torch.randn(before + n + behind, kv * group, dim, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    for hint in (2, None):
        moved = dfh.CacheBatch(b.tables, b.lengths, b.starts + before, max_new=hint)
        got, lse = dfh.cached_attention(q, cache, moved, return_lse=True)
        pad = list(range(before)) + list(range(before + n, len(q)))
        assert not got[pad].any() and bool((lse[pad] == -math.inf).all())
        mid = slice(before, before + n)
        check(torch, got[mid], lse[mid], q[mid], kvs, new, lengths, dim ** -0.5, None, bits)


@pytest.mark.parametrize("hint", [1, None])
def test_starts_that_are_out_of_order(torch, hint):
    # nothing is said of what such a batch gives; it reads and writes within its tensors,
    # and the next call is right
    page, new, lengths = 16, [3, 150, 70, 40], [30, 160, 70, 90]
    b, tables, pages = batch_of(torch, new, lengths, page)
    cache = spoiled(torch, dfh.KVCache(pages, 1, 64, page_size=page))
    kvs = filled(torch, cache, tables, lengths)
    q = torch.randn(sum(new), 2, 64, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    top = (1 << 31) - 1
    for starts in ([200, 100, 150, 20, 263], [263, 0, 263, 0, 100], [-5, 400, -top, top, 5], [top, -top, top, 0, 0]):
        odd = dfh.CacheBatch(b.tables, b.lengths, torch.tensor(starts, dtype=torch.int32).cuda(), max_new=hint)
        dfh.cached_attention(q, cache, odd, return_lse=True)
        dfh.cache_read(cache, odd, len(q))
        torch.cuda.synchronize()
    got, lse = dfh.cached_attention(q, cache, b, return_lse=True)
    check(torch, got, lse, q, kvs, new, lengths, 64 ** -0.5, None, 16)


def test_a_long_sequence(torch):
    # 150000 positions: a few rows, and a chunk, sampled
    kv, group, dim, page, length = 1, 4, 64, 256, 150001
    for new, rows in (([1], [0]), ([40], [0, 13, 39]), ([400], [0, 200, 399])):
        b, tables, pages = batch_of(torch, new, [length], page)
        cache = spoiled(torch, dfh.KVCache(pages, kv, dim, page_size=page, bits=8))
        kvs = filled(torch, cache, tables, [length])
        q = torch.randn(new[0], kv * group, dim, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
        got, lse = dfh.cached_attention(q, cache, b, return_lse=True)
        check(torch, got, lse, q, kvs, new, [length], dim ** -0.5, None, 8, rows=torch.tensor(rows, device="cuda"))


def test_refused_calls(torch):
    b, _, pages = batch_of(torch, [2], [5], 16)
    cache = dfh.KVCache(pages, 2, 64, page_size=16)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError):
        dfh.cached_attention(q.clone().requires_grad_(), cache, b)
    for a in (q[:, :3], q[..., :32], q[0], q.cpu(), q[:, :0]):
        with pytest.raises(ValueError):
            dfh.cached_attention(a, cache, b)
    for a in (q.half(), q.float()):
        with pytest.raises(TypeError):
            dfh.cached_attention(a, cache, b)
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(window=0), dict(window=-3)):
        with pytest.raises(ValueError):
            dfh.cached_attention(q, cache, b, **kw)
