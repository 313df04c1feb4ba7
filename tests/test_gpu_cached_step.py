"""Blocks that answer over paged caches on the GPU: the products, the cache and the attention
run together as a model runs them, each checked as in test_cached_step."""
import pytest

import lossless_entropy_coded_huffman_amd as dfh
from lossless_entropy_coded_huffman_amd import forward as fw, synth
from test_cached_step import CALLS, LENGTHS, SHAPE, Watch, inputs, ints, plan, run, starts_of

pytestmark = pytest.mark.gpu
PAGE, WIDTH = 16, 3


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def caches(blocks, bits):
    return [dfh.KVCache(20, SHAPE.kv_heads, SHAPE.head_dim, page_size=PAGE, bits=bits) for _ in range(blocks)]


def tables(torch, seqs, seed=3):
    order = torch.randperm(20, generator=torch.Generator().manual_seed(seed))[:seqs * WIDTH]
    return ints(order.reshape(seqs, WIDTH).tolist(), "cuda")


def batch(torch, done, new, table):
    return dfh.CacheBatch(table, ints(done, "cuda"), ints(starts_of(new), "cuda"), max_new=max(new))


def made(torch, how, blocks=2):
    """(QuantizedBlocks or None, float64 weights of each block as product takes them, host)."""
    host = fw.random_blocks(blocks, SHAPE, 4)
    if how == "bf16":
        return None, [{n: t.double() for n, t in fw.weight_views(fw.to_torch(h, "cpu"), SHAPE).items()} for h in host], host
    bits = int(how[1:])
    layers = [fw.quantize_block(h, SHAPE, 32 if bits == 4 else None, asymmetric=bool(i), bits=bits) for i, h in enumerate(host)]
    wide = []
    for h, block in zip(host, layers):
        w, off = {}, 0
        for (name, r, c), (_, s, z) in zip(SHAPE.matrices(), block):
            x = synth.bf16_to_f32(h[off:off + r * c]).reshape(r, c)
            off += r * c
            i = len(wide)
            if bits == 8:
                q, s, z = (torch.from_numpy(a).double() for a in synth.quantize_u8_rows(x, bool(i)))
                w[name] = q - z[:, None], s
            else:
                q, s, z = (torch.from_numpy(a) for a in synth.quantize_u4_groups(x, 32, bool(i)))
                s, z = (t.double().repeat_interleave(32, 1)[:, :c] for t in (s.bfloat16(), z))
                w[name] = s * (q.double() - z), s * (q.double() + z + 16)
        wide.append(w)
    return fw.QuantizedBlocks(layers, SHAPE, "cuda:0", 32 if bits == 4 else None, bits=bits), wide, host


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("how", ["bf16", "u4", "u8"])
def test_step(torch, monkeypatch, how, bits):
    blocks, wide, host = made(torch, how)
    watch = Watch(monkeypatch, len(LENGTHS), wide, how, bits)
    held, table = caches(2, bits), tables(torch, len(LENGTHS))
    if blocks is None:
        flat = [fw.weight_views(fw.to_torch(h, "cuda"), SHAPE) for h in host]
        products = watch.product(fw._products(torch.nn.functional.linear), CALLS)
    else:
        blocks._products = watch.product(blocks._products, CALLS)

    def step(x, done, new):
        watch.step(done, new)
        b = batch(torch, done, new, table)
        x = x.cuda()
        if blocks is not None:
            x = blocks.step(x, held, b)
        else:
            at = b.positions(len(x))
            for w, cache in zip(flat, held):
                x = fw.block_step(x, w, SHAPE, cache, b, at, products)
        assert torch.equal(x, watch.out)

    run(step, inputs(LENGTHS), plan(LENGTHS, 5))
    assert watch.worst <= 1, watch.worst


@pytest.mark.parametrize("overlap", [False, True])
def test_compressed_blocks(torch, overlap):
    # from containers bit for bit as with resident weights
    host = fw.random_blocks(3, SHAPE, 9)
    blocks = fw.CompressedBlocks([dfh.compress(dfh.KIND_BF16, h) for h in host], SHAPE, "cuda:0")
    flat = [fw.weight_views(fw.to_torch(h, "cuda"), SHAPE) for h in host]
    ours, theirs, table = caches(3, 8), caches(3, 8), tables(torch, len(LENGTHS))

    def step(x, done, new):
        b, x = batch(torch, done, new, table), x.cuda()
        y = blocks.step(x, ours, b, overlap=overlap)
        at = b.positions(len(x))
        for w, cache in zip(flat, theirs):
            x = fw.block_step(x, w, SHAPE, cache, b, at)
        assert torch.equal(x, y)

    run(step, inputs(LENGTHS), plan(LENGTHS, 4))


@pytest.mark.parametrize("how", ["u4", "u8"])
def test_captured_step(torch, how):
    # one graph for steps of up to 8 tokens: rows behind the last sequence are padding
    blocks, _, _ = made(torch, how)
    rows, seqs = 8, len(LENGTHS)
    ours, theirs = caches(2, 8), caches(2, 8)
    x = torch.zeros(rows, SHAPE.hidden, dtype=torch.bfloat16, device="cuda")
    b = dfh.CacheBatch(tables(torch, seqs), ints([0] * seqs, "cuda"), ints([0] * (seqs + 1), "cuda"), max_new=rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blocks.step(x, ours, b)                     # nothing new: nothing is written
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = blocks.step(x, ours, b)
    done = [0] * seqs
    g = torch.Generator().manual_seed(1)
    for new in ([1, 3, 0, 2], [0, 5, 0, 1], [2, 2, 2, 2], [0, 0, 0, 1], [0, 0, 0, 0], [1, 6, 1, 0]):
        done = [d + n for d, n in zip(done, new)]
        x.copy_(torch.randn(rows, SHAPE.hidden, generator=g).to(torch.bfloat16))
        b.lengths.copy_(ints(done))
        b.starts.copy_(ints(starts_of(new)))
        graph.replay()
        got = y.clone()
        want = blocks.step(x, theirs, b)
        assert torch.equal(got, want)
        for c, d in zip(ours, theirs):
            for s, t in zip(c._tensors(), d._tensors()):
                assert torch.equal(s, t)
        torch.cuda.synchronize()


def test_uint8_blocks_have_no_gradient(torch):
    blocks, wide, _ = made(torch, "u8", 1)
    x = inputs([7])[0].cuda()
    y = blocks.forward(x)
    assert y.shape == x.shape and bool(torch.isfinite(y).all())
    leaf = x.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="no gradient"):
        blocks.forward(leaf)
    b = batch(torch, [7], [7], tables(torch, 1))
    with pytest.raises(RuntimeError, match="no gradient"):
        blocks.step(leaf, caches(1, 16), b)
    with torch.no_grad():
        assert torch.equal(blocks.forward(leaf), y)
