"""One set of uint4 blocks used from several streams and threads, and its gradient
captured into a graph: every result is the one a lone call gives."""
import threading

import pytest

from lossless_entropy_coded_huffman_amd import forward as fw

pytestmark = pytest.mark.gpu
SHAPE = fw.BlockShape(hidden=256, heads=8, kv_heads=2, ffn=768)
GROUP = 64


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


@pytest.fixture(scope="module")
def blocks(torch):
    host = fw.random_blocks(3, SHAPE, 5)
    layers = [fw.quantize_block(h, SHAPE, GROUP, asymmetric=bool(i % 2)) for i, h in enumerate(host)]
    return fw.QuantizedBlocks(layers, SHAPE, torch.device("cuda:0"), GROUP)


def acts(torch, tokens, seed):
    return (torch.randn(tokens, SHAPE.hidden, generator=torch.Generator().manual_seed(seed)) * 0.5) \
        .to(torch.bfloat16).cuda()


def test_one_set_of_blocks_on_two_streams(torch, blocks):
    xs = [acts(torch, t, t) for t in (5, 130)]
    dy = [acts(torch, t, 90 + t) for t in (5, 130)]

    def step(i, grad):
        if not grad:
            return blocks.forward(xs[i])
        leaf = xs[i].clone().requires_grad_()
        return torch.autograd.grad(blocks.forward(leaf), leaf, dy[i])[0]

    want = {(i, grad): step(i, grad) for i in (0, 1) for grad in (False, True)}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for r in range(6):
        for i in (0, 1):
            with torch.cuda.stream(streams[(i + r) % 2]):
                outs.append((i, bool(r % 2), step(i, bool(r % 2))))
    torch.cuda.synchronize()
    for i, grad, out in outs:
        assert torch.equal(out, want[i, grad])


def test_one_set_of_blocks_in_two_threads(torch, blocks):
    xs = [acts(torch, t, t) for t in (3, 64)]
    want = [blocks.forward(x) for x in xs]
    torch.cuda.synchronize()
    outs, errors = [[], []], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(6):
                    outs[i].append(blocks.forward(xs[i]))
            s.synchronize()
        except Exception as e:   # seen by the test, not lost with the thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors and [len(o) for o in outs] == [6, 6]
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_blocks_gradient_captured_and_replayed(torch, blocks):
    x, dy = acts(torch, 6, 1), acts(torch, 6, 2)

    def step():
        leaf = x.detach().requires_grad_()
        return torch.autograd.grad(blocks.forward(leaf), leaf, dy)[0]

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
        x.copy_(acts(torch, 6, 30 + r))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())
        torch.cuda.synchronize()


def test_first_use_on_a_stream_other_than_the_one_that_made_them(torch, monkeypatch):
    # the scales are tensors of the device, converted behind a busy spell of the
    # stream that makes the blocks; the first call, on another stream, waits for them
    host = fw.random_blocks(1, SHAPE, 5)
    layers = [[(con, torch.from_numpy(s).cuda(), torch.from_numpy(z).cuda()) for con, s, z in
               fw.quantize_block(h, SHAPE, GROUP)] for h in host]
    x = acts(torch, 5, 1)
    want = fw.QuantizedBlocks(layers, SHAPE, torch.device("cuda:0"), GROUP).forward(x)
    upload = fw.dfh.to_device

    def late(con, device):
        out = upload(con, device)   # returns when the copy is done
        torch.cuda._sleep(5_000_000)
        return out

    monkeypatch.setattr(fw.dfh, "to_device", late)
    torch.cuda.synchronize()
    made = fw.QuantizedBlocks(layers, SHAPE, torch.device("cuda:0"), GROUP)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = made.forward(x)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
