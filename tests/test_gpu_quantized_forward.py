"""The quantised model end to end: uint4 containers decoded and multiplied block
by block, a compressed LM head, cross entropy and distillation against the
lossless model, and gradients back through all of it."""
import numpy as np
import pytest

import lossless_entropy_coded_huffman_amd as dfh
from lossless_entropy_coded_huffman_amd import forward as fw
from lossless_entropy_coded_huffman_amd import synth

pytestmark = pytest.mark.gpu
SHAPE = fw.BlockShape(hidden=256, heads=8, kv_heads=2, ffn=768)
VOCAB, GROUP = 3001, 64


@pytest.fixture(scope="module")
def model():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda:0")
    host = fw.random_blocks(3, SHAPE, 5)
    layers = [fw.quantize_block(h, SHAPE, GROUP, asymmetric=bool(i % 2)) for i, h in enumerate(host)]
    head = synth.bf16_rne(np.random.default_rng(1).normal(0, 0.15, VOCAB * SHAPE.hidden).astype(np.float32))
    return dict(torch=torch, dev=dev, host=host, layers=layers, head=head,
                quant=fw.QuantizedBlocks(layers, SHAPE, dev, GROUP),
                lossless=fw.CompressedBlocks([dfh.compress(0, h) for h in host], SHAPE, dev),
                chead=fw.CompressedHead(dfh.compress(0, head), VOCAB, SHAPE.hidden, dev))


def resident(model):
    """The quantised blocks with every layer's nibbles resident (never coded)."""
    torch, dev = model["torch"], model["dev"]
    out = []
    for block in model["layers"]:
        ws = {}
        for (name, r, c), (con, s, z) in zip(SHAPE.matrices(), block):
            buf = dfh.to_device(con, dev).empty_output()
            dfh.df_decompress(dfh.to_device(con, dev), buf)
            ws[name] = dfh.U4Matrix(buf.clone(), torch.from_numpy(s).to(dev, torch.bfloat16), torch.from_numpy(z).to(dev),
                                    cols=c, group_size=GROUP)
        out.append(ws)
    torch.cuda.synchronize()
    return out


def run_resident(x, weights):
    for ws in weights:
        x = fw.block_forward(x, ws, SHAPE, dfh.linear_u4)
    return x


def acts(model, tokens, seed=0):
    torch = model["torch"]
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(tokens, SHAPE.hidden, generator=g) * 0.5).to(torch.bfloat16).to(model["dev"])


@pytest.mark.parametrize("tokens", [1, 7, 130])
def test_decoded_blocks_equal_resident_ones(model, tokens):
    torch = model["torch"]
    x = acts(model, tokens)
    ref = run_resident(x, resident(model))
    assert torch.isfinite(ref.float()).all()
    for _ in range(2):
        assert torch.equal(model["quant"].forward(x).view(torch.int16), ref.view(torch.int16))


def test_codes_are_the_weights_they_came_from(model):
    # the plain product with the dequantised weights, one layer of each kind
    torch, dev = model["torch"], model["dev"]
    x = acts(model, 9)
    for block in range(2):
        r, c = SHAPE.matrices()[0][1:]
        codes, s, z = synth.quantize_u4_groups(synth.bf16_to_f32(model["host"][block][: r * c]).reshape(r, c), GROUP,
                                               bool(block % 2))
        s = torch.from_numpy(s).to(torch.bfloat16).double().repeat_interleave(GROUP, 1)
        w = s * (torch.from_numpy(codes).double() - torch.from_numpy(z).double().repeat_interleave(GROUP, 1))
        # quantisation moves a weight by half a step at most (and the scale's rounding)
        orig = torch.from_numpy(synth.bf16_to_f32(model["host"][block][: r * c]).reshape(r, c)).double()
        step = s * (1 + 2.0 ** -7)
        assert bool(((w - orig).abs() <= 0.5 * step + 15 * 2.0 ** -8 * s + step * (block % 2)).all())
        dcs = model["quant"].blocks[block]
        dfh.df_decompress_batch(dcs, model["quant"].scratch)
        y = dfh.linear_u4(x, model["quant"].weights[block]["q"]).double().cpu()
        ref = x.double().cpu() @ w.t()
        mag = x.double().cpu().abs() @ (s * 286).t()
        bound = (128 + c / 128 + 16) * 2.0 ** -24 * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs() + 1e-40
        assert bool(((y - ref).abs() <= bound).all())


def test_gradients_through_decoded_blocks(model):
    torch = model["torch"]
    weights = resident(model)
    for tokens in (3, 65):
        x = acts(model, tokens, seed=tokens)
        dy = acts(model, tokens, seed=99)
        a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
        ga, = torch.autograd.grad(model["quant"].forward(a), a, dy)
        gb, = torch.autograd.grad(run_resident(b, weights), b, dy)
        assert torch.isfinite(ga.float()).all() and float(ga.float().abs().max()) > 0
        assert torch.equal(ga, gb)


def test_scoring_and_distillation_together(model):
    torch, dev = model["torch"], model["dev"]
    x = acts(model, 40, seed=3)
    labels = torch.randint(0, VOCAB, (40,), generator=torch.Generator().manual_seed(2)).to(dev)
    labels[:5] = -100
    head = torch.from_numpy(model["head"].view(np.int16)).to(dev).view(torch.bfloat16).view(VOCAB, SHAPE.hidden)
    # the lossless teacher: its top logits from the plain product
    with torch.no_grad():
        t = model["lossless"].forward(x)
        top, index = (t.float() @ head.float().t()).topk(16, dim=1)
    leaf = x.clone().requires_grad_()
    h = model["quant"].forward(leaf)
    ce = model["chead"].loss(h, labels)
    kl = model["chead"].distill(h, top, index, temperature=2.0)
    g, = torch.autograd.grad(ce + kl, leaf)
    assert torch.isfinite(g.float()).all() and float(g.float().abs().max()) > 0
    # the same with everything resident
    leaf2 = x.clone().requires_grad_()
    h2 = run_resident(leaf2, resident(model))
    ce2 = dfh.vocab_loss(h2, head, labels)
    kl2 = dfh.distill_loss(h2, head, top, index, temperature=2.0)
    g2, = torch.autograd.grad(ce2 + kl2, leaf2)
    assert torch.equal(h, h2) and torch.equal(ce, ce2) and torch.equal(kl, kl2) and torch.equal(g, g2)
    # and in float64 from the hidden states
    z = h.detach().double().cpu() @ head.double().cpu().t()
    lab = labels.cpu()
    ref = torch.nn.functional.cross_entropy(z, lab, ignore_index=-100)
    err = (SHAPE.hidden + 16) * 2.0 ** -24 * (h.detach().double().cpu().abs() @ head.double().cpu().abs().t()).amax()
    assert abs(float(ce.detach()) - float(ref)) <= 2 * float(err) + 64 * 2.0 ** -24 * (float(ref) + 8)
    tq = torch.softmax(top.double().cpu() / 2, 1)
    ref = 4 * (tq * (tq.log() - torch.log_softmax(z / 2, 1).gather(1, index.cpu()))).sum(1).mean()
    assert abs(float(kl.detach()) - float(ref)) <= 4 * (2 * float(err) + 64 * 2.0 ** -24 * (float(ref) + 16))


def test_captured_and_replayed(model):
    torch, dev = model["torch"], model["dev"]
    x = acts(model, 6, seed=8)
    labels = torch.arange(6, device=dev)

    def step():
        with torch.no_grad():
            return model["chead"].loss(model["quant"].forward(x), labels, reduction="none")

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
        x.copy_(acts(model, 6, seed=20 + r))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())
        torch.cuda.synchronize()


def test_refusals(model):
    dev, layers = model["dev"], model["layers"]
    with pytest.raises(ValueError):
        fw.QuantizedBlocks([layers[0][:3]], SHAPE, dev, GROUP)
    with pytest.raises(ValueError):
        fw.QuantizedBlocks([[layers[0][1], *layers[0][1:]]], SHAPE, dev, GROUP)
    with pytest.raises(ValueError):
        fw.QuantizedBlocks(layers, SHAPE, dev, 32)
    with pytest.raises(ValueError):
        fw.CompressedHead(dfh.compress(0, model["head"]), VOCAB + 1, SHAPE.hidden, dev)
