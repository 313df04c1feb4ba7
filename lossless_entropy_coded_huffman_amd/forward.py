"""Transformer-block decompression overlapped with the forward pass.

The DF11 digest ("Descompressão por bloco de transformer") decompresses all
weight matrices of one transformer block together, just before the block
runs, and notes that the cost is amortised over the batch.  This module runs
a Llama-shaped forward pass whose block weights live only as compressed
containers in HBM: while block i computes on the caller's stream, block i+1
is decoded on a side stream into the other of two scratch buffers; events
order the reuse of each scratch buffer (decode waits for the compute that
last read it, compute waits for its decode).

The block itself is plain PyTorch in BF16 (RMSNorm, grouped-query attention
with rotary embeddings, SwiGLU MLP), weights random, norms at one.  Every
batched product takes contiguous operands.

The EntroLLM summary ("Metodologia") stores quantised weights instead.
``QuantizedBlocks`` runs the same blocks from uint4 containers: a block's seven
layers are decoded in one batch to packed nibbles and multiplied as they are
(``linear_u4``; a long prompt and a gradient expand one layer at a time in a call's
workspace), so no dequantised copy is kept; gradients to the activations
decode a block again.  ``CompressedHead`` holds an LM head as one BF16 container
and scores hidden states against it (``vocab_loss``, ``distill_loss``): what the
quantised model loses against the lossless one, and the gradient to mend it.
"""
from __future__ import annotations

import contextlib
import threading
from dataclasses import dataclass

import numpy as np
import torch

from . import dfh
from .ops import U4Matrix, distill_loss, linear_u4, vocab_loss


@dataclass(frozen=True)
class BlockShape:
    hidden: int = 4096
    heads: int = 32
    kv_heads: int = 8
    ffn: int = 14336
    rope_theta: float = 500000.0

    @property
    def head_dim(self) -> int:
        return self.hidden // self.heads

    def matrices(self):
        """(name, rows, cols) in the order the block's container concatenates them."""
        d, kv = self.hidden, self.kv_heads * self.head_dim
        return (("q", d, d), ("k", kv, d), ("v", kv, d), ("o", d, d),
                ("gate", self.ffn, d), ("up", self.ffn, d), ("down", d, self.ffn))

    def elements(self) -> int:
        return sum(r * c for _, r, c in self.matrices())


LLAMA3_8B = BlockShape()


def weight_views(flat: torch.Tensor, shape: BlockShape) -> dict:
    """Row-major matrix views into one block's flat BF16 weight buffer."""
    out, off = {}, 0
    for name, r, c in shape.matrices():
        out[name] = flat[off: off + r * c].view(r, c)
        off += r * c
    return out


def _rms_norm(x: torch.Tensor, eps: float = 1e-5) -> torch.Tensor:
    xf = x.float()
    return (xf * torch.rsqrt(xf.pow(2).mean(-1, keepdim=True) + eps)).to(x.dtype)


def _rope(x: torch.Tensor, theta: float) -> torch.Tensor:
    # x: [heads, T, head_dim]; rotate pairs (i, i + head_dim / 2) in float32
    _, t, hd = x.shape
    half = hd // 2
    inv = 1.0 / (theta ** (torch.arange(0, half, device=x.device, dtype=torch.float32) / half))
    ang = torch.arange(t, device=x.device, dtype=torch.float32)[:, None] * inv[None, :]
    cos, sin = ang.cos(), ang.sin()
    xf = x.float()
    a, b = xf[..., :half], xf[..., half:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1).to(x.dtype)


class _Bmm(torch.autograd.Function):
    """torch.bmm of contiguous operands whose derivatives take contiguous operands
    too (torch's own hands transposed views on).  They are made of the same
    product, so they can be differentiated and transformed (torch.func) again."""
    generate_vmap_rule = True

    @staticmethod
    def forward(a, b):
        return torch.bmm(a, b)

    @staticmethod
    def setup_context(ctx, inputs, output):
        ctx.save_for_backward(*inputs)
        ctx.save_for_forward(*inputs)

    @staticmethod
    def backward(ctx, dy):
        a, b = (t.to(dy.dtype) for t in ctx.saved_tensors)   # autocast's type, where that was on
        dy = dy.contiguous()
        da = _Bmm.apply(dy, b.transpose(1, 2).contiguous()) if ctx.needs_input_grad[0] else None
        db = _Bmm.apply(a.transpose(1, 2).contiguous(), dy) if ctx.needs_input_grad[1] else None
        return da, db

    @staticmethod
    def jvp(ctx, da, db):
        a, b = ctx.saved_tensors
        return _Bmm.apply(da.contiguous(), b) + _Bmm.apply(a, db.contiguous())


def block_forward(x: torch.Tensor, w: dict, shape: BlockShape, linear=torch.nn.functional.linear) -> torch.Tensor:
    """One Llama block on activations x [T, hidden] (BF16), causal attention.
    linear(x, w[name]) multiplies by a layer's weights."""
    t = x.shape[0]
    hd, nh, nkv = shape.head_dim, shape.heads, shape.kv_heads
    h = _rms_norm(x)
    q = linear(h, w["q"]).view(t, nh, hd).transpose(0, 1).contiguous()
    k = linear(h, w["k"]).view(t, nkv, hd).transpose(0, 1).contiguous()
    v = linear(h, w["v"]).view(t, nkv, hd).transpose(0, 1).contiguous()
    q, k = _rope(q, shape.rope_theta), _rope(k, shape.rope_theta)
    rep = nh // nkv
    k = k.repeat_interleave(rep, dim=0)
    v = v.repeat_interleave(rep, dim=0).contiguous()
    kt = k.transpose(1, 2).contiguous()                       # [heads, hd, T]
    scores = _Bmm.apply(q, kt).float() * (hd ** -0.5)           # [heads, T, T]
    mask = torch.ones(t, t, device=x.device, dtype=torch.bool).triu(1)
    scores.masked_fill_(mask, float("-inf"))
    probs = torch.softmax(scores, dim=-1).to(x.dtype).contiguous()
    att = _Bmm.apply(probs, v).transpose(0, 1).reshape(t, nh * hd)
    x = x + linear(att, w["o"])
    h2 = _rms_norm(x)
    g = linear(h2, w["gate"])
    u = linear(h2, w["up"])
    return x + linear(torch.nn.functional.silu(g) * u, w["down"])


class CompressedBlocks:
    """Blocks held as device-resident containers, decoded one block ahead.

    containers: one host container per block (BF16 kind, matrices in
    BlockShape.matrices() order).  Two scratch buffers of one block each are
    allocated up front; the side stream has the default priority.
    decode_workgroups caps the workgroups of a decode on the side stream
    (0: no cap), so that it runs beside the block's kernels on the CUs they
    leave rather than taking every CU."""

    def __init__(self, containers, shape: BlockShape, device, decode_workgroups: int = 0):
        self.shape = shape
        self.decode_workgroups = int(decode_workgroups)
        self.device = torch.device(device)
        n = shape.elements()
        for c in containers:
            if int(c.info()["n"]) != n or int(c.info()["kind"]) != dfh.KIND_BF16:
                raise ValueError("container does not hold one BF16 block of this shape")
        self.blocks = [dfh.to_device(c, self.device) for c in containers]
        self.scratch = [torch.empty(n, dtype=torch.bfloat16, device=self.device) for _ in range(2)]
        self.side = torch.cuda.Stream(device=self.device)
        self.decoded = [torch.cuda.Event() for _ in range(2)]  # scratch j holds its block
        self.released = [torch.cuda.Event() for _ in range(2)]  # compute done with scratch j

    def _decode(self, i: int, main: torch.cuda.Stream):
        j = i % 2
        self.side.wait_event(self.released[j])
        dfh.df_decompress(self.blocks[i], self.scratch[j], self.side, max_workgroups=self.decode_workgroups)
        self.decoded[j].record(self.side)

    def forward(self, x: torch.Tensor, overlap: bool = True) -> torch.Tensor:
        """All blocks in order.  overlap=False decodes each block on the
        caller's stream right before it runs (no overlap)."""
        main = torch.cuda.current_stream(self.device)
        for j in range(2):
            self.released[j].record(main)
        if overlap:
            self._decode(0, main)
        for i in range(len(self.blocks)):
            j = i % 2
            if overlap:
                if i + 1 < len(self.blocks):
                    self._decode(i + 1, main)
                main.wait_event(self.decoded[j])
            else:
                dfh.df_decompress(self.blocks[i], self.scratch[j], main)
            x = block_forward(x, weight_views(self.scratch[j], self.shape), self.shape)
            self.released[j].record(main)
        return x


class _Made:
    """Device tensors that an object made on the stream then current, and uses on
    others: the first use on another stream waits until they are there, and keeps
    their memory until that stream has passed.  A captured use does neither; its
    capture and replays are ordered by the caller."""

    def __init__(self, device, tensors):
        self.device, self.tensors = device, tensors
        stream = torch.cuda.current_stream(device)
        self.seen = {stream.cuda_stream}
        self.event = torch.cuda.Event()
        self.event.record(stream)

    def use(self, stream=None):
        ts = dfh._torch_stream(stream, self.device)
        if ts.cuda_stream in self.seen:
            return
        with torch.cuda.stream(ts):
            if torch.cuda.is_current_stream_capturing():
                return
        ts.wait_event(self.event)
        for t in self.tensors:
            t.record_stream(ts)
        self.seen.add(ts.cuda_stream)


class QuantizedBlocks:
    """Blocks held as uint4 containers with group scales, decoded to packed
    nibbles right before they run.

    layers: per block a list of (container, scales, zeros) in
    BlockShape.matrices() order, as quantize_block makes them; scales [rows,
    groups] in float32, zeros uint8 of that shape or None.  Scales are kept in
    scale_dtype: bfloat16, the weights' own type, rounds each by up to 2^-8 of itself
    and halves their bytes; torch.float32 keeps the quantiser's.
    One scratch buffer of a block's nibbles is allocated up front.  Calls take turns
    with it, from any thread and on any stream (each waits for the one before); a
    captured call's replays are for the caller to order with what else uses these
    blocks."""

    def __init__(self, layers, shape: BlockShape, device, group_size: int, scale_dtype=torch.bfloat16):
        self.shape = shape
        self.device = torch.device(device)
        mats = shape.matrices()
        self.scratch = [torch.empty(r * c // 2, dtype=torch.uint8, device=self.device) for _, r, c in mats]
        self.blocks, self.weights = [], []
        for block in layers:
            if len(block) != len(mats):
                raise ValueError("a block needs %d layers" % len(mats))
            dcs, ws = [], {}
            for (name, r, c), packed, (con, scales, zeros) in zip(mats, self.scratch, block):
                inf = con.info()
                if int(inf["n"]) != r * c or int(inf["kind"]) != dfh.KIND_U4:
                    raise ValueError("container does not hold the uint4 codes of layer %r" % name)
                dcs.append(dfh.to_device(con, self.device))
                s = torch.as_tensor(scales).to(self.device, scale_dtype)
                z = None if zeros is None else torch.as_tensor(zeros).to(self.device)
                ws[name] = U4Matrix(packed, s, z, cols=c, group_size=group_size)
            self.blocks.append(dcs)
            self.weights.append(ws)
        self._made = _Made(self.device, self.scratch
                           + [t for dcs in self.blocks for dc in dcs for t in dc.sections.values()]
                           + [t for ws in self.weights for w in ws.values() for t in w._tensors()[1:] if t is not None])
        self._lock = threading.RLock()
        self._stream, self._used = None, torch.cuda.Event()  # the last turn's stream, and its end

    @contextlib.contextmanager
    def _turn(self):
        """A block's use of the scratch buffer, from its decode to its last reader."""
        with self._lock, torch.cuda.device(self.device):
            stream = torch.cuda.current_stream(self.device)
            capturing = torch.cuda.is_current_stream_capturing()
            self._made.use(stream)
            if not capturing and self._stream is not None and self._stream != stream:
                stream.wait_event(self._used)
            try:
                yield
            finally:
                if not capturing:
                    self._used.record(stream)
                    self._stream = stream

    def _run(self, i: int, x: torch.Tensor) -> torch.Tensor:
        dfh.df_decompress_batch(self.blocks[i], self.scratch, torch.cuda.current_stream(self.device))
        return block_forward(x, self.weights[i], self.shape, linear_u4)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """All blocks in order on the current stream.  Differentiable in x, once: a
        block keeps its input and is decoded and run again for its gradient."""
        for i in range(len(self.blocks)):
            if x.requires_grad and torch.is_grad_enabled():
                x = _QuantizedBlock.apply(x, self, i)
            else:
                with torch.no_grad(), self._turn():
                    x = self._run(i, x)
        return x


class _QuantizedBlock(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, blocks, i):
        ctx.save_for_backward(x)
        ctx.blocks, ctx.i = blocks, i
        with blocks._turn():
            return blocks._run(i, x)

    @staticmethod
    def backward(ctx, dy):
        return _QuantizedBlockGrad.apply(dy, *ctx.saved_tensors, ctx.blocks, ctx.i), None, None


class _QuantizedBlockGrad(torch.autograd.Function):
    """A block's gradient as a function of all it depends on: a second derivative
    is refused on whatever path it comes."""

    @staticmethod
    def forward(ctx, dy, x, blocks, i):
        with blocks._turn(), torch.enable_grad():
            leaf = x.detach().requires_grad_()
            return torch.autograd.grad(blocks._run(i, leaf), leaf, dy)[0]

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("QuantizedBlocks have no second gradient")


class CompressedHead:
    """An LM head [vocab, hidden] held as one BF16 container (the DF11 digest
    compresses embedding and LM head on their own), decoded into one scratch
    buffer before each use.  The caller orders uses on several streams."""

    def __init__(self, container, vocab: int, hidden: int, device):
        inf = container.info()
        if int(inf["n"]) != vocab * hidden or int(inf["kind"]) != dfh.KIND_BF16:
            raise ValueError("container does not hold a BF16 head of this shape")
        self.device = torch.device(device)
        self.head = dfh.to_device(container, self.device)
        self.scratch = torch.empty((vocab, hidden), dtype=torch.bfloat16, device=self.device)
        self._made = _Made(self.device, [self.scratch, *self.head.sections.values()])

    def weight(self, stream=None) -> torch.Tensor:
        """The decoded head, on a stream (default: the current one; the same bits
        every time)."""
        with torch.cuda.device_of(self.scratch):
            self._made.use(stream)
            dfh.df_decompress(self.head, self.scratch, stream)
        return self.scratch

    def loss(self, x: torch.Tensor, labels: torch.Tensor, *, stream=None, **kw) -> torch.Tensor:
        """Cross entropy of hidden states x against labels (vocab_loss); the head is
        decoded on the loss's stream."""
        return vocab_loss(x, self.weight(stream), labels, stream=stream, **kw)

    def distill(self, x: torch.Tensor, teacher: torch.Tensor, index: torch.Tensor, *, stream=None, **kw) -> torch.Tensor:
        """Divergence from a teacher's top logits (distill_loss), likewise."""
        return distill_loss(x, self.weight(stream), teacher, index, stream=stream, **kw)


def resident_forward(x: torch.Tensor, weights, shape: BlockShape) -> torch.Tensor:
    """The same blocks with every weight buffer resident (the reference)."""
    for flat in weights:
        x = block_forward(x, weight_views(flat, shape), shape)
    return x


def random_blocks(n_blocks: int, shape: BlockShape, seed: int = 0):
    """Host BF16 weights, one flat array per block: N(0, s^2) per matrix with
    s ~ U[0.01, 0.04], from the same generator family as the benchmark."""
    from . import synth
    return [synth.bf16_block(seed, config=synth.CONFIG_FORWARD, block=b, shapes=shape.matrices())[0]
            for b in range(n_blocks)]


def quantize_block(host: np.ndarray, shape: BlockShape, group_size: int, asymmetric: bool = True):
    """One block's host BF16 weights -> QuantizedBlocks' layers: per matrix the
    uint4 container of its codes, its group scales and zero points."""
    from . import synth
    out, off = [], 0
    for _, r, c in shape.matrices():
        w = synth.bf16_to_f32(host[off: off + r * c]).reshape(r, c)
        codes, scales, zeros = synth.quantize_u4_groups(w, group_size, asymmetric)
        out.append((dfh.compress(dfh.KIND_U4, synth.pack_u4(codes), n=r * c), scales, zeros))
        off += r * c
    return out


def to_torch(host: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(host.view(np.int16)).to(device).view(torch.bfloat16)
