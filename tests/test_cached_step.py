"""A block's step over a paged cache: every operator it calls against the formulas in
float64, from the inputs that it was called with, and every operator's inputs bit for
bit from the outputs before it; and what the step refuses.  Here the cache's operators are
stood in for by plain ones on the CPU.

Tolerances.  ``Bounded`` carries with each float64 value how far a computed one may be from
it: each rounding is off by up to half a step (u = eps / 2 of the value, and a subnormal's half
step), float32 sums of n terms by n 2^-24 of the sum of magnitudes, float32 functions by 8
2^-24.
"""
import math
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from lossless_entropy_coded_huffman_amd import forward as fw, synth
from lossless_entropy_coded_huffman_amd.cache import _positions

E = 2.0 ** -24
SHAPE = fw.BlockShape(hidden=128, heads=4, kv_heads=2, ffn=256, rope_theta=10000.0)


class Bounded:
    """Values and how far the computed ones may be from them."""

    def __init__(self, v, e):
        self.v, self.e = v, e

    def most(self):
        return self.v.abs() + self.e

    def rounded(self, dt):
        tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
        return Bounded(self.v, self.e + torch.finfo(dt).eps / 2 * self.most() + tiny)

    def at(self, i):
        return Bounded(self.v[i], self.e[i])


def exact(t):
    t = t.detach().cpu().double()
    return Bounded(t, torch.zeros_like(t))


def quantised(x):
    """What the cache holds of x in 8 bits: the scale is rounded."""
    top = x.v.abs().amax(dim=-1, keepdim=True)
    kept = torch.round(127 * x.v / torch.where(top > 0, top, 1.0)) * top / 127
    return Bounded(kept, 2 * E * kept.abs())


def product(x, w, dt, how):
    """x W^T; how: "bf16" (16-bit weights), "u4" (their products may round a weight too,
    and sum it with a bias of 16 steps: w is then (W, the magnitudes)), "u8" (w is then
    (codes less zero points, scales))."""
    if how == "u8":
        q, scales = w
        top = x.v.abs().amax(dim=-1, keepdim=True)
        codes = torch.round(127 * x.v / torch.where(top > 0, top, 1.0))
        v = (codes @ q.t()) * (top / 127) * scales         # integers' sums are exact, zeros among them
        return Bounded(v, 5 * E * v.abs()).rounded(dt)
    w, magnitudes = w if how == "u4" else (w, w.abs())
    u = torch.finfo(dt).eps / 2 if how == "u4" else 0.0
    y = Bounded(x.v @ w.t(), x.e @ w.abs().t() + x.most() @ (u * w.abs() + w.shape[1] * E * magnitudes).t())
    return y.rounded(dt)


def norm(x, dt, eps=1e-5):
    n = x.v.shape[-1]
    r = (x.v.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    dr = x.e.pow(2).mean(-1, keepdim=True).sqrt()
    v = x.v / r
    e = (x.e + v.abs() * dr) / (r - dr).clamp(min=1e-9)
    return Bounded(v, e + (n + 8) * E * (v.abs() + e)).rounded(dt)


def rope(x, at, theta, dt):
    half = x.v.shape[-1] // 2
    inv = theta ** -(torch.arange(half).double() / half)
    ang = at.double()[:, None, None] * inv
    off = 8 * E * (1 + ang.abs())                       # the angle in float32, its sine and cosine
    c, s = ang.cos(), ang.sin()
    a, b, ea, eb = x.v[..., :half], x.v[..., half:], x.e[..., :half], x.e[..., half:]
    v = torch.cat([a * c - b * s, a * s + b * c], -1)
    both = off * (a.abs() + ea + b.abs() + eb)
    e = torch.cat([ea * c.abs() + eb * s.abs() + both, ea * s.abs() + eb * c.abs() + both], -1)
    return Bounded(v, e).rounded(dt)


def attention(q, k, v, dt, first):
    """q [n, heads, d], the sequence's last tokens from position first on, over k, v
    [len, kv_heads, d]."""
    n, heads, d = q.v.shape
    rep = heads // k.v.shape[1]
    out = Bounded(torch.zeros_like(q.v), torch.zeros_like(q.v))
    for h in range(heads if n else 0):
        Q, K, V = q.at((slice(None), h)), k.at((slice(None), h // rep)), v.at((slice(None), h // rep))
        s = Q.v @ K.v.t() / math.sqrt(d)
        es = (Q.v.abs() @ K.e.t() + Q.e @ K.most().t() + 2 * d * E * Q.most() @ K.most().t()) / math.sqrt(d)
        seen = torch.arange(len(K.v))[None, :] <= first + torch.arange(n)[:, None]
        s, es = s.masked_fill(~seen, -math.inf), es.masked_fill(~seen, 0.0)
        p = torch.softmax(s, -1)
        u = torch.finfo(dt).eps / 2
        # each weight is off by its score's error and the sum's, and is rounded
        off = (es + es.amax(-1, keepdim=True)).exp() * (1 + u) ** 2 * (1 + (len(K.v) + 64) * E) - 1
        out.v[:, h] = p @ V.v
        out.e[:, h] = (p * (1 + off)) @ V.e + (p * off) @ V.v.abs() + len(K.v) * E * (p * (1 + off)) @ V.most()
    return out.rounded(dt)


class Watch:
    """Wraps what block_step calls, and checks each call.  how: the weights' kind; ws: the
    float64 weights of each block; theta, shift, swap: planted mistakes of the oracle."""

    def __init__(self, monkeypatch, seqs, ws, how="bf16", bits=16, theta=SHAPE.rope_theta, shift=0, swap=False):
        self.kept = [[([], []) for _ in range(seqs)] for _ in ws]
        self.seen, self.worst, self.block, self.products = [], 0.0, 0, None
        self.ws, self.how, self.bits, self.theta, self.shift, self.swap = ws, how, bits, theta, shift, swap
        for name in ("_rms_norm", "_rope", "cache_write", "cached_attention"):
            monkeypatch.setattr(fw, name, self.wrapped(name, getattr(fw, name)))

    def wrapped(self, name, f):
        def call(*args):
            out = f(*args)
            getattr(self, name)(out, *args)
            self.seen.append((name, args, out))
            return out
        return call

    def near(self, got, want):
        if got.numel():
            assert bool(torch.isfinite(got).all())
            self.worst = max(self.worst, float(((got.detach().cpu().double() - want.v).abs() / want.e).max()))

    def _rms_norm(self, out, x):
        self.near(out, norm(exact(x), x.dtype))

    def _rope(self, out, x, theta, at):
        at = torch.cat([torch.arange(d - n, d) for d, n in zip(self.done, self.new)]) if sum(self.new) else at[:0].cpu()
        want = rope(exact(x.transpose(0, 1)), at + self.shift, self.theta, x.dtype)
        self.near(out.transpose(0, 1), want)

    def cache_write(self, out, k, v, cache, batch):
        self.rows = 0
        for kept, n in zip(self.kept[self.block], self.new):
            kept[0].append(k[self.rows:self.rows + n].cpu().double())
            kept[1].append(v[self.rows:self.rows + n].cpu().double())
            self.rows += n

    def cached_attention(self, out, q, cache, batch):
        at = 0
        for kept, d, n in zip(self.kept[self.block], self.done, self.new):
            K, V = (Bounded(torch.cat(t), torch.zeros(())) for t in kept)
            assert len(K.v) == d
            K, V = (quantised(t) if self.bits == 8 and d else Bounded(t.v, torch.zeros_like(t.v)) for t in (K, V))
            if self.swap:
                K, V = K.at((slice(None), [1, 0])), V.at((slice(None), [1, 0]))
            self.near(out[at:at + n], attention(exact(q[at:at + n]), K, V, q.dtype, d - n))
            at += n

    def product(self, f, names):
        """products, for the calls of a block in turn: those of names[i] the i-th."""
        def call(x, *ws):
            outs = f(x, *ws)
            turn = names[self.turn % len(names)]
            assert len(turn) == len(ws) == len(outs)
            for n, y in zip(turn, outs):
                self.near(y, product(exact(x), self.ws[self.block][n], x.dtype, self.how))
            self.seen.append(("products", (x,) + ws, outs))
            self.turn += 1
            if self.turn % len(names) == 0:
                self.joined()
                self.block += 1
            return outs
        return call

    def step(self, done, new):
        self.done, self.new, self.block, self.turn, self.seen = done, new, 0, 0, []

    def joined(self):
        """Each call's inputs are the outputs before it; self.out is the block's output."""
        names = [n for n, _, _ in self.seen]
        assert names == ["_rms_norm", "products", "_rope", "_rope", "cache_write", "cached_attention", "products",
                         "_rms_norm", "products", "products"]
        n1, qkv, rq, rk, wr, at, o, n2, gu, down = self.seen
        t = len(n1[1][0])
        flat = lambda y: y.reshape(t, -1)
        q, k, v = qkv[2]
        g, u = gu[2]
        x = n1[1][0]
        mid = x + o[2][0]
        pairs = [(qkv[1][0], n1[2]), (flat(rq[1][0].transpose(0, 1)), q), (flat(rk[1][0].transpose(0, 1)), k),
                 (wr[1][0], rk[2].transpose(0, 1)), (flat(wr[1][1]), v), (at[1][0], rq[2].transpose(0, 1)),
                 (o[1][0], flat(at[2])), (n2[1][0], mid), (gu[1][0], n2[2]),
                 (down[1][0], torch.nn.functional.silu(g) * u)]
        if self.block:
            pairs.append((x, self.out))
        for a, b in pairs:
            assert torch.equal(a, b)
        self.out = mid + down[2][0]
        self.seen = []


CALLS = [("q", "k", "v"), ("o",), ("gate", "up"), ("down",)]


class Held:
    """A cache and a batch on the CPU, as plain lists of tokens."""

    def __init__(self, seqs, shape, dtype=torch.bfloat16):
        self.kv = [([], []) for _ in range(seqs)]
        self.kv_heads, self.head_dim, self.dtype = shape.kv_heads, shape.head_dim, dtype


def held_write(k, v, cache, batch):
    for s, kept in enumerate(cache.kv):
        for r in range(int(batch.starts[s]), int(batch.starts[s + 1])):
            kept[0].append(k[r].clone())
            kept[1].append(v[r].clone())


def held_attention(q, cache, batch):
    out = torch.zeros(q.shape, dtype=q.dtype)
    for s, kept in enumerate(cache.kv):
        a, b = int(batch.starts[s]), int(batch.starts[s + 1])
        if a < b:
            K, V = (exact(torch.stack(t)) for t in kept)
            out[a:b] = attention(exact(q[a:b]), K, V, q.dtype, len(K.v) - (b - a)).v.to(q.dtype)
    return out


def plan(lengths, pieces, seed=0):
    """Steps that bring sequences to their lengths: for each step the new tokens of each."""
    g = np.random.default_rng(seed)
    left, steps = list(lengths), []
    for i in range(pieces - 1):
        new = [int(g.integers(0, n + 1)) if i % 2 else min(n, 1) for n in left]
        left = [n - m for n, m in zip(left, new)]
        steps.append(new)
    return steps + [left]


def run(step, x, steps):
    """step(rows, lengths, new) for each step of the sequences x."""
    done = [0] * len(x)
    for new in steps:
        rows = torch.cat([s[d:d + n] for s, d, n in zip(x, done, new)])
        done = [d + n for d, n in zip(done, new)]
        step(rows, done, new)


def ints(a, device="cpu"):
    return torch.tensor(a, dtype=torch.int32, device=device)


def starts_of(new):
    return [0] + [int(n) for n in np.cumsum(new)]


def inputs(lengths, dt=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, SHAPE.hidden, generator=g).to(dt) for n in lengths]


LENGTHS = [1, 37, 0, 20]


def weights(blocks, seed=4):
    return [fw.weight_views(fw.to_torch(h, "cpu"), SHAPE) for h in fw.random_blocks(blocks, SHAPE, seed)]


@pytest.mark.parametrize("mistake", [{}, dict(theta=20000.0), dict(shift=1), dict(swap=True)])
def test_block_step(monkeypatch, mistake):
    monkeypatch.setattr(fw, "cache_write", held_write)
    monkeypatch.setattr(fw, "cached_attention", held_attention)
    ws = weights(2)
    watch = Watch(monkeypatch, len(LENGTHS), [{n: t.double() for n, t in w.items()} for w in ws], **mistake)
    caches = [Held(len(LENGTHS), SHAPE) for _ in ws]
    products = watch.product(fw._products(torch.nn.functional.linear), CALLS)

    def step(x, done, new):
        watch.step(done, new)
        batch = SimpleNamespace(starts=ints(starts_of(new)))
        at = _positions(ints(done), batch.starts, len(x))
        for w, cache in zip(ws, caches):
            x = fw.block_step(x, w, SHAPE, cache, batch, at, products)
        assert torch.equal(x, watch.out)

    run(step, inputs(LENGTHS), plan(LENGTHS, 5))
    assert (watch.worst > 1) == bool(mistake)        # the oracle's mistakes are seen


def test_positions():
    def at(lengths, starts, tokens):
        return _positions(torch.tensor(lengths, dtype=torch.int32), torch.tensor(starts, dtype=torch.int32), tokens).tolist()

    assert at([5, 9, 2, 1], [0, 2, 2, 4, 5], 7) == [3, 4, 0, 1, 0, -1, -1]
    assert at([3], [1, 3], 4) == [-1, 1, 2, -1]
    assert at([1], [0, 3], 3) == [-1, -1, 0]              # rows before position 0
    assert at([], [0], 2) == [-1, -1] and at([4], [0, 0], 0) == []
    big = (1 << 31) - 1
    assert at([big], [0, 2], 2) == [big - 2, big - 1]


def test_rope_at_positions():
    x = torch.randn(3, 9, 16).to(torch.bfloat16)
    whole = fw._rope(x, 500.0)
    for order in (torch.arange(9), torch.tensor([4, 0, 8, 8, 3, 1, 2, 7, 5])):
        assert torch.equal(fw._rope(x[:, order], 500.0, order), whole[:, order])


def test_refused_steps():
    cache = Held(1, SHAPE)
    x = torch.zeros(2, SHAPE.hidden, dtype=torch.bfloat16)
    fw._check_step(x, [cache], 1, SHAPE)
    for bad in (x[0], x[:, :-1], x[None]):
        with pytest.raises(ValueError):
            fw._check_step(bad, [cache], 1, SHAPE)
    with pytest.raises(ValueError):
        fw._check_step(x, [cache, cache], 1, SHAPE)
    with pytest.raises(ValueError):
        fw._check_step(x, [], 1, SHAPE)
    for name, v in (("kv_heads", 4), ("head_dim", 64), ("dtype", torch.float16)):
        other = Held(1, SHAPE)
        setattr(other, name, v)
        with pytest.raises(ValueError):
            fw._check_step(x, [other], 1, SHAPE)
    with pytest.raises(RuntimeError):
        fw._check_step(x.float().requires_grad_(), [cache], 1, SHAPE)


@pytest.mark.parametrize("asymmetric", [False, True])
def test_uint8_rows(asymmetric):
    x = np.random.default_rng(1).normal(size=(6, 80)).astype(np.float32) * np.float32(0.02)
    x[2] = 0
    x[3] = 0.5
    codes, s, z = synth.quantize_u8_rows(x, asymmetric)
    assert codes.shape == x.shape and s.shape == z.shape == (6,) and s.dtype == np.float32 and z.dtype == np.uint8
    for r in (0, 1, 2, 4, 5):
        assert np.array_equal(codes[r], synth.quantize_u8(x[r], asymmetric))
        back = s[r].astype(np.float64) * (codes[r].astype(np.float64) - z[r])
        # a code and the zero point are each off by half a step, and the ends may be cut by as much
        assert np.abs(back - x[r]).max() <= s[r] * (1 + 1e-5)


@pytest.mark.parametrize("kw", [dict(group_size=None), dict(group_size=64, bits=8), dict(group_size=64, bits=16)])
def test_refused_blocks(kw):
    with pytest.raises(ValueError):
        fw.QuantizedBlocks([], SHAPE, "cpu", **kw)
