"""Where a call that is given a stream does its work: everything that it enqueues
lies inside the launch on that stream.  Plain stand-ins for the kernels, no GPU
needed."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from lossless_entropy_coded_huffman_amd import dfh, ops
from lossless_entropy_coded_huffman_amd import forward as fw


class Launches(TorchDispatchMode):
    """Notes the copies made outside a launch."""

    def __init__(self):
        super().__init__()
        self.inside, self.early = False, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if not self.inside and func in (torch.ops.aten.clone.default, torch.ops.aten.copy_.default):
            self.early.append(func)
        return func(*args, **(kwargs or {}))


class Dense:
    def __init__(self, weight):
        self.weight, self.device = weight, weight.device
        self.rows, self.cols = weight.shape

    def _tensors(self):
        return (self.weight, None)


@pytest.fixture
def launches(monkeypatch):
    mode = Launches()

    def launch(stream, dev, tensors, call):
        mode.inside = True
        try:
            return call(0)
        finally:
            mode.inside = False

    monkeypatch.setattr(ops, "_launch", launch)
    return mode


@pytest.mark.parametrize("shape", [(3, 4, 16), (2, 3, 5, 16)])
def test_linear_u4_lays_x_out_on_its_stream(launches, monkeypatch, shape):
    # leading dimensions that are no view of rows: reshape copies
    w = Dense(torch.randn(8, 16, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16))
    x = torch.randn(shape, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).transpose(0, -2)
    monkeypatch.setattr(ops, "_linear_on", lambda x, w, ty, handle: x @ w.weight.t())
    want = x.reshape(-1, 16) @ w.weight.t()
    with launches:
        y = ops._linear(x, w, object())
    assert not launches.early
    assert y.shape == x.shape[:-1] + (8,) and torch.equal(y.reshape(-1, 8), want)


class Made:
    def use(self, stream=None):
        pass


@pytest.mark.parametrize("call", ["loss", "distill"])
def test_compressed_head_decodes_on_the_losses_stream(monkeypatch, call):
    where = []
    monkeypatch.setattr(dfh, "df_decompress", lambda dc, dst, stream=None: where.append(("decode", stream)))
    for fn in ("vocab_loss", "distill_loss"):
        monkeypatch.setattr(fw, fn, lambda *a, stream=None, **kw: where.append(("loss", stream)))
    head = fw.CompressedHead.__new__(fw.CompressedHead)
    head.device, head.head, head.scratch = torch.device("cpu"), None, torch.zeros(4, 8)
    head._made = Made()
    args = (None,) * (2 if call == "loss" else 3)
    getattr(head, call)(*args, stream=77, reduction="sum")
    assert where == [("decode", 77), ("loss", 77)]
    # and without one, both on the one that is current
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    del where[:]
    getattr(head, call)(*args)
    assert where == [("decode", None), ("loss", None)]


def test_gradient_of_a_product_waits_for_the_stream_of_its_forward_call(monkeypatch):
    log = []

    class Event:
        def record(self, stream):
            log.append(("record", stream))

    class Current:
        def wait_event(self, event):
            log.append("wait")

    w = Dense(torch.ones(8, 16))
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Current())
    monkeypatch.setattr(dfh, "_torch_stream", lambda stream, device: stream)
    monkeypatch.setattr(ops, "_linear", lambda x, w, stream: log.append(("product", stream)) or x @ w.weight.t())
    monkeypatch.setattr(ops, "_linear_grad", lambda dy, w, stream: log.append(("gradient", stream)) or dy @ w.weight)
    x = torch.ones(3, 16, requires_grad=True)
    ops.linear_u4(x, w, stream=5).sum().backward()
    assert log == [("product", 5), ("record", 5), "wait", ("gradient", None)]
    del log[:]
    ops.linear_u4(x, w).sum().backward()
    assert log == [("product", None), ("gradient", None)]


def test_what_an_object_made_is_waited_for_once_on_each_other_stream(monkeypatch):
    log, capturing = [], [False]

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

        def wait_event(self, event):
            log.append(("wait", self.cuda_stream))

    class Event:
        def record(self, stream):
            log.append(("made", stream.cuda_stream))

    class Tensor:
        def record_stream(self, stream):
            log.append(("keep", stream.cuda_stream))

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(1))
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(dfh, "_torch_stream", lambda stream, device: Stream(1) if stream is None else Stream(stream))
    made = fw._Made("cuda", [Tensor(), Tensor()])
    assert log == [("made", 1)]
    made.use()
    capturing[0] = True
    made.use(2)
    assert log == [("made", 1)]
    capturing[0] = False
    made.use(2)
    made.use(2)
    made.use(3)
    assert log == [("made", 1)] + [(what, s) for s in (2, 3) for what in ("wait", "keep", "keep")]


def test_saved_tensor_hooks_wait_for_the_stream_of_the_forward_call(monkeypatch):
    log = []

    class Current:
        def wait_event(self, event):
            log.append(("wait", event))

    class Kept(torch.Tensor):
        def record_stream(self, stream):
            log.append("keep")

    class Call:
        done, dev = "end", None

        def __init__(self, x):
            self.inputs = (x, x.detach())

        def forward(self, stream):
            return self.inputs[0].sum(), (torch.zeros(1).as_subclass(Kept),)

    def pack(t):
        log.append("pack")
        return t

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Current())
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        ops._run_loss(Call(torch.ones(3, requires_grad=True)), 5)
    assert log[:3] == [("wait", "end"), "keep", "pack"]
    del log[:]
    ops._run_loss(Call(torch.ones(3, requires_grad=True)), 5)
    assert not log
