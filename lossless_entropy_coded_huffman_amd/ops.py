"""Operators on what the codec stores, through the C ABI (include/dfh.h):

* ``linear_u4``: products with uint4 weights and group scales, the packed
  nibbles that ``df_decompress`` yields for a uint4 container, for one token up
  to long prompts, with the gradient to the input;
* ``vocab_loss``: softmax cross entropy of hidden states against an LM head,
  the logits never stored, with the gradients to both;
* ``distill_loss``: the divergence from a teacher's top logits over the same
  head, with the gradients to both.

Everything is enqueued on ``stream`` (default: the current stream of the
tensors' device) and returns without synchronising.  Outputs and workspaces are
torch tensors allocated on that stream, so a call can be captured into a HIP
graph, and two calls never share one.  A call given another stream than the
current one does not wait for the current one: the caller orders the streams.  An
input that another stream may free while the call runs is recorded on the call's
stream.

In autograd a gradient runs on the stream that was current in the forward call,
after a forward call that was given another one.  linear_u4 can be differentiated
again; a gradient of a loss's gradient is refused, and so is forward mode.  To
capture a training step into a HIP graph, make its leaves inside the capture
(``x.detach().requires_grad_()``): a leaf that an eager graph still holds ties the
captured backward to that graph's stream.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad

from . import dfh

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_REDUCE = {"none": 0, "sum": 1, "mean": 2}


def _type(t: torch.Tensor, what: str, f32: bool = False) -> int:
    if t.dtype not in _TYPES or (t.dtype == torch.float32 and not f32):
        raise TypeError("%s must be bfloat16%s, got %s" % (what, ", float16 or float32" if f32 else " or float16",
                                                           t.dtype))
    return _TYPES[t.dtype]


def _on(t: torch.Tensor, dev: torch.device, what: str):
    if not t.is_cuda or t.device != dev:
        raise ValueError("%s must be a tensor on %s" % (what, dev))


def _no_tangent(*tensors):
    """Refuses forward mode, whose tangents the kernels would drop (they are there
    only inside a dual level, and without gradients enabled too)."""
    if forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError("no forward-mode derivative is offered")


_MAX_STRIDE = 1 << 21   # the kernels' largest row stride


def _copied(t: torch.Tensor) -> torch.Tensor:
    """A copy with a contiguous tensor's strides (contiguous() may return t itself,
    with any stride in a dimension of one element)."""
    return t.clone(memory_format=torch.contiguous_format)


def _rows16(t: torch.Tensor) -> torch.Tensor:
    """t [r, c] with a row stride that is a multiple of 8 elements and at most 2^21,
    unit column stride and a 16-byte aligned base: itself, or a copy."""
    step, one = t.stride()
    if one == 1 and step % 8 == 0 and t.shape[1] <= step <= _MAX_STRIDE and t.data_ptr() % 16 == 0:
        return t
    return _copied(t)


def _flat(t: torch.Tensor) -> torch.Tensor:
    """t [..., c] as rows."""
    return t if t.dim() == 2 else t.reshape(-1, t.shape[-1])


# the current device, and the raw handle of a device's current stream, without
# the objects that torch.cuda makes around them (a token's product is short)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(stream, dev, tensors, call):
    """call(stream handle) with the stream it runs on current (and its device);
    inputs are recorded on a stream that was not."""
    if stream is None and _current_device() == dev.index:
        return call(_raw_stream(dev.index))
    cur = torch.cuda.current_stream(dev)
    ts = cur if stream is None else dfh._torch_stream(stream, dev)
    with torch.cuda.device(dev), torch.cuda.stream(ts):
        out = call(ts.cuda_stream)
        if ts.cuda_stream != cur.cuda_stream:
            for t in tensors:
                if t is not None:
                    t.record_stream(ts)
    return out


def _workspace(nbytes: int, dev) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=dev)


def _p(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------- uint4 products
class U4Matrix:
    """A layer's uint4 weights on the device (df_u4_matrix; the tensors are
    borrowed and kept alive).

    packed: the nibbles, rows * cols / 2 bytes (what ``df_decompress`` writes
    for a uint4 container of the layer); scales [rows, groups] in bfloat16,
    float16 or float32, groups = ceil(cols / group_size); zeros: uint8 zero
    points of the same shape, or None for 8.  group_size (default: cols) is a
    multiple of 32, or at least cols.  scales and zeros may be broadcast over
    the rows (stride 0): one scale for a layer is
    ``scale.reshape(1, 1).expand(rows, 1)``."""

    def __init__(self, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None, *, cols: int,
                 group_size: int | None = None):
        cols = int(cols)
        group_size = cols if group_size is None else int(group_size)
        if not packed.is_cuda or not packed.is_contiguous() or packed.element_size() != 1:
            raise ValueError("packed must be a contiguous byte tensor on the device")
        if cols < 8 or cols % 8 or cols > 1 << 20:
            raise ValueError("cols must be a multiple of 8 from 8 to 2^20, got %d" % cols)
        if group_size < 1 or (group_size < cols and group_size % 32):
            raise ValueError("group_size must be a multiple of 32, or at least cols")
        if scales.dim() != 2:
            raise ValueError("scales must be [rows, groups]")
        rows, groups = int(scales.shape[0]), (cols + group_size - 1) // group_size
        if rows < 1 or rows > 1 << 21 or scales.shape[1] != groups:
            raise ValueError("scales must be [rows, %d] with 1 to 2^21 rows, got %s" % (groups, tuple(scales.shape)))
        if packed.numel() < rows * cols // 2:
            raise ValueError("packed holds fewer than %d x %d nibbles" % (rows, cols))
        if packed.data_ptr() % 4:
            raise ValueError("packed must be 4-byte aligned")
        _on(scales, packed.device, "scales")
        self.scale_type = _type(scales, "scales", f32=True)
        if zeros is not None:
            _on(zeros, packed.device, "zeros")
            if zeros.dtype != torch.uint8 or zeros.shape != scales.shape:
                raise ValueError("zeros must be uint8 of the scales' shape")
        if scales.requires_grad:
            raise ValueError("no gradient goes to the scales: detach them")
        _no_tangent(scales)
        if groups > 1 and scales.stride(1) != 1:
            scales = scales.contiguous()
        if zeros is not None and groups > 1 and zeros.stride(1) != 1:
            zeros = zeros.contiguous()
        self.packed, self.scales, self.zeros = packed, scales, zeros
        self.rows, self.cols, self.group_size, self.device = rows, cols, group_size, packed.device
        self.view = dfh.df_u4_matrix(rows, cols, min(group_size, 0xFFFFFFFF), self.scale_type, scales.stride(0),
                                     0 if zeros is None else zeros.stride(0), packed.data_ptr(), scales.data_ptr(),
                                     _p(zeros))
        self._ref = ctypes.byref(self.view)
        self._need, self._need_grad = {}, {}   # workspace bytes by row count

    def _tensors(self):
        return (self.packed, self.scales, self.zeros)


def _linear_on(x: torch.Tensor, w: U4Matrix, ty: int, handle: int) -> torch.Tensor:
    """y [m, rows] for x [..., cols] on a stream, which a copy of x is made on too."""
    x = _rows16(_flat(x))
    m = x.shape[0]
    y = x.new_empty((m, w.rows))
    L = dfh.lib()
    need = w._need.get(m)
    if need is None:
        need = w._need[m] = L.df_linear_u4_workspace_bytes(w._ref, m)
    ws = _workspace(need, w.device) if need else None
    st = L.df_linear_u4(w._ref, ty, x.data_ptr(), m, x.stride(0), y.data_ptr(), _p(ws), need, handle)
    if st:
        dfh._check(st, "df_linear_u4")
    return y


def _linear(x: torch.Tensor, w: U4Matrix, stream) -> torch.Tensor:
    dev, shape = w.device, x.shape
    if x.device != dev:
        _on(x, dev, "x")
    ty = _type(x, "x")
    if not shape or shape[-1] != w.cols:
        raise ValueError("x must be [..., %d], got %s" % (w.cols, tuple(shape)))
    if stream is None and _current_device() == dev.index:
        y = _linear_on(x, w, ty, _raw_stream(dev.index))
    else:
        y = _launch(stream, dev, (x,) + w._tensors(), lambda handle: _linear_on(x, w, ty, handle))
    return y if len(shape) == 2 else y.view(shape[:-1] + (w.rows,))


def _linear_grad(dy: torch.Tensor, w: U4Matrix, stream) -> torch.Tensor:
    dev = w.device
    if dy.device != dev:
        _on(dy, dev, "dy")
    ty = _type(dy, "dy")
    if dy.dim() < 1 or dy.shape[-1] != w.rows:
        raise ValueError("dy must be [..., %d], got %s" % (w.rows, tuple(dy.shape)))
    L = dfh.lib()

    def call(handle):
        d2 = _flat(dy)
        if w.rows % 8 == 0:
            d2 = _rows16(d2)
        elif d2.stride(1) != 1 or not w.rows <= d2.stride(0) <= _MAX_STRIDE:
            d2 = _copied(d2)
        m = d2.shape[0]
        dx = torch.empty((m, w.cols), dtype=dy.dtype, device=dev)
        need = w._need_grad.get(m)
        if need is None:
            need = w._need_grad[m] = L.df_linear_u4_grad_workspace_bytes(w._ref, m)
        ws = _workspace(need, dev)
        st = L.df_linear_u4_grad(w._ref, ty, d2.data_ptr(), m, d2.stride(0), dx.data_ptr(), ws.data_ptr(), need, handle)
        if st:
            dfh._check(st, "df_linear_u4_grad")
        return dx

    dx = _launch(stream, dev, (dy,) + w._tensors(), call)
    return dx if dy.dim() == 2 else dx.view(dy.shape[:-1] + (w.cols,))


def _keep_weights(ctx, w: U4Matrix, stream):
    """For a derivative, which reads the weights again: a change that torch sees in
    between is refused, and a call that was given a stream is waited for."""
    ctx.w, ctx.done = w, None
    ctx.save_for_backward(*[t for t in w._tensors() if t is not None])
    if stream is not None:
        ctx.done = torch.cuda.Event()
        ctx.done.record(dfh._torch_stream(stream, w.device))


def _kept_weights(ctx) -> U4Matrix:
    ctx.saved_tensors
    if ctx.done is not None:
        torch.cuda.current_stream(ctx.w.device).wait_event(ctx.done)
    return ctx.w


class _LinearU4(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, stream):
        y = _linear(x, w, stream)
        _keep_weights(ctx, w, stream)
        return y

    @staticmethod
    def backward(ctx, dy):
        return linear_u4_grad(dy, _kept_weights(ctx)), None, None


class _LinearU4Grad(torch.autograd.Function):
    """dx is linear in dy, and its derivative the product itself."""

    @staticmethod
    def forward(ctx, dy, w, stream):
        dx = _linear_grad(dy, w, stream)
        _keep_weights(ctx, w, stream)
        return dx

    @staticmethod
    def backward(ctx, ddx):
        return linear_u4(ddx, _kept_weights(ctx)), None, None


def linear_u4_grad(dy: torch.Tensor, w: U4Matrix, stream=None) -> torch.Tensor:
    """dx[..., k] = sum over n of dy[..., n] W[n, k]: the gradient of linear_u4
    to its input, in dy's type (bfloat16 or float16).  Differentiable in dy."""
    _no_tangent(dy)
    if dy.requires_grad and torch.is_grad_enabled():
        return _LinearU4Grad.apply(dy, w, stream)
    return _linear_grad(dy, w, stream)


def linear_u4(x: torch.Tensor, w: U4Matrix, stream=None) -> torch.Tensor:
    """y = x W^T for W[n, k] = scales[n, k // group_size] * (q[n, k] - zeros[...]),
    x [..., cols] in bfloat16 or float16, y [..., rows] in the same type.  Sums
    are float32; few rows (up to 192; 384 for at most 2^24 weights, 512 for at most
    2^22) round no weight (float16 sums x (q - z); bfloat16 x (16 + q), and takes
    16 + z times the sum of x off), more (and every gradient) round each weight once
    to x's type, with scales of any size within range.  Differentiable in x;
    the nibbles must stay as they are until the gradient has run (df_decompress
    into the same buffer is not seen by autograd)."""
    _no_tangent(x)
    if x.requires_grad and torch.is_grad_enabled():
        return _LinearU4.apply(x, w, stream)
    return _linear(x, w, stream)


# ---------------------------------------------------------------------- losses
class _Loss:
    """A call's df_loss and, until autograd has them, the tensors it points to."""

    def __init__(self, x, head, reduction, labels=None, ignore_index=-100, teacher=None, index=None, temperature=1.0):
        if reduction not in _REDUCE:
            raise ValueError("reduction must be 'none', 'sum' or 'mean', got %r" % (reduction,))
        if not head.is_cuda or head.dim() != 2:
            raise ValueError("head must be a [vocab, hidden] tensor on the device")
        vocab, hidden = int(head.shape[0]), int(head.shape[1])
        dev = head.device
        _on(x, dev, "x")
        ty = _type(head, "head")
        if x.dtype != head.dtype:
            raise TypeError("x and head must have one type, got %s and %s" % (x.dtype, head.dtype))
        if x.dim() < 1 or x.shape[-1] != hidden:
            raise ValueError("x must be [..., %d], got %s" % (hidden, tuple(x.shape)))
        if hidden < 8 or hidden % 8 or hidden > 1 << 17:
            raise ValueError("hidden must be a multiple of 8 from 8 to 2^17, got %d" % hidden)
        if vocab < 1 or vocab > 1 << 21:
            raise ValueError("vocab must lie in 1 .. 2^21, got %d" % vocab)
        self.shape = tuple(x.shape[:-1])
        self.reduction = reduction
        d = dfh.df_loss()
        d.type, d.reduce, d.vocab, d.hidden = ty, _REDUCE[reduction], vocab, hidden
        d.temperature = float(temperature)
        d.ignore_index = int(ignore_index)
        if labels is not None:
            _on(labels, dev, "labels")
            if labels.dtype != torch.int64 or tuple(labels.shape) != self.shape:
                raise ValueError("labels must be int64 of shape %s" % (self.shape,))
        else:
            if not 1e-3 <= float(temperature) <= 1e3:
                raise ValueError("temperature must lie in 0.001 .. 1000, got %r" % (temperature,))
            _on(teacher, dev, "teacher")
            _on(index, dev, "index")
            d.teacher_type = _type(teacher, "teacher", f32=True)
            if index.dtype != torch.int64 or tuple(index.shape[:-1]) != self.shape or index.shape != teacher.shape:
                raise ValueError("index must be int64 of shape %s + (top,), like teacher" % (self.shape,))
            d.top = int(index.shape[-1])
            if not 1 <= d.top <= 1024:
                raise ValueError("top must lie in 1 .. 1024, got %d" % d.top)
        self.inputs = (x, head, labels) if labels is not None else (x, head, teacher, index)
        self.desc, self.dev = d, dev
        self.done = None   # an event behind the forward call, where that ran on another stream

    @staticmethod
    def bind(d, x, head, *targets):
        """Lays the inputs out and points the descriptor d at them (on the call's
        stream).  Returns them as they lie, in the same order."""
        x, head = _rows16(_flat(x)), _rows16(head)
        d.rows = x.shape[0]
        d.x, d.x_stride, d.head, d.head_stride = x.data_ptr(), x.stride(0), head.data_ptr(), head.stride(0)
        if not d.top:
            labels = targets[0] if targets[0].dim() == 1 else targets[0].reshape(-1)
            if not labels.is_contiguous():
                labels = labels.contiguous()
            d.labels = labels.data_ptr()
            return x, head, labels
        teacher, index = _flat(targets[0].detach()), _flat(targets[1])
        if teacher.stride(1) != 1:
            teacher = teacher.contiguous()
        if index.stride(1) != 1:
            index = index.contiguous()
        d.teacher, d.teacher_stride = teacher.data_ptr(), teacher.stride(0)
        d.index, d.index_stride = index.data_ptr(), index.stride(0)
        return x, head, teacher, index

    def forward(self, stream):
        """The loss and what the gradient wants kept beside the inputs: their laid
        out copies, where there are any, and the rows' statistics."""
        L, dev = dfh.lib(), self.dev
        none = self.reduction == "none"
        current = _raw_stream(dev.index)

        def call(handle):
            laid = self.bind(self.desc, *self.inputs)
            ref = ctypes.byref(self.desc)
            loss = torch.empty(self.shape if none else (), dtype=torch.float32, device=dev)
            saved = torch.empty(max(L.df_loss_saved_bytes(ref) // 4, 1), dtype=torch.float32, device=dev)
            need = L.df_loss_workspace_bytes(ref)
            ws = _workspace(need, dev)
            st = L.df_vocab_loss(ref, loss.data_ptr(), saved.data_ptr(), ws.data_ptr(), need, handle)
            if st:
                dfh._check(st, "df_vocab_loss")
            if handle != current:
                self.done = torch.cuda.Event()
                self.done.record()   # on the call's stream
            # which of the kept tensors the kernels read for each input, and where they lie
            self.forms = [(t.shape, t.dtype) for t in self.inputs]
            self.places, copies = list(range(len(laid))), []
            for i, t in enumerate(self.inputs):
                if laid[i].data_ptr() != t.data_ptr():
                    self.places[i] = len(laid) + len(copies)
                    copies.append(laid[i])
            kept = (*copies, saved)
            self.lie = self.where((*self.inputs, *kept))
            return loss, kept

        return _launch(stream, dev, self.inputs, call)

    def where(self, kept):
        return [(kept[i].data_ptr(), kept[i].stride()) for i in self.places]

    def grads(self, kept, gout, want_x, want_head):
        """kept: the inputs, then what the forward call returned."""
        L, dev = dfh.lib(), self.dev
        saved = kept[-1]

        def call(handle):
            if self.done is not None:
                # what the forward call keeps is written, and was allocated, on its stream
                here = torch.cuda.current_stream(dev)
                here.wait_event(self.done)
                for t in kept:
                    t.record_stream(here)
            desc, laid = self.desc, None
            if self.where(kept) != self.lie:   # saved-tensor hooks put them elsewhere
                if [(t.shape, t.dtype) for t in kept[:len(self.forms)]] != self.forms:
                    raise RuntimeError("the loss's inputs came back with other shapes or types")
                desc = dfh.df_loss.from_buffer_copy(desc)
                laid = self.bind(desc, *[kept[i] for i in self.places])
            ref = ctypes.byref(desc)
            g = gout.to(torch.float32).contiguous()
            (xs, ty), (hs, _) = self.forms[:2]
            dx = torch.empty(xs, dtype=ty, device=dev) if want_x else None
            dh = torch.empty(hs, dtype=ty, device=dev) if want_head else None
            need = L.df_loss_grad_workspace_bytes(ref, int(want_head))
            ws = _workspace(need, dev)
            st = L.df_vocab_loss_grad(ref, saved.data_ptr(), g.data_ptr(), _p(dx), _p(dh), ws.data_ptr(), need, handle)
            if st:
                dfh._check(st, "df_vocab_loss_grad")
            del laid   # enqueued: the copies' memory follows in the stream's order
            return dx, dh

        return _launch(None, dev, (), call)


class _LossFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, head, call, stream):
        loss, kept = call.forward(stream)
        if call.done is not None and torch._C._autograd._top_saved_tensors_default_hooks(False) is not None:
            # a hook reads what the call on the other stream still writes
            here = torch.cuda.current_stream(call.dev)
            here.wait_event(call.done)
            for t in kept:
                t.record_stream(here)
        # the tensors that the gradient reads again: kept by autograd alone, so that
        # a change made to one in between is refused and saved-tensor hooks see all
        ctx.save_for_backward(*call.inputs, *kept)
        call.inputs = None
        ctx.call = call
        return loss

    @staticmethod
    def backward(ctx, gout):
        _no_tangent(gout)
        call, kept, want = ctx.call, ctx.saved_tensors, ctx.needs_input_grad
        if torch.is_grad_enabled():   # under create_graph
            dx, dh = _LossGrad.apply(gout, kept[0], kept[1], call, kept, want)
        else:
            dx, dh = call.grads(kept, gout, want[0], want[1])
        return dx, dh, None, None


class _LossGrad(torch.autograd.Function):
    """The gradients as a function of all they depend on: a second derivative is
    refused on whatever path it comes."""

    @staticmethod
    def forward(ctx, gout, x, head, call, kept, want):
        return call.grads(kept, gout, want[0], want[1])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("vocab_loss and distill_loss have no second gradient")


def _run_loss(call, stream):
    x, head = call.inputs[0], call.inputs[1]
    _no_tangent(x, head)
    if torch.is_grad_enabled() and (x.requires_grad or head.requires_grad):
        return _LossFunction.apply(x, head, call, stream)
    return call.forward(stream)[0]


def vocab_loss(x: torch.Tensor, head: torch.Tensor, labels: torch.Tensor, *, ignore_index: int = -100,
               reduction: str = "mean", stream=None) -> torch.Tensor:
    """Softmax cross entropy of the logits x head^T against labels.

    x [..., hidden] and head [vocab, hidden] in bfloat16 or float16 (one type),
    labels [...] int64.  Rows labelled ignore_index have no loss and no gradient,
    whatever x holds there; another label outside the vocabulary gives NaN in
    its row's loss and no gradient.  reduction "mean" is over the rows that have
    a loss (0 when there are none), "sum", or "none" (the shape of labels).
    The loss is float32.  Differentiable in x and head."""
    return _run_loss(_Loss(x, head, reduction, labels=labels, ignore_index=ignore_index), stream)


def distill_loss(x: torch.Tensor, head: torch.Tensor, teacher: torch.Tensor, index: torch.Tensor, *,
                 temperature: float = 1.0, reduction: str = "mean", stream=None) -> torch.Tensor:
    """Divergence of the student's softmax over the whole vocabulary from the
    teacher's over its top logits:

        t = softmax(teacher / T),  q = softmax(x head^T / T)
        loss = T^2 sum_j t_j (log t_j - log q[index_j])

    teacher [..., top] (bfloat16, float16 or float32) and index [..., top]
    (int64), as torch.topk gives them; entries whose index lies outside the
    vocabulary (-1) are padding, a row of padding has no loss and no gradient.
    top is at most 1024, T lies in 0.001 .. 1000.  x, head, reduction and the result as in vocab_loss.
    Differentiable in x and head; the teacher gets no gradient."""
    return _run_loss(_Loss(x, head, reduction, teacher=teacher, index=index, temperature=temperature), stream)
