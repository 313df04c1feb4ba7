"""What the operators on quantised and scored models cost: the cases, their
inputs and the plain forms.

The operators:

* ``linear_u4``: products with uint4 weights and group scales, the packed
  nibbles that a uint4 container decodes to, and the gradient to the input;
* ``vocab_loss``: softmax cross entropy over a large vocabulary from hidden
  states and head weights, without keeping the logits, with its gradients;
* ``distill_loss``: the divergence from a teacher's top logits over the same
  head, with its gradients.

``own`` False runs each in its plain form (elementary torch operations in
float32, rounded once at the end), True through the package's calls.
``exact`` gives the same outputs from the definitions in float64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one token through the k or v projection of an 8B-shaped block: the
        # smallest product, where latency counts
        dict(name="u4_token_kv", op="linear", rows=1, n=1024, k=4096, group=128, dtype="bf16", scale="bf16",
             zeros=True),
        # one token through the gate projection of the same block
        dict(name="u4_token_gate", op="linear", rows=1, n=14336, k=4096, group=128, dtype="bf16", scale="bf16",
             zeros=True),
        # one token through the gate projection of a 405B-shaped block
        dict(name="u4_token_405b", op="linear", rows=1, n=53248, k=16384, group=64, dtype="bf16", scale="bf16",
             zeros=True),
        # a batch of 23 sequences, one token each, through the down projection,
        # one scale per row, no zero points
        dict(name="u4_batch_down", op="linear", rows=23, n=4096, k=14336, group=14336, dtype="fp16", scale="fp32",
             zeros=False),
        # a prompt through the down projection
        dict(name="u4_prompt_down", op="linear", rows=2048, n=4096, k=14336, group=128, dtype="bf16", scale="bf16",
             zeros=True),
        # the product and its gradient for a short odd batch, odd outputs
        dict(name="u4_grad_odd", op="linear_grad", rows=333, n=2047, k=1416, group=32, dtype="fp16", scale="fp16",
             zeros=True),
        # the product and its gradient in a training step through the gate
        dict(name="u4_grad_gate", op="linear_grad", rows=2048, n=14336, k=4096, group=128, dtype="bf16",
             scale="bf16", zeros=True),
        # scoring seven continuations by their next token, the 8B head
        dict(name="loss_score", op="vocab", rows=7, vocab=128256, hidden=4096, dtype="bf16", ignored=0.0,
             grad="none", reduction="none"),
        # a short odd batch over a middle-sized head, a third of the rows
        # ignored (prompts), both gradients, scaled loss
        dict(name="loss_odd", op="vocab", rows=517, vocab=32003, hidden=2056, dtype="fp16", ignored=0.33,
             grad="both", reduction="mean"),
        # a training step over the 8B head, both gradients
        dict(name="loss_train", op="vocab", rows=2048, vocab=128256, hidden=4096, dtype="bf16", ignored=0.1,
             grad="both", reduction="mean"),
        # a small student's short batch against 16 teacher logits, both gradients
        dict(name="distill_small", op="distill", rows=96, vocab=32000, hidden=1024, top=16, temperature=2.0,
             dtype="fp16", ignored=0.1, grad="both", reduction="mean"),
        # a frozen 8B head, the hidden states' gradient, 64 teacher logits
        dict(name="distill_train", op="distill", rows=1024, vocab=128256, hidden=4096, top=64, temperature=1.0,
             dtype="bf16", ignored=0.1, grad="x", reduction="mean"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "vocab", "distill"])
    dtype = rng.choice(["bf16", "fp16"])
    while True:
        if op in ("linear", "linear_grad"):
            k = 8 * _log_uniform(rng, 8, 2048)
            c = dict(op=op, rows=_log_uniform(rng, 1, 4096), n=_log_uniform(rng, 16, 53248), k=k,
                     group=rng.choice([32, 64, 128, k]), dtype=dtype,
                     scale=rng.choice([dtype, "fp32"]), zeros=rng.random() < 0.7)
            if c["group"] == k and k % 32:
                c["group"] = 32
        else:
            c = dict(op=op, rows=_log_uniform(rng, 1, 4096), vocab=_log_uniform(rng, 1000, 150000),
                     hidden=8 * _log_uniform(rng, 16, 1024), dtype=dtype, ignored=rng.choice([0.0, 0.1, 0.5]),
                     grad=rng.choice(["none", "x", "both"]), reduction=rng.choice(["none", "sum", "mean"]))
            if op == "distill":
                c.update(top=_log_uniform(rng, 1, 128), temperature=rng.choice([1.0, 2.0, 4.0]))
        w = work(c)
        if w["flops"] <= 6.0e12 and w["bytes"] <= 2.1e9:
            return c


# --------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = dict(case=case)
    if case["op"] in ("linear", "linear_grad"):
        n, k, grp = case["n"], case["k"], case["group"]
        # codes of normal weights with 16 levels: peaked round the middle
        q = torch.empty(n, k, dtype=torch.uint8, device=dev)
        for lo in range(0, n, 8192):
            q[lo: lo + 8192] = (torch.randn(min(8192, n - lo), k, generator=g, device=dev) * 2.3 + 7.5) \
                .round_().clamp_(0, 15).to(torch.uint8)
        st["packed"] = (q[:, 0::2] | (q[:, 1::2] << 4)).reshape(-1)
        ng = (k + grp - 1) // grp
        st["scales"] = ((0.5 + torch.rand(n, ng, generator=g, device=dev)) * 0.01).to(DTYPES[case["scale"]])
        st["zeros"] = torch.randint(6, 10, (n, ng), generator=g, device=dev, dtype=torch.uint8) \
            if case["zeros"] else None
        st["x"] = torch.randn(case["rows"], k, generator=g, device=dev).to(dt)
        if case["op"] == "linear_grad":
            st["dy"] = torch.randn(case["rows"], n, generator=g, device=dev).to(dt)
            st["x"].requires_grad_()
        if own:
            import lossless_entropy_coded_huffman_amd as dfh
            st["w"] = dfh.U4Matrix(st["packed"], st["scales"], st["zeros"], cols=k, group_size=grp)
        return st
    m, v, h = case["rows"], case["vocab"], case["hidden"]
    st["x"] = torch.randn(m, h, generator=g, device=dev).to(dt)
    st["head"] = (torch.randn(v, h, generator=g, device=dev) * (2.5 / math.sqrt(h))).to(dt)
    ignored = torch.rand(m, generator=g, device=dev) < case["ignored"]
    if case["op"] == "vocab":
        st["labels"] = torch.randint(0, v, (m,), generator=g, device=dev).masked_fill_(ignored, -100)
    else:
        vals, idx = [], []
        for lo in range(0, m, 256):
            a, i = (torch.randn(min(256, m - lo), v, generator=g, device=dev) * 2.5).topk(case["top"], dim=1)
            vals.append(a)
            idx.append(i)
        st["teacher"] = torch.cat(vals)
        st["index"] = torch.cat(idx).masked_fill_(ignored[:, None], -1)
    if case["grad"] != "none":
        st["x"].requires_grad_()
        if case["grad"] == "both":
            st["head"].requires_grad_()
        # the gradient that reaches the loss: float16 steps scale theirs so
        # that the head's gradient stays in range
        s = 1.0
        if case["dtype"] == "fp16":
            s = 64.0 * min(m, 64) if case["reduction"] == "mean" else 64.0
        st["gout"] = (torch.rand(m, generator=g, device=dev) + 0.5) * s if case["reduction"] == "none" \
            else torch.full((), s, device=dev)
    return st


# ----------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(case, state)


def _run_own(case, st):
    import lossless_entropy_coded_huffman_amd as dfh
    if case["op"] == "linear":
        return dfh.linear_u4(st["x"], st["w"])
    if case["op"] == "linear_grad":
        y = dfh.linear_u4(st["x"], st["w"])
        dx, = torch.autograd.grad(y, st["x"], st["dy"])
        return y.detach(), dx
    if case["op"] == "vocab":
        loss = dfh.vocab_loss(st["x"], st["head"], st["labels"], reduction=case["reduction"])
    else:
        loss = dfh.distill_loss(st["x"], st["head"], st["teacher"], st["index"],
                                temperature=case["temperature"], reduction=case["reduction"])
    if case["grad"] == "none":
        return loss
    leaves = [st["x"], st["head"]] if case["grad"] == "both" else [st["x"]]
    return (loss.detach(),) + torch.autograd.grad(loss, leaves, st["gout"])


@torch.no_grad()
def _run_plain(case, st):
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("linear", "linear_grad"):
        n, k, grp = case["n"], case["k"], case["group"]
        p = st["packed"].view(n, k // 2)
        q = torch.stack((p & 15, p >> 4), dim=-1).view(n, k).float()
        z = st["zeros"].float() if st["zeros"] is not None else torch.full_like(st["scales"], 8.0).float()
        s = st["scales"].float()
        if grp < k:
            s = s.repeat_interleave(grp, dim=1)[:, :k]
            z = z.repeat_interleave(grp, dim=1)[:, :k]
        w = (q - z) * s
        y = (st["x"].float() @ w.t()).to(dt)
        if case["op"] == "linear":
            return y
        return y, (st["dy"].float() @ w).to(dt)
    x, head = st["x"].float(), st["head"].float()
    z = x @ head.t()
    m = x.shape[0]
    if case["op"] == "vocab":
        temp = 1.0
        valid = st["labels"] != -100
        idx = st["labels"].clamp(min=0)[:, None]
        t = valid.float()[:, None]
        ent = torch.zeros(m, device=x.device)
    else:
        temp = case["temperature"]
        present = st["index"] >= 0
        valid = present.any(dim=1)
        idx = st["index"].clamp(min=0)
        a = (st["teacher"].float() / temp).masked_fill(~present, -math.inf)
        a = a - a.amax(dim=1, keepdim=True).masked_fill(~valid[:, None], 0.0)
        e = a.exp()
        total = e.sum(dim=1, keepdim=True).masked_fill(~valid[:, None], 1.0)
        t = e / total
        ent = torch.where(t > 0, t * (a - total.log()), torch.zeros_like(t)).sum(dim=1)
    z = z / temp
    top = z.amax(dim=1, keepdim=True)
    p = (z - top).exp()
    denom = p.sum(dim=1, keepdim=True)
    lse = top + denom.log()
    picked = z.gather(1, idx)
    loss = temp * temp * (ent + (t * (lse - picked)).sum(dim=1))
    loss = torch.where(valid, loss, torch.zeros_like(loss))
    count = valid.sum().clamp(min=1).float()
    out = loss if case["reduction"] == "none" else loss.sum() if case["reduction"] == "sum" else loss.sum() / count
    if case["grad"] == "none":
        return out
    gm = st["gout"].expand(m) if case["reduction"] != "mean" else (st["gout"] / count).expand(m)
    gm = torch.where(valid, gm, torch.zeros_like(gm)) * temp
    dz = p.div_(denom)
    dz.scatter_add_(1, idx, -t)
    dz.mul_(gm[:, None])
    dx = (dz @ head).to(dt)
    if case["grad"] == "x":
        return out, dx
    return out, dx, (dz.t() @ x).to(dt)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(dict(case), seed)
    if case["op"] in ("linear", "linear_grad"):
        # even and odd columns apart, group by group where there are several
        with torch.no_grad():
            n, k, grp = case["n"], case["k"], case["group"]
            p = st["packed"].view(n, k // 2)
            cols = torch.arange(k, device=p.device) // grp
            s = st["scales"].double()
            z = st["zeros"].double() if st["zeros"] is not None else torch.full_like(s, 8.0)
            y = 0
            dx = torch.empty(case["rows"], k, dtype=torch.float64, device=p.device)
            for half in (0, 1):
                part = (p >> (4 * half)) % 16
                c = cols[half::2]
                w = (part.double() - z[:, c]) * s[:, c]
                y = y + st["x"][:, half::2].double() @ w.t()
                if case["op"] == "linear_grad":
                    dx[:, half::2] = st["dy"].double() @ w
        return y if case["op"] == "linear" else (y, dx)
    x = st["x"].detach().double().requires_grad_()
    head = st["head"].detach().double().requires_grad_(case["grad"] == "both")
    if case["op"] == "vocab":
        rows = torch.nonzero(st["labels"] != -100)[:, 0]
        logq = torch.log_softmax(x[rows] @ head.t(), dim=1)
        per = -logq[torch.arange(rows.numel(), device=rows.device), st["labels"][rows]]
    else:
        temp = case["temperature"]
        rows = torch.nonzero((st["index"] >= 0).any(dim=1))[:, 0]
        there = st["index"][rows] >= 0
        logt = torch.log_softmax((st["teacher"][rows].double() / temp).masked_fill(~there, -math.inf), dim=1)
        logq = torch.log_softmax((x[rows] @ head.t()) / temp, dim=1)
        term = torch.where(there, logt.exp() * (logt - logq.gather(1, st["index"][rows].clamp(min=0))), 0.0)
        per = temp ** 2 * term.sum(dim=1)
    if case["reduction"] == "none":
        out = torch.zeros(case["rows"], dtype=torch.float64, device=x.device).index_copy(0, rows, per)
    else:
        out = per.sum() if case["reduction"] == "sum" else per.sum() / max(1, rows.numel())
    if case["grad"] == "none":
        return out.detach()
    leaves = [x, head] if case["grad"] == "both" else [x]
    return (out.detach(),) + torch.autograd.grad(out, leaves, st["gout"].double())


# ------------------------------------------------------------------------ work
def work(case):
    """Bytes and operations one pass cannot do without."""
    es = 2
    if case["op"] in ("linear", "linear_grad"):
        m, n, k = case["rows"], case["n"], case["k"]
        ng = (k + case["group"] - 1) // case["group"]
        w = n * k // 2 + n * ng * ((4 if case["scale"] == "fp32" else 2) + (1 if case["zeros"] else 0))
        both = 2 if case["op"] == "linear_grad" else 1
        return {"bytes": w + both * es * m * (k + n), "flops": both * 2 * m * n * k}
    m, v, h = case["rows"], case["vocab"], case["hidden"]
    grads = {"none": 0, "x": 1, "both": 2}[case["grad"]]
    b = es * (m + v) * h + 4 * m
    b += 8 * m if case["op"] == "vocab" else m * case["top"] * 12
    b += es * m * h if grads else 0
    b += es * v * h if grads == 2 else 0
    # the logits once, and one product for each gradient
    return {"bytes": b, "flops": 2 * m * v * h * (1 + grads)}
