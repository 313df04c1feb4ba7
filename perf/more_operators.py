"""What the operators of serving from quantised storage cost: the cases, their
inputs and the plain forms.

The operators:

* ``linear_u8``: products in 8-bit integers: the codes that a uint8 container
  decodes to, a scale and zero point for each output channel, and rows of
  activations that are quantised with a scale for each token;
* ``cache_write`` and ``cache_read``: new keys and values into the pages of a
  cache, kept in 16 bits or quantised to 8 with a scale for each token and head,
  and back;
* ``cached_attention``: attention of the new tokens of several sequences over
  that cache.

``own`` False runs each in its plain form (elementary torch operations in
float32, rounded once at the end), True through the package's calls.
``exact`` gives the same outputs from the definitions in float64.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one token through the k or v projection of an 8B-shaped block: the
        # smallest product, where latency counts
        dict(name="u8_token_kv", op="linear", rows=1, n=1024, k=4096, dtype="bf16", scale="fp32", zeros=True),
        # one token through the gate projection of a 405B-shaped block, symmetric
        # codes
        dict(name="u8_token_405b", op="linear", rows=1, n=53248, k=16384, dtype="bf16", scale="bf16", zeros=False),
        # a batch of 23 sequences, one token each, through the down projection of
        # the 8B-shaped block
        dict(name="u8_batch_down", op="linear", rows=23, n=4096, k=14336, dtype="fp16", scale="fp32", zeros=True),
        # a short odd batch, odd outputs
        dict(name="u8_odd", op="linear", rows=333, n=2047, k=1424, dtype="fp16", scale="fp16", zeros=True),
        # a prompt through the gate projection of the 8B-shaped block
        dict(name="u8_prompt_gate", op="linear", rows=2048, n=14336, k=4096, dtype="bf16", scale="fp32", zeros=True),
        # a token of each of five sequences, into 8 bits: the smallest write
        dict(name="write_step", op="write", seqs=5, new_from=1, new_to=1, past_from=10, past_to=3000,
             kv_heads=8, head_dim=128, page=64, dtype="bf16", bits=8, layout=1),
        # eight prompts at once, into 8 bits
        dict(name="write_prompts", op="write", seqs=8, new_from=700, new_to=5000, past_from=0, past_to=0,
             kv_heads=8, head_dim=128, page=64, dtype="bf16", bits=8, layout=2),
        # sequences of a small model read back whole, small pages
        dict(name="read_sequences", op="read", seqs=13, new_from=300, new_to=20000, past_from=0, past_to=0,
             kv_heads=4, head_dim=64, page=16, dtype="fp16", bits=8, layout=3),
        # a token of one sequence over 16 bits: the smallest attention
        dict(name="attend_token", op="attend", seqs=1, new_from=1, new_to=1, past_from=1999, past_to=1999,
             heads=32, kv_heads=8, head_dim=128, page=64, dtype="bf16", bits=16, window=0, layout=4),
        # a decoding batch of 48 sequences between 300 and 30000 tokens, 8 bits
        dict(name="attend_batch", op="attend", seqs=48, new_from=1, new_to=1, past_from=300, past_to=30000,
             heads=32, kv_heads=8, head_dim=128, page=64, dtype="bf16", bits=8, window=0, layout=5),
        # prompts and decoding sequences of a small model together, some with no
        # new token, seven heads to a key head, a sliding window, 8 bits
        dict(name="attend_mixed", op="attend", seqs=19, new_from=0, new_to=700, past_from=0, past_to=2500,
             heads=14, kv_heads=2, head_dim=64, page=16, dtype="fp16", bits=8, window=1000, layout=6),
        # the last chunk of a long prompt over 16 bits
        dict(name="attend_prompt", op="attend", seqs=1, new_from=4096, new_to=4096, past_from=12288, past_to=12288,
             heads=32, kv_heads=8, head_dim=128, page=128, dtype="bf16", bits=16, window=0, layout=7),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "write", "read", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "fp16"])
    while True:
        if op == "linear":
            c = dict(op=op, rows=_log_uniform(rng, 1, 4096), n=_log_uniform(rng, 16, 53248),
                     k=16 * _log_uniform(rng, 4, 1024), dtype=dtype, scale=rng.choice([dtype, "fp32"]),
                     zeros=rng.random() < 0.7)
        else:
            kv = rng.choice([1, 2, 4, 8])
            c = dict(op=op, seqs=_log_uniform(rng, 1, 64), kv_heads=kv, head_dim=rng.choice([64, 128, 128, 256]),
                     page=rng.choice([16, 32, 64, 128]), dtype=dtype, bits=rng.choice([8, 8, 16]),
                     layout=rng.randrange(1 << 30))
            a, b = _log_uniform(rng, 1, 30000), _log_uniform(rng, 1, 30000)
            c["past_from"], c["past_to"] = min(a, b), max(a, b)
            most = _log_uniform(rng, 1, 4096)
            c["new_from"], c["new_to"] = (1, 1) if rng.random() < 0.4 else (rng.choice([0, 1, most]), most)
            if op != "attend":
                c["new_to"] = _log_uniform(rng, c["new_to"], 8192)
            else:
                c.update(heads=kv * rng.choice([1, 2, 3, 4, 7, 8, 16]),
                         window=rng.choice([0, 0, _log_uniform(rng, 16, 8192)]))
            if sum(lay(c)[0]) == 0:
                continue
        w = work(c)
        if w["flops"] <= 1.8e12 and w["bytes"] <= 9e8 and _padded(c) <= 2.2e9:
            return c


def lay(case):
    """New tokens and whole lengths of a case's sequences, spread over the
    logarithm."""
    rng = random.Random(case["layout"])
    def between(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))) - 0.5) if hi > lo else lo
    new = [between(case["new_from"], case["new_to"]) for _ in range(case["seqs"])]
    return new, [t + between(case["past_from"], case["past_to"]) for t in new]


def _padded(case):
    """The elements of the plain form's largest tensor."""
    if case["op"] != "attend":
        return 0
    new, length = lay(case)
    return max(len(new) * max(new) * case["heads"] * max(length),
               len(new) * max(length) * case["kv_heads"] * case["head_dim"])


# --------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = dict(case=case)
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        # codes of normal weights with 256 levels: peaked round the middle
        q = torch.empty(n, k, dtype=torch.uint8, device=dev)
        for lo in range(0, n, 8192):
            q[lo: lo + 8192] = (torch.randn(min(8192, n - lo), k, generator=g, device=dev) * 32 + 127.5) \
                .round_().clamp_(0, 255).to(torch.uint8)
        st["q"] = q
        st["scales"] = ((0.5 + torch.rand(n, generator=g, device=dev)) * 6e-4).to(DTYPES[case["scale"]])
        st["zeros"] = torch.randint(110, 145, (n,), generator=g, device=dev, dtype=torch.uint8) \
            if case["zeros"] else None
        # tokens of different size, a few channels far out
        x = torch.randn(case["rows"], k, generator=g, device=dev)
        x *= 0.5 + torch.rand(case["rows"], 1, generator=g, device=dev)
        x *= 1 + 15 * (torch.rand(k, generator=g, device=dev) < 0.005)
        st["x"] = x.to(dt)
        if own:
            import lossless_entropy_coded_huffman_amd as dfh
            st["w"] = dfh.U8Matrix(q, st["scales"], st["zeros"], cols=k)
        return st
    new, length = lay(case)
    seqs, page, kv, hd = case["seqs"], case["page"], case["kv_heads"], case["head_dim"]
    width = (max(length) + page - 1) // page + 1
    used = [(t + page - 1) // page for t in length]
    pages = sum(used) + 3
    # every sequence's pages lie anywhere in the pool
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    tables = torch.zeros(seqs, width, dtype=torch.int32, device=dev)
    at = 0
    for s, c in enumerate(used):
        tables[s, :c] = order[at: at + c]
        at += c
    starts = [0]
    for t in new:
        starts.append(starts[-1] + t)
    st["tables"] = tables
    st["lengths"] = torch.tensor(length, dtype=torch.int32, device=dev)
    st["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    st["tokens"] = starts[-1]
    st["most_new"], st["most"] = max(new), max(length)
    shape = (pages, kv, page, hd)
    names = ("k", "v", "k_scales", "v_scales") if case["bits"] == 8 else ("k", "v")
    if case["op"] == "write":
        for name in names:
            st[name] = torch.zeros(shape if len(name) == 1 else shape[:3], device=dev,
                                   dtype=torch.float32 if len(name) > 1 else torch.int8 if case["bits"] == 8 else dt)
    elif case["bits"] == 8:
        for name in ("k", "v"):
            st[name] = (torch.randn(shape, generator=g, device=dev) * 45).round_().clamp_(-127, 127).to(torch.int8)
            st[name + "_scales"] = (0.5 + torch.rand(shape[:3], generator=g, device=dev)) * 0.02
    else:
        st["k"], st["v"] = (torch.randn(shape, generator=g, device=dev).to(dt) for _ in range(2))
    if own:
        import lossless_entropy_coded_huffman_amd as dfh
        st["cache"] = dfh.KVCache(pages, kv, hd, page_size=page, dtype=dt, bits=case["bits"], device=dev)
        for name in names:
            getattr(st["cache"], name).copy_(st.pop(name))
        st["batch"] = dfh.CacheBatch(tables, st["lengths"], st["starts"], max_new=max(new))
    if case["op"] == "write":
        st["new_k"], st["new_v"] = (torch.randn(st["tokens"], kv, hd, generator=g, device=dev).to(dt)
                                    for _ in range(2))
    if case["op"] == "attend":
        st["q"] = torch.randn(st["tokens"], case["heads"], hd, generator=g, device=dev).to(dt)
    return st


# ----------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(case, state)


def _run_own(case, st):
    import lossless_entropy_coded_huffman_amd as dfh
    if case["op"] == "linear":
        return dfh.linear_u8(st["x"], st["w"])
    if case["op"] == "write":
        c = st["cache"]
        dfh.cache_write(st["new_k"], st["new_v"], c, st["batch"])
        return (c.k, c.v, c.k_scales, c.v_scales) if case["bits"] == 8 else (c.k, c.v)
    if case["op"] == "read":
        return dfh.cache_read(st["cache"], st["batch"], st["tokens"])
    return dfh.cached_attention(st["q"], st["cache"], st["batch"], window=case["window"] or None)


def _quantised(x):
    """Codes of rows in 127 steps to either side of zero, and the rows' scales."""
    top = x.double().abs().amax(dim=-1, keepdim=True)
    codes = (x.double() * 127 / top.masked_fill(top == 0, 1.0)).round()
    return codes.to(torch.int8), (top / 127).float().squeeze(-1)


def _places(st, page):
    """Page and row of every new token."""
    t = torch.arange(st["tokens"], dtype=torch.int32, device=st["starts"].device)
    s = torch.searchsorted(st["starts"], t, right=True) - 1
    pos = st["lengths"][s] - st["starts"][s + 1] + t
    return st["tables"][s, pos // page].long(), pos % page


@torch.no_grad()
def _run_plain(case, st):
    dt = DTYPES[case["dtype"]]
    if case["op"] == "linear":
        codes, xs = _quantised(st["x"])
        q = st["q"].float()
        q -= 128.0 if st["zeros"] is None else st["zeros"].float()[:, None]
        y = codes.float() @ q.t()
        return (y * xs[:, None] * st["scales"].float()).to(dt)
    if case["op"] == "write":
        at, row = _places(st, case["page"])
        names = []
        for name in ("k", "v"):
            names.append(name)
            new = st["new_" + name]
            if case["bits"] == 8:
                new, scales = _quantised(new)
                st[name + "_scales"][at, :, row] = scales
            st[name][at, :, row] = new
        if case["bits"] == 8:
            names += ["k_scales", "v_scales"]
        return tuple(st[name] for name in names)
    if case["op"] == "read":
        at, row = _places(st, case["page"])
        out = []
        for name in ("k", "v"):
            t = st[name][at, :, row]
            if case["bits"] == 8:
                t = (t.float() * st[name + "_scales"][at, :, row][..., None]).to(dt)
            out.append(t)
        return tuple(out)
    # attention: keys, values and new tokens padded to the longest
    seqs, heads, kv, hd, page = case["seqs"], case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    dev = st["q"].device
    most = (st["most"] + page - 1) // page * page
    tables = st["tables"][:, : most // page].long()
    def gather(name):
        t = st[name][tables].float()                                  # [seqs, pages, kv, page, hd]
        if case["bits"] == 8:
            t *= st[name + "_scales"][tables][..., None]
        return t.transpose(1, 2).reshape(seqs, kv, most, hd)
    n = st["most_new"]
    i = torch.arange(n, device=dev)
    new = st["starts"][1:] - st["starts"][:-1]
    there = i[None] < new[:, None]                                     # [seqs, n]
    flat = (st["starts"][:-1, None] + i[None]).clamp(max=st["tokens"] - 1)
    rep = heads // kv
    q = st["q"][flat].float().reshape(seqs, n, kv, rep, hd).permute(0, 2, 3, 1, 4).reshape(seqs, kv, rep * n, hd)
    z = (q @ gather("k").transpose(2, 3).contiguous()).view(seqs, kv, rep, n, most)
    z *= 1.0 / math.sqrt(hd)
    pos = (st["lengths"] - new)[:, None] + i[None]                     # [seqs, n]
    j = torch.arange(most, device=dev)
    hidden = j[None, None] > pos[:, :, None]
    if case["window"]:
        hidden |= j[None, None] <= pos[:, :, None] - case["window"]
    z.masked_fill_(hidden[:, None, None], -math.inf)
    z -= z.amax(dim=-1, keepdim=True)
    p = z.exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = (p.view(seqs, kv, rep * n, most) @ gather("v")).view(seqs, kv, rep, n, hd) / total
    out = torch.empty_like(st["q"])
    out[flat[there]] = o.permute(0, 3, 1, 2, 4).reshape(seqs, n, heads, hd)[there].to(dt)
    return out


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(dict(case), seed)
    if case["op"] == "linear":
        # rows as multiples of a 127th of their largest value
        x = st["x"].double()
        top = x.abs().max(dim=1, keepdim=True).values.clamp(min=1e-300)
        z = st["zeros"].double()[:, None] if st["zeros"] is not None else 128.0
        w = (st["q"].double() - z) * st["scales"].double()[:, None]
        return (torch.round(127 * x / top) * (top / 127)) @ w.t()
    new, length = lay(case)
    page, hd = case["page"], case["head_dim"]
    if own:
        for name in ("k", "v", "k_scales", "v_scales"):
            if case["bits"] == 8 or len(name) == 1:
                st[name] = getattr(st["cache"], name)
    if case["op"] == "write":
        out = {name: st[name].double() if "_" in name or case["bits"] == 16 else st[name].clone()
               for name in ("k", "v", "k_scales", "v_scales") if name in st}
        begin = 0
        for s, (t, whole) in enumerate(zip(new, length)):
            where = torch.arange(whole - t, whole, device=st["tables"].device)
            at = st["tables"][s].long()[torch.div(where, page, rounding_mode="floor")]
            for name in ("k", "v"):
                x = st["new_" + name][begin: begin + t].double()
                if case["bits"] == 8:
                    top = x.abs().max(dim=2).values
                    out[name + "_scales"][at, :, where % page] = top / 127
                    x = torch.round(127 * x / top.clamp(min=1e-300)[:, :, None]).to(torch.int8)
                out[name][at, :, where % page] = x
            begin += t
        return tuple(out.values())
    def whole_of(name, s, lo, hi):
        where = torch.arange(lo, hi, device=st["tables"].device)
        at = st["tables"][s].long()[torch.div(where, page, rounding_mode="floor")]
        t = st[name][at, :, where % page].double()
        return t * st[name + "_scales"][at, :, where % page].double()[:, :, None] if case["bits"] == 8 else t
    if case["op"] == "read":
        return tuple(torch.cat([whole_of(name, s, b - t, b) for s, (t, b) in enumerate(zip(new, length))])
                     for name in ("k", "v"))
    out, begin, rep = [], 0, case["heads"] // case["kv_heads"]
    for s, (t, whole) in enumerate(zip(new, length)):
        if t == 0:
            continue
        k, v = whole_of("k", s, 0, whole), whole_of("v", s, 0, whole)
        q = st["q"][begin: begin + t].double()
        begin += t
        pos = torch.arange(whole - t, whole, device=q.device)[:, None]
        j = torch.arange(whole, device=q.device)[None]
        seen = (j <= pos) & (pos - j < (case["window"] or whole + 1))
        each = []
        for h in range(case["heads"]):
            a = (q[:, h] @ k[:, h // rep].t()) / hd ** 0.5
            each.append(torch.softmax(a.where(seen, torch.full_like(a, -math.inf)), dim=1) @ v[:, h // rep])
        out.append(torch.stack(each, dim=1))
    return torch.cat(out)


# ------------------------------------------------------------------------ work
def work(case):
    """Bytes and operations one pass cannot do without."""
    if case["op"] == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        w = n * k + n * ((4 if case["scale"] == "fp32" else 2) + (1 if case["zeros"] else 0))
        return {"bytes": w + 2 * m * (k + n), "flops": 2 * m * n * k}
    new, length = lay(case)
    kv, hd = case["kv_heads"], case["head_dim"]
    # a token's key and value in the cache
    kept = 2 * kv * (hd + 4 if case["bits"] == 8 else 2 * hd)
    if case["op"] != "attend":
        return {"bytes": sum(new) * (kept + 4 * kv * hd) + 8 * case["seqs"] + 4, "flops": 4 * sum(new) * kv * hd}
    window = case["window"] or 1 << 30
    read = sum(min(b, t + window - 1) for t, b in zip(new, length) if t)
    # keys that a sequence's new tokens see: 1, 2, .. of them up to the window
    def upto(p):
        return p * (p + 1) // 2 if p <= window else window * (window + 1) // 2 + (p - window) * window
    seen = sum(upto(b) - upto(b - t) for t, b in zip(new, length))
    return {"bytes": read * kept + 4 * sum(new) * case["heads"] * hd, "flops": 4 * seen * case["heads"] * hd}
