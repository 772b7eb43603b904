"""Workloads of the operators that complete a decode step around the quantized paged cache.

    pages      pages handed to the new tokens of every sequence from their lengths, with the slots, positions and sequence
               of each new token, then taken back (a step whose proposed tokens are all rejected, or a finished request)
    rotary     queries and keys turned by their positions
    append     the same, with the turned keys and the values quantized into a paged cache, and those rows read back
    experts    a mixture-of-experts block on group-wise affine experts, from the router's logits to the block's output

`listed` names the cases, `draw` gives more of the same ranges, `prepare` makes the inputs, `run` makes one pass: in elementary
torch operations, or with the library's own operators where `own` is true.  `exact` evaluates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

# widths of the decoder layers whose linears the library is measured on
_WIDTHS = (1024, 2048, 4096, 8192)
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _pages(name, batch, max_len, new, page, padding):
    return {"name": name, "op": "pages", "batch": batch, "max_len": max_len, "new": new, "page": page, "padding": padding}


def _rotary(name, tokens, heads, kv_heads, head_dim, rotary_dim, interleaved, scaling, far, dtype):
    return {"name": name, "op": "rotary", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "rotary_dim": rotary_dim, "interleaved": interleaved, "scaling": scaling, "far": far, "dtype": dtype}


def _append(name, *a, group, bits, page):
    return {**_rotary(name, *a), "op": "append", "group": group, "bits": bits, "page": page}


def _experts(name, rows, width, inner, experts, top_k, group, bits, renormalize, logits, resid, dtype):
    return {"name": name, "op": "experts", "rows": rows, "width": width, "inner": inner, "experts": experts, "top_k": top_k,
            "group": group, "bits": bits, "renormalize": renormalize, "logits": logits, "resid": resid, "dtype": dtype}


def listed():
    return [
        # a decode step of 64 sequences with five proposed tokens each: the launch is the cost
        _pages("pages 64 sequences +5", 64, 8192, 5, 64, 0),
        # prompts of 32 requests arrive at once, in small pages, the batch's tail padded
        _pages("pages 32 sequences +2048", 32, 1000, 2048, 16, 100),
        # the new token of one sequence, heads of the 2048-wide layer
        _rotary("rotary 1 d64", 1, 32, 8, 64, 64, False, "none", 8192, "bf16"),
        # a small decode batch, half of each head turned, neighbours paired
        _rotary("rotary 16 d128 half interleaved", 16, 32, 8, 128, 64, True, "linear", 16384, "f16"),
        # a prompt of 8192 tokens in a context past a million: bound by memory
        _rotary("rotary 8192 d128 far", 8192, 32, 8, 128, 128, False, "bands", 1 << 20, "bf16"),
        # one decode step of 16 sequences, 4-bit rows
        _append("append 16 d128 4-bit", 16, 32, 8, 128, 128, False, "bands", 131072, "bf16", group=64, bits=4, page=16),
        # a prompt of 4096 tokens, 8-bit rows
        _append("append 4096 d128 8-bit", 4096, 32, 8, 128, 128, False, "base", 16384, "f16", group=64, bits=8, page=64),
        # one token and two experts of eight, the narrowest layer: latency
        _experts("experts 1x1024 2 of 8", 1, 1024, 2048, 8, 2, 64, 4, True, "f32", True, "bf16"),
        # one token, eight small experts of 64
        _experts("experts 1x2048 8 of 64", 1, 2048, 1024, 64, 8, 64, 4, True, "act", True, "bf16"),
        # a decode batch that reaches most experts, each with one or two tokens
        _experts("experts 16x2048 8 of 64", 16, 2048, 1024, 64, 8, 64, 4, True, "f32", True, "f16"),
        # a larger batch over many small experts: bound by memory
        _experts("experts 64x2048 8 of 128", 64, 2048, 768, 128, 8, 32, 4, False, "f32", False, "bf16"),
        # few wide experts in 8 bits
        _experts("experts 5x4096 2 of 8 8-bit", 5, 4096, 14336, 8, 2, 64, 8, True, "f32", True, "bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("pages", "rotary", "append", "experts", "experts", "experts"))
    dtype = rng.choice(("bf16", "f16"))
    if op == "pages":
        batch = _spread(rng, 1, 512)
        new = _spread(rng, 1, max(1, 65536 // batch))
        c = _pages("", batch, _spread(rng, 1, 8192), new, rng.choice((16, 32, 48, 64, 128)), rng.choice((0, 0, 7, 64)))
    elif op == "experts":
        experts, top_k = rng.choice(((8, 1), (8, 2), (16, 4), (32, 4), (60, 4), (64, 6), (64, 8), (128, 8), (256, 8)))
        group, bits = rng.choice((32, 64, 64, 128)), rng.choice((2, 4, 4, 4, 8))
        width = rng.choice(_WIDTHS) if rng.random() < 0.7 else 128 * rng.randint(2, 40)
        most = 8 * 4096 * 14336 // (experts * width)  # the inner width at which all experts are as large as the largest case's
        inner = 128 * max(1, _spread(rng, min(256, most), min(14336, most)) // 128)
        c = _experts("", _spread(rng, 1, 64), width, inner, experts, top_k, group, bits, rng.random() < 0.7,
                     rng.choice(("f32", "act")), rng.random() < 0.6, dtype)
    else:
        head_dim, group = rng.choice(((64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (256, 64)))
        kv_heads = rng.choice((1, 2, 4, 8))
        heads = kv_heads * rng.choice((1, 2, 4, 5, 8))
        rotary_dim = rng.choice((head_dim, head_dim, head_dim // 2, 32))
        tokens = _spread(rng, 1, 8192 * 40 * 128 // ((heads + 2 * kv_heads) * head_dim))
        a = ("", tokens, heads, kv_heads, head_dim, rotary_dim, rng.random() < 0.4,
             rng.choice(("none", "linear", "base", "bands")), _spread(rng, 16, 1 << 20), dtype)
        if op == "rotary":
            c = _rotary(*a)
        else:
            c = _append(*a, group=group, bits=rng.choice((2, 4, 4, 8)), page=rng.choice((16, 32, 48, 64, 128)))
    del c["name"]
    return c


def _lens(case):
    """Cached and new tokens of each sequence, the same for every seed: in a batch of eight or more one row is empty, one
    has nothing new and one has nothing at all."""
    n, most, new = case["batch"], case["max_len"], case["new"]
    r = random.Random(n * 1000003 + most)
    lens = [most] + [r.randint(0, most) for _ in range(n - 1)]
    news = [new if new < 16 else r.randint(1, new) for _ in range(n)]
    if n >= 8:
        lens[1] = lens[3] = news[2] = news[3] = 0
    return lens, news


def _active(case):
    """How many experts a batch of independent tokens is expected to reach."""
    e = case["experts"]
    return e * (1.0 - (1.0 - case["top_k"] / e) ** case["rows"])


def work(case):
    if case["op"] == "pages":
        lens, news = _lens(case)
        p = case["page"]
        pages = sum(-(-(n + m) // p) - -(-n // p) for n, m in zip(lens, news))
        # out: a slot, a position and a sequence a token, a length a sequence; pages off the list, into the table and back
        return {"bytes": 16 * (sum(news) + case["padding"]) + 5 * 4 * case["batch"] + 5 * 4 * pages, "flops": 0}
    if case["op"] == "experts":
        m, k, i = case["rows"], case["width"], case["inner"]
        weights = _active(case) * 3 * k * i
        rows = 2 * m * k * (3 if case["resid"] else 2) + (4 if case["logits"] == "f32" else 2) * m * case["experts"]
        return {"bytes": int(weights * (case["bits"] / 8 + 4 / case["group"])) + rows, "flops": 6 * m * case["top_k"] * k * i}
    t, d = case["tokens"], case["head_dim"]
    flops = 3 * t * (case["heads"] + case["kv_heads"]) * case["rotary_dim"]
    if case["op"] == "rotary":
        return {"bytes": 4 * t * (case["heads"] + case["kv_heads"]) * d + 4 * t + 4 * case["rotary_dim"], "flops": flops}
    row = d * case["bits"] // 8 + 4 * (d // case["group"])
    n = 2 * t * case["kv_heads"]
    # queries in and out; keys and values in, their rows out, and those read back into dense ones
    return {"bytes": 4 * t * case["heads"] * d + n * (2 * d + row) + n * (row + 2 * d) + 20 * t, "flops": flops + 10 * n * d}


_BASE, _ORIGINAL, _FACTOR, _LOW, _HIGH = 10000.0, 8192, 8.0, 1.0, 4.0


def _frequencies(case):
    """Radians a position of each pair, in 64 bits on the host."""
    r, kind = case["rotary_dim"], case["scaling"]
    base = _BASE * _FACTOR ** (r / (r - 2)) if kind == "base" else _BASE
    f = [base ** (-2.0 * j / r) for j in range(r // 2)]
    if kind == "linear":
        f = [x / _FACTOR for x in f]
    if kind == "bands":
        keep = [min(1.0, max(0.0, (_ORIGINAL * x / (2 * math.pi) - _LOW) / (_HIGH - _LOW))) for x in f]
        f = [x * (g + (1.0 - g) / _FACTOR) for x, g in zip(f, keep)]
    return f


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] == "pages":
        return _prepare_pages(case, gen)
    dt = _DTYPES[case["dtype"]]
    if case["op"] == "experts":
        m, k, i, e, g, bits = (case[n] for n in ("rows", "width", "inner", "experts", "group", "bits"))

        def weight(rows, cols):
            packed = torch.randint(-2**31, 2**31, (e, rows, cols * bits // 32), generator=gen, device="cuda",
                                   dtype=torch.int32)
            sigma = torch.empty((e, rows, cols // g), device="cuda").uniform_(0.5, 1.5, generator=gen).div_(math.sqrt(cols))
            scales = (sigma * (5.5 / (2**bits - 1))).to(dt)  # a normal group's range is about 5.5 of its deviations
            return packed, scales, (sigma * torch.empty_like(sigma).uniform_(-2.9, -2.6, generator=gen)).to(dt)

        st = {**case, "x": normal(m, k).to(dt), "logit": (1.5 * normal(m, e)).to(torch.float32 if case["logits"] == "f32" else dt),
              "r": normal(m, k).to(dt) if case["resid"] else None, "gate_up": weight(2 * i, k), "down": weight(k, i)}
        if own:
            import group_wise_affine_unpack_amd as qa
            st["weights"] = qa.AffineExperts(st["gate_up"], st["down"], g, bits)
        return st
    t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
    st = {**case, "freq": torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda"),
          "pos": torch.randint(0, case["far"], (t,), generator=gen, device="cuda", dtype=torch.int32)}
    channel = 1.0 + 3.0 * (torch.rand((hk, d), generator=gen, device="cuda") < 0.05)  # keys' few wide channels
    st["q"], st["key"], st["value"] = (1.5 * normal(t, h, d)).to(dt), (normal(t, hk, d) * channel).to(dt), normal(t, hk, d).to(dt)
    if case["op"] == "append":
        s, pages = case["page"], -(-t // case["page"]) + 2
        rows = (pages, hk, s)
        st["k"], st["v"] = ((torch.zeros((*rows, d * case["bits"] // 32), device="cuda", dtype=torch.int32),
                             torch.zeros((*rows, d // case["group"]), device="cuda", dtype=dt),
                             torch.zeros((*rows, d // case["group"]), device="cuda", dtype=dt)) for _ in range(2))
        at = torch.randperm(pages, generator=gen, device="cuda")[: -(-t // s)]  # whole pages, in any order
        st["slots"] = (at[:, None] * s + torch.arange(s, device="cuda")).reshape(-1)[:t].contiguous()
        if t >= 8:
            st["slots"][t - t // 8:] = -1  # the rows that fill a padded batch up
    if own:
        import group_wise_affine_unpack_amd as qa
        st["rot"] = qa.Rotary(st["freq"], interleaved=case["interleaved"])
        if case["op"] == "append":
            st["cache"] = qa.AffineKVCache(st["k"], st["v"], case["group"], case["bits"])
    return st


def _prepare_pages(case, gen):
    lens, news = _lens(case)
    n, p = case["batch"], case["page"]
    had = [-(-a // p) for a in lens]
    most = max(-(-(a + b) // p) for a, b in zip(lens, news))
    pages = sum(-(-(a + b) // p) for a, b in zip(lens, news)) + 5
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    mine = (torch.arange(most, device="cuda") < torch.tensor(had, device="cuda")[:, None])
    table = torch.full((n, most), -1, dtype=torch.int32, device="cuda")
    table[mine] = order[: sum(had)]
    free = torch.zeros(pages, dtype=torch.int32, device="cuda")
    free[: pages - sum(had)] = order[sum(had):]
    count = torch.tensor([pages - sum(had)], dtype=torch.int32, device="cuda")
    st = {**case, "table": table, "free": free, "count": count, "rows": sum(news) + case["padding"],
          "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
          "news": torch.tensor(news, dtype=torch.int32, device="cuda")}
    if own:
        import group_wise_affine_unpack_amd as qa
        st["pool"] = qa.KVPagePool(pages, p, device="cuda")
        st["pool"].free_pages.copy_(free)
        st["pool"].state[:1].copy_(count)
    return st


def run(st):
    return _own(st) if own else _PLAIN[st["op"]](st)


def _own(st):
    import group_wise_affine_unpack_amd as qa
    if st["op"] == "pages":
        pool = st["pool"]
        slots, positions, rows, lens = qa.kv_pages_assign(pool, st["table"], st["lens"], st["news"], st["rows"])
        kept = qa.kv_pages_trim(pool, st["table"], lens, st["lens"])
        return {"slots": slots, "positions": positions, "rows": rows, "lens": lens, "kept": kept, "table": st["table"],
                "free": pool.free_pages, "count": pool.state[:1]}
    if st["op"] == "rotary":
        return qa.rotary(st["q"], st["key"], st["pos"], st["rot"])
    if st["op"] == "append":
        q = qa.kv_cache_append_rotary_affine(st["cache"], st["q"], st["key"], st["value"], st["pos"], st["slots"], st["rot"])
        return (q, *qa.kv_cache_read_affine(st["cache"], st["slots"]))
    return qa.qmoe_affine(st["x"], st["logit"], st["weights"], st["top_k"], renormalize=st["renormalize"], resid=st["r"])


def _ceil_div(a, b):
    return torch.div(a + (b - 1), b, rounding_mode="floor")


def _plain_pages(st):
    p, lens, news, table, free = st["page"], st["lens"].long(), st["news"].long(), st["table"], st["free"]
    dev, count = lens.device, st["count"].long()
    ends, had = news.cumsum(0), _ceil_div(lens, p)
    need = _ceil_div(lens + news, p) - had
    first = need.cumsum(0) - need  # of each sequence's pages among all that are handed out
    # the table with the pages handed out: entry j of a sequence is page first + j - had of the list, from its end
    j = torch.arange(table.shape[1], device=dev)
    fresh = (j >= had[:, None]) & (j < (had + need)[:, None])
    at = (count - 1 - (first[:, None] + j - had[:, None])).clamp(0, free.shape[0] - 1)
    full = torch.where(fresh, free[at], table)
    # a row a new token
    r = torch.arange(st["rows"], device=dev)
    seq = (r[:, None] >= ends[None, :]).sum(1)
    there = seq < lens.shape[0]
    b = seq.clamp(max=lens.shape[0] - 1)
    pos = lens[b] + r - (ends - news)[b]
    entry = torch.div(pos, p, rounding_mode="floor").clamp(0, table.shape[1] - 1)
    slots = torch.where(there, full[b, entry].long() * p + pos % p, -1)
    # taken back: entries go, and the list ends with the same pages
    total = need.sum()
    back = torch.where(fresh, -1, full)
    k = torch.where(fresh, at, free.shape[0])
    again = torch.cat([torch.where(torch.arange(free.shape[0], device=dev) < count - total, free, 0), free[:1]])
    again = again.scatter(0, k.flatten(), full.flatten())[:-1]
    return {"slots": slots, "positions": torch.where(there, pos, 0).int(), "rows": torch.where(there, seq, -1).int(),
            "lens": (lens + news).int(), "kept": torch.minimum(lens + news, lens).int(), "table": back,
            "free": torch.where(torch.arange(free.shape[0], device=dev) < count, again, free),
            "count": (count - total + total).int()}


def _plain_turn(x, pos, freq, interleaved):
    """Rows of x turned, in 64 bits (the angles of far positions, and keys next to a border of their rounding)."""
    half = freq.shape[0]
    angle = pos.double()[:, None, None] * freq
    c, s = angle.cos(), angle.sin()
    y = x.double()
    a, b = (y[..., 0 : 2 * half : 2], y[..., 1 : 2 * half : 2]) if interleaved else (y[..., :half], y[..., half : 2 * half])
    ta, tb = a * c - b * s, b * c + a * s
    turned = torch.stack([ta, tb], -1).flatten(-2) if interleaved else torch.cat([ta, tb], -1)
    return torch.cat([turned, y[..., 2 * half :]], -1).to(x.dtype)


def _plain_rotary(st):
    return tuple(_plain_turn(st[n], st["pos"], st["freq"], st["interleaved"]) for n in ("q", "key"))


def _plain_values(packed, scales, biases, bits):
    """fp32 values of packed rows: code * scale + bias, group by group."""
    shifts = torch.arange(0, 32, bits, device=packed.device, dtype=torch.int32)
    codes = ((packed.unsqueeze(-1) >> shifts) & (2**bits - 1)).flatten(-2).unflatten(-1, (scales.shape[-1], -1))
    return (codes.float() * scales.float().unsqueeze(-1) + biases.float().unsqueeze(-1)).flatten(-2)


def _plain_append(st):
    bits, g, s, most = st["bits"], st["group"], st["page"], float(2 ** st["bits"] - 1)
    q, key = _plain_rotary(st)
    ok = st["slots"] >= 0
    at = st["slots"].clamp(min=0)
    rows = ((at // s)[:, None], torch.arange(st["kv_heads"], device=at.device)[None], (at % s)[:, None])
    outs = []
    for triple, x in ((st["k"], key), (st["v"], st["value"])):
        x = x.float().unflatten(-1, (-1, g))
        lo, hi = x.amin(-1), x.amax(-1)
        new = [((hi - lo) / torch.full_like(hi, most)).to(q.dtype), lo.to(q.dtype)]
        sc, bi = (t.float().unsqueeze(-1) for t in new)
        codes = torch.where(sc != 0, torch.round((x - bi) / sc), 0.0).clamp(0, most).flatten(-2).to(torch.int64)
        words = (codes.unflatten(-1, (-1, 32 // bits)) << torch.arange(0, 32, bits, device=at.device)).sum(-1)
        new.insert(0, torch.where(words >= 2**31, words - 2**32, words).to(torch.int32))
        kept = ok.nonzero()[:, 0]
        where = (rows[0][kept], rows[1], rows[2][kept])
        for store, value in zip(triple, new):
            store[where] = value[kept]
        dense = _plain_values(*(t[rows] for t in triple), bits)
        outs.append(torch.where(ok[:, None, None], dense, 0.0).to(q.dtype))
    return (q, *outs)


def _plain_route(st):
    """The chosen experts of each row, the largest logit first and ties to the lowest index, and their weights."""
    z = st["logit"].float()
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, : st["top_k"]]
    e = torch.exp(z - z.amax(-1, keepdim=True))
    chosen = e.gather(1, order)
    return order, chosen / (chosen if st["renormalize"] else e).sum(-1, keepdim=True)


def _plain_experts(st):
    bits, x, k = st["bits"], st["x"].float(), st["top_k"]
    order, weight = _plain_route(st)
    y = st["r"].float() if st["resid"] else torch.zeros_like(x)

    def product(rows, triple, index):  # [..., rows, in] times the transposed weights of the experts `index`
        w = _plain_values(*(t[index] for t in triple), bits)
        return rows @ w.transpose(-1, -2)

    def block(rows, index):
        g, u = product(rows, st["gate_up"], index).chunk(2, -1)
        return product(g / (1.0 + torch.exp(-g)) * u, st["down"], index)

    if st["rows"] * k < st["experts"]:  # the chosen experts of each row, side by side
        parts = [(block(x[m].expand(k, 1, -1), order[m])[:, 0] * weight[m][:, None]).sum(0) for m in range(st["rows"])]
        return (y + torch.stack(parts)).to(st["x"].dtype)
    dense = torch.zeros((st["rows"], st["experts"]), device=x.device).scatter(1, order, weight)
    for e in range(st["experts"]):  # every row through every expert, weighted by zero where it was not chosen
        y = y + block(x, e) * dense[:, e : e + 1]
    return y.to(st["x"].dtype)


_PLAIN = {"pages": _plain_pages, "rotary": _plain_rotary, "append": _plain_append, "experts": _plain_experts}


def _exact_codes(packed, bits):
    """Codes of packed rows, lowest bits first, from their bytes."""
    b = packed.contiguous().view(torch.uint8)
    parts = [(b >> i) & (2**bits - 1) for i in range(0, 8, bits)]
    return torch.stack(parts, -1).flatten(-2).double()


def _exact_matrix(triple, e, bits, g):
    scale, bias = (t[e].double().repeat_interleave(g, -1) for t in triple[1:])
    return _exact_codes(triple[0][e], bits) * scale + bias


def _exact_pages(case, st):
    """The definition, sequence by sequence and token by token on the host."""
    lens, news = st["lens"].tolist(), st["news"].tolist()
    table, free, n, p = st["table"].tolist(), st["free"].tolist(), int(st["count"]), case["page"]
    slots, positions, rows = [], [], []
    for b, (a, m) in enumerate(zip(lens, news)):
        for i in range(a, a + m):
            if i % p == 0:
                n -= 1
                table[b][i // p] = free[n]
            slots.append(table[b][i // p] * p + i % p)
            positions.append(i)
            rows.append(b)
    pad = st["rows"] - len(slots)

    def whole(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device="cuda")

    return {"slots": whole(slots + [-1] * pad, torch.int64), "positions": whole(positions + [0] * pad),
            "rows": whole(rows + [-1] * pad), "lens": whole([a + m for a, m in zip(lens, news)]), "kept": st["lens"],
            "table": st["table"], "free": st["free"], "count": st["count"]}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "pages":
        return _exact_pages(case, st)
    if case["op"] == "experts":
        x, z = st["x"].double(), st["logit"].double()
        y = st["r"].double() if case["resid"] else torch.zeros_like(x)
        k, i = case["top_k"], case["inner"]
        chosen = []
        for row in z.tolist():  # ties to the lowest index
            best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
            total = sum(math.exp(row[e] - row[best[0]]) for e in (best if case["renormalize"] else range(len(row))))
            chosen.append({e: math.exp(row[e] - row[best[0]]) / total for e in best})
        for e in range(case["experts"]):
            rows = [m for m in range(case["rows"]) if e in chosen[m]]
            if not rows:
                continue
            w = _exact_matrix(st["gate_up"], e, case["bits"], case["group"])
            a = x[rows] @ w.T
            h = a[:, :i] * torch.sigmoid(a[:, :i]) * a[:, i:]
            w = _exact_matrix(st["down"], e, case["bits"], case["group"])
            p = torch.tensor([chosen[m][e] for m in rows], dtype=torch.float64, device="cuda")
            y[rows] += (h @ w.T) * p[:, None]
            del w
        return y
    angle = st["pos"].double()[:, None] * st["freq"]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]  # complex
    out = {}
    for name in ("q", "key"):
        v = st[name].double()
        r = case["rotary_dim"]
        part = v[..., :r].unflatten(-1, (-1, 2)) if case["interleaved"] else v[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
        v[..., :r] = turned.flatten(-2) if case["interleaved"] else turned.transpose(-1, -2).flatten(-2)
        out[name] = v
    if case["op"] == "rotary":
        return out["q"], out["key"]
    dt, bits, g = st["q"].dtype, case["bits"], case["group"]
    kept = (st["slots"] >= 0)[:, None, None]
    rows = []
    for v in (out["key"].to(dt), st["value"]):  # what is stored is the quantized row of the key as it was rounded
        v = v.double().unflatten(-1, (-1, g))
        bias = v.min(-1, keepdim=True).values
        scale = ((v.max(-1, keepdim=True).values - bias) / (2**bits - 1)).to(dt).double()
        codes = ((v - bias) / torch.where(scale > 0, scale, 1.0)).round().clamp(0, 2**bits - 1)
        rows.append((codes * scale + bias).flatten(-2) * kept)
    return (out["q"], *rows)
