"""Workloads of the operators that run between the quantized linears of a decoder layer.

    norm       root-mean-square norm with the residual's addition, into the activation type or into int8 codes with one
               scale a token (the activations of the W4A8 product)
    append     keys and values quantized as they are written into a paged cache (codes, scales and biases of the affine
               layout), then read back
    read       rows of such a cache dequantized
    attention  one new token a sequence attending to such a cache through its page table

`listed` names the cases, `draw` gives more of the same ranges, `prepare` makes the inputs, `run` makes one pass: in elementary
torch operations, or with the library's own operators where `own` is true.  `exact` evaluates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

# widths of the decoder layers whose linears the library is measured on
_WIDTHS = (1024, 2048, 4096, 8192, 14336)
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_EPS = 1e-5


def _norm(name, rows, width, dtype, to, resid=True):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "dtype": dtype, "to": to, "resid": resid}


def _append(name, tokens, kv_heads, head_dim, group, bits, page, dtype):
    return {"name": name, "op": "append", "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim, "group": group,
            "bits": bits, "page": page, "dtype": dtype}


def _read(name, *a):
    return {**_append(name, *a), "op": "read"}


def _attn(name, batch, max_len, ragged, heads, kv_heads, head_dim, group, bits, page, window, dtype):
    return {"name": name, "op": "attention", "batch": batch, "max_len": max_len, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "group": group, "bits": bits, "page": page, "window": window,
            "dtype": dtype}


def listed():
    return [
        # one token of one sequence, 2048 wide: the launch is the cost
        _norm("norm 1x2048 codes", 1, 2048, "f16", "codes"),
        # a small decode batch whose linears take 16-bit activations
        _norm("norm 16x4096 dense", 16, 4096, "bf16", "dense"),
        # a prompt of 2048 tokens ahead of a W4A8 product: bound by memory
        _norm("norm 2048x4096 codes", 2048, 4096, "f16", "codes"),
        # one decode step of 16 sequences, heads of the 2048-wide layer
        _append("append 16 d64 4-bit", 16, 8, 64, 64, 4, 16, "bf16"),
        # a prompt of 8192 tokens, heads of the 4096-wide layer
        _append("append 8192 d128 8-bit", 8192, 8, 128, 64, 8, 64, "f16"),
        # a short context read back, for a kernel that takes dense keys
        _read("read 1000 d128 4-bit", 1000, 8, 128, 64, 4, 16, "bf16"),
        # a long context read back
        _read("read 65536 d128 4-bit", 65536, 8, 128, 32, 4, 64, "f16"),
        # one sequence, a short context: the smallest call
        _attn("attn 1x517 d64 4-bit", 1, 517, False, 32, 8, 64, 64, 4, 16, 0, "bf16"),
        # a ragged decode batch, one of whose rows is empty
        _attn("attn 16x4096 d128 4-bit", 16, 4096, True, 32, 8, 128, 64, 4, 16, 0, "bf16"),
        # the cache of a large batch: bound by memory
        _attn("attn 64x8192 d128 8-bit", 64, 8192, True, 32, 8, 128, 64, 8, 64, 0, "f16"),
        # one long context, split over the whole chip
        _attn("attn 1x131072 d128 4-bit", 1, 131072, False, 32, 8, 128, 64, 4, 64, 0, "bf16"),
        # wide heads, twelve of them to a key head, the last 1024 tokens only
        _attn("attn 8x3000 d256 window", 8, 3000, True, 24, 2, 256, 128, 4, 32, 1024, "bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "append", "read", "attention", "attention", "attention"))
    dtype = rng.choice(("bf16", "f16"))
    if op == "norm":
        width = rng.choice(_WIDTHS) if rng.random() < 0.7 else _spread(rng, 256, 16384)
        rows = _spread(rng, 1, max(1, min(4096, 2048 * 4096 // width)))
        c = _norm("", rows, width, dtype, rng.choice(("codes", "dense")), rng.random() < 0.7)
    else:
        head_dim, group = rng.choice(((64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (256, 64),
                                      (256, 128)))
        bits, page = rng.choice((4, 4, 8)), rng.choice((16, 32, 48, 64, 128))
        kv_heads = rng.choice((1, 2, 4, 8, 12))
        if op == "append":
            c = _append("", _spread(rng, 1, 8192 * 8 * 128 // (kv_heads * head_dim)), kv_heads, head_dim, group, bits, page,
                        dtype)
        elif op == "read":
            c = _read("", _spread(rng, 1, 65536 * 8 * 128 // (kv_heads * head_dim)), kv_heads, head_dim, group, bits, page,
                      dtype)
        else:
            most = 64 * 4096 * 8 * 128 // (kv_heads * head_dim)  # tokens of all sequences
            batch = _spread(rng, 1, 64)
            max_len = _spread(rng, 1, min(131072, most // batch))
            heads = kv_heads * rng.choice((1, 2, 3, 4, 5, 8, 16, 20))
            window = _spread(rng, 1, max_len) if rng.random() < 0.25 else 0
            c = _attn("", batch, max_len, rng.random() < 0.7, heads, kv_heads, head_dim, group, bits, page, window, dtype)
    del c["name"]
    return c


def _lens(case):
    """The sequences' lengths, the same multiset for every seed: up to max_len, and in a ragged batch of eight or more an
    empty row."""
    n, most = case["batch"], case["max_len"]
    if not case["ragged"]:
        return [most] * n
    r = random.Random(n * 1000003 + most)
    lens = [most] + [r.randint(1, most) for _ in range(n - 1)]
    if n >= 8:
        lens[1] = 0
    return lens


def _seen(case):
    """How many tokens each sequence's query sees."""
    return [min(n, case["window"]) if case["window"] else n for n in _lens(case)]


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        tensors = 2 * (3 if case["resid"] else 1)  # x, and with a residual that and the sum
        out = n + 4 * case["rows"] if case["to"] == "codes" else 2 * n
        return {"bytes": tensors * n + out + 2 * case["width"], "flops": 6 * n}
    d, g, bits = case["head_dim"], case["group"], case["bits"]
    row = d * bits // 8 + 4 * (d // g)  # a key's or a value's codes, scales and biases
    if case["op"] == "attention":
        seen = sum(_seen(case))
        vec = 2 * 2 * case["batch"] * case["heads"] * d
        table = 4 * sum(-(-n // case["page"]) for n in _seen(case)) + 4 * case["batch"]
        return {"bytes": 2 * seen * case["kv_heads"] * row + vec + table, "flops": 4 * seen * case["heads"] * d}
    n = 2 * case["tokens"] * case["kv_heads"]  # keys and values
    if case["op"] == "read":
        return {"bytes": n * (row + 2 * d) + 8 * case["tokens"], "flops": 2 * n * d}
    # append: the dense rows in, their codes out, and those read back into dense rows
    return {"bytes": n * (2 * d + row) + n * (row + 2 * d) + 16 * case["tokens"], "flops": 8 * n * d}


def _cache(case, gen, pages, random_rows):
    """The triples (packed, scales, biases) of keys and values, over `pages` pages."""
    h, s, d, g, bits, dt = (case["kv_heads"], case["page"], case["head_dim"], case["group"], case["bits"],
                            _DTYPES[case["dtype"]])
    made = []
    for _ in range(2):
        if random_rows:
            packed = torch.randint(-2**31, 2**31, (pages, h, s, d * bits // 32), generator=gen, device="cuda",
                                   dtype=torch.int32)
            sigma = torch.empty((pages, h, s, d // g), device="cuda").uniform_(0.5, 1.5, generator=gen)
            scales = (sigma * (5.5 / (2**bits - 1))).to(dt)  # a normal group's range is about 5.5 of its deviations
            biases = (sigma * torch.empty_like(sigma).uniform_(-3.0, -2.5, generator=gen)).to(dt)
        else:
            packed = torch.zeros((pages, h, s, d * bits // 32), device="cuda", dtype=torch.int32)
            scales = torch.zeros((pages, h, s, d // g), device="cuda", dtype=dt)
            biases = torch.zeros_like(scales)
        made.append((packed, scales, biases))
    return made


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] == "norm":
        m, k = case["rows"], case["width"]
        x = normal(m, k)
        x[:, :: max(1, k // 8)] *= 20.0  # the few wide channels of a residual stream
        return {**case, "x": x.to(dt), "r": normal(m, k).to(dt) if case["resid"] else None,
                "w": (1.0 + 0.1 * normal(k)).to(dt)}
    if case["op"] == "attention":
        n, s = case["batch"], case["page"]
        per = max(1, -(-case["max_len"] // s))
        pages = n * per + 3
        lens = torch.tensor(_lens(case))[torch.randperm(n, generator=torch.Generator().manual_seed(seed))]
        table = torch.randperm(pages, generator=gen, device="cuda")[: n * per].to(torch.int32).view(n, per)
        k, v = _cache(case, gen, pages, True)
        st = {**case, "q": (1.5 * normal(n, case["heads"], case["head_dim"])).to(dt), "k": k, "v": v, "table": table,
              "lens": lens.to(torch.int32).to("cuda")}
    else:
        t, s, shape = case["tokens"], case["page"], (case["tokens"], case["kv_heads"], case["head_dim"])
        pages = -(-t // s) + 2
        k, v = _cache(case, gen, pages, case["op"] == "read")
        at = torch.randperm(pages, generator=gen, device="cuda")[: -(-t // s)]  # whole pages, in any order
        slots = (at[:, None] * s + torch.arange(s, device="cuda")).reshape(-1)[:t].contiguous()
        if case["op"] == "append" and t >= 8:
            slots[t - t // 8:] = -1  # the rows that fill a padded batch up
        st = {**case, "k": k, "v": v, "slots": slots}
        if case["op"] == "append":
            # keys carry a few channels that are wide in every token
            channel = 1.0 + 3.0 * (torch.rand(shape[1:], generator=gen, device="cuda") < 0.05)
            st["k_new"], st["v_new"] = (normal(*shape) * channel).to(dt), normal(*shape).to(dt)
    if own:
        import group_wise_affine_unpack_amd as qa
        st["cache"] = qa.AffineKVCache(st["k"], st["v"], case["group"], case["bits"])
    return st


def run(st):
    return _own(st) if own else _PLAIN[st["op"]](st)


def _own(st):
    import group_wise_affine_unpack_amd as qa
    if st["op"] == "norm":
        if st["to"] == "dense":
            y, h = qa.rmsnorm(st["x"], st["w"], _EPS, resid=st["r"])
            return {"y": y, "h": h} if st["resid"] else {"y": y}
        x_q, s_x, h = qa.rmsnorm_w4a8(st["x"], st["w"], _EPS, resid=st["r"])
        y = torch.mul(x_q, s_x[:, None], out=torch.empty_like(st["x"]))  # the values that the codes stand for
        return {"y": y, "s": s_x, "h": h} if st["resid"] else {"y": y, "s": s_x}
    if st["op"] == "attention":
        return qa.paged_attention_affine(st["q"], st["cache"], st["table"], st["lens"], window=st["window"])
    if st["op"] == "append":
        qa.kv_cache_append_affine(st["cache"], st["k_new"], st["v_new"], st["slots"])
    return qa.kv_cache_read_affine(st["cache"], st["slots"])


def _plain_norm(st):
    x, dt = st["x"], st["x"].dtype
    h = (x.float() + st["r"].float()).to(dt) if st["resid"] else x
    mean = h.double().square().mean(-1, keepdim=True)
    y = h.float() * (mean + _EPS).rsqrt().float() * st["w"].float()
    out = {"h": h} if st["resid"] else {}
    if st["to"] == "dense":
        return {"y": y.to(dt), **out}
    s = (y.abs().amax(-1, keepdim=True).double() / 127.0).float()
    q = torch.where(s > 0, torch.round(y / s), 0.0).clamp(-127, 127)
    return {"y": (q * s).to(dt), "s": s[:, 0], **out}


def _plain_values(triple, rows, case):
    """fp32 values of cache rows given as (pages, offsets) or (pages,): code * scale + bias, group by group."""
    packed, scales, biases = (t[rows] for t in triple)
    bits, g = case["bits"], case["group"]
    shifts = torch.arange(0, 32, bits, device=packed.device, dtype=torch.int32)
    codes = ((packed.unsqueeze(-1) >> shifts) & (2**bits - 1)).flatten(-2).unflatten(-1, (-1, g))
    return (codes.float() * scales.float().unsqueeze(-1) + biases.float().unsqueeze(-1)).flatten(-2)


def _plain_read(st):
    at, s = st["slots"], st["page"]
    ok = (at >= 0)[:, None, None]
    page, off = at.clamp(min=0) // s, at.clamp(min=0) % s
    rows = (page[:, None], torch.arange(st["kv_heads"], device=at.device)[None], off[:, None])
    dt = _DTYPES[st["dtype"]]
    return tuple(torch.where(ok, _plain_values(st[n], rows, st), 0.0).to(dt) for n in ("k", "v"))


def _plain_write(triple, x, rows, case):
    bits, g, most = case["bits"], case["group"], float(2 ** case["bits"] - 1)
    x = x.float().unflatten(-1, (-1, g))
    lo, hi = x.amin(-1), x.amax(-1)
    scales = ((hi - lo) / torch.full_like(hi, most)).to(triple[1].dtype)
    biases = lo.to(triple[2].dtype)
    s, b = scales.float().unsqueeze(-1), biases.float().unsqueeze(-1)
    codes = torch.where(s != 0, torch.round((x - b) / s), 0.0).clamp(0, most).flatten(-2).to(torch.int64)
    shifts = torch.arange(0, 32, bits, device=x.device)
    words = (codes.unflatten(-1, (-1, 32 // bits)) << shifts).sum(-1)
    triple[0][rows] = torch.where(words >= 2**31, words - 2**32, words).to(torch.int32)
    triple[1][rows] = scales
    triple[2][rows] = biases


def _plain_append(st):
    at, s = st["slots"], st["page"]
    kept = (at >= 0).nonzero()[:, 0]
    at = at[kept]
    rows = ((at // s)[:, None], torch.arange(st["kv_heads"], device=at.device)[None], (at % s)[:, None])
    _plain_write(st["k"], st["k_new"][kept], rows, st)
    _plain_write(st["v"], st["v_new"][kept], rows, st)
    return _plain_read(st)


def _plain_attention(st):
    q, table, lens = st["q"], st["table"].long(), st["lens"].long()
    n, heads, d = q.shape
    kv = st["kv_heads"]

    def dense(triple):  # [batch, kv_heads, tokens, head_dim]
        return _plain_values(triple, (table,), st).transpose(1, 2).flatten(2, 3)

    k = dense(st["k"])
    at = torch.arange(k.shape[2], device=q.device)
    first = (lens - st["window"]).clamp(min=0) if st["window"] else torch.zeros_like(lens)
    seen = ((at >= first[:, None]) & (at < lens[:, None]))[:, None, None]
    logits = (q.float().view(n, kv, heads // kv, d) @ k.transpose(2, 3)) / math.sqrt(d)
    del k
    logits = logits.masked_fill(~seen, -math.inf)
    most = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(most == -math.inf, 0.0, most))
    total = p.sum(-1, keepdim=True)
    out = (p @ dense(st["v"])) / torch.where(total > 0, total, 1.0)
    return out.view(n, heads, d).to(q.dtype)


_PLAIN = {"norm": _plain_norm, "append": _plain_append, "read": _plain_read, "attention": _plain_attention}


def _exact_codes(packed, bits):
    """Codes of packed rows, lowest bits first, from their bytes."""
    b = packed.contiguous().view(torch.uint8)
    parts = [(b >> i) & (2**bits - 1) for i in range(0, 8, bits)]
    return torch.stack(parts, -1).flatten(-2).double()


def _exact_values(triple, index, bits, g):
    codes = _exact_codes(triple[0][index], bits)
    scale = triple[1][index].double().repeat_interleave(g, -1)
    return codes * scale + triple[2][index].double().repeat_interleave(g, -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        x, dt = st["x"].double(), st["x"].dtype
        h = (x + st["r"].double()).to(dt).double() if case["resid"] else x
        y = h / torch.sqrt((h * h).sum(-1) / case["width"] + _EPS)[:, None] * st["w"].double()
        out = {"h": x + st["r"].double()} if case["resid"] else {}
        if case["to"] == "dense":
            return {"y": y, **out}
        s = y.abs().max(-1).values / 127
        q = (y / torch.where(s > 0, s, 1.0)[:, None]).round().clamp(-127, 127)
        return {"y": q * s[:, None], "s": s, **out}
    bits, g, size = case["bits"], case["group"], case["page"]
    if case["op"] == "attention":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        kv, d = case["kv_heads"], case["head_dim"]
        for i, n in enumerate(st["lens"].tolist()):
            first = max(0, n - case["window"]) if case["window"] else 0
            at = torch.arange(first, n, device="cuda")
            if not len(at):
                continue
            index = (st["table"][i].long()[at // size], slice(None), at % size)
            k = _exact_values(st["k"], index, bits, g).permute(1, 2, 0).contiguous()  # [kv_heads, head_dim, tokens]
            p = torch.softmax(st["q"][i].double().view(kv, -1, d) @ k / math.sqrt(d), -1)
            del k
            out[i] = (p @ _exact_values(st["v"], index, bits, g).transpose(0, 1).contiguous()).view(-1, d)
        return out
    at = st["slots"]
    kept = at >= 0
    if case["op"] == "read":
        index = (at // size, slice(None), at % size)
        return tuple(_exact_values(st[n], index, bits, g) for n in ("k", "v"))
    outs = []
    for name in ("k", "v"):
        x = st[name + "_new"].double().view(*st[name + "_new"].shape[:2], -1, g)
        bias, dt = x.min(-1, keepdim=True).values, st[name + "_new"].dtype
        scale = ((x.max(-1, keepdim=True).values - bias) / (2**bits - 1)).to(dt).double()
        codes = ((x - bias) / torch.where(scale > 0, scale, 1.0)).round().clamp(0, 2**bits - 1)
        outs.append((codes * scale + bias).flatten(2) * kept[:, None, None])
    return tuple(outs)
