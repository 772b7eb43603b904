"""A serving loop's steps with the operators in a row, as they would be used:
pages for the new tokens, the norm, the q/k/v product, positions turned while
keys and values go to the cache, attention over it, the output product, the
norm with the residual, the router's product and the experts.  Each stage is
checked against fp64 on what it was given; then the whole step captured and
replayed, its sequences growing, ending and starting on the device."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle
import oracle.decoder as od
from gpu_util import host_f64, require_gpu

pytestmark = pytest.mark.gpu

WIDTH, HEADS, KVH, D, G, PAGE, EPS = 256, 8, 2, 64, 64, 16, 1e-5
EXPERTS, TOP_K, INNER = 8, 2, 128
PER = 6  # pages of a row of the table


def _bits(t):
    t = t.cpu().contiguous()
    return t.numpy().view(np.uint32) if t.dtype == torch.int32 else t.view(torch.int16).numpy().view(np.uint16)


class Layer:
    def __init__(self, act, pages, batch, dev):
        g = torch.Generator(device=dev).manual_seed(11)
        self.act, self.dt, self.dev = act, {"bf16": torch.bfloat16, "f16": torch.float16}[act], dev

        def weight(*shape):
            w = (torch.randn((int(np.prod(shape[:-1])), shape[-1]), generator=g, device=dev) / shape[-1] ** 0.5).to(self.dt)
            return tuple(t.view(*shape[:-1], -1) for t in qa.quantize_pack_affine(w, G, 4, self.dt))
        self.qkv, self.o = weight((HEADS + 2 * KVH) * D, WIDTH), weight(WIDTH, HEADS * D)
        self.router = weight(EXPERTS, WIDTH)
        self.experts = qa.AffineExperts(weight(EXPERTS, 2 * INNER, WIDTH), weight(EXPERTS, WIDTH, INNER), G, 4)
        self.norms = [(1 + 0.1 * torch.randn(WIDTH, generator=g, device=dev)).to(self.dt) for _ in range(2)]
        self.cache = qa.AffineKVCache.empty(pages, PAGE, KVH, D, G, 4, self.dt, dev)
        self.pool = qa.KVPagePool(pages, PAGE, dev)
        self.rot = qa.Rotary.make(D, scaling="bands", factor=8.0, original_len=8192.0, device=dev)
        self.table = torch.full((batch, PER), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)

    def tokens(self, h, new, rows):
        """Everything up to the cache write, for rows of new tokens."""
        slots, pos, seq, _ = qa.kv_pages_assign(self.pool, self.table, self.lens, new, rows, lens_out=self.lens)
        x, _ = qa.rmsnorm(h, self.norms[0], EPS)
        qkv = qa.qmm_affine(x, *self.qkv, G, 4).view(rows, HEADS + 2 * KVH, D)
        q, k, v = qkv.split((HEADS, KVH, KVH), 1)
        return slots, pos, seq, x, qkv, qa.kv_cache_append_rotary_affine(self.cache, q, k, v, pos, slots, self.rot)

    def step(self, h, new):
        slots, pos, seq, x, qkv, q = self.tokens(h, new, len(h))
        a = qa.paged_attention_affine(q, self.cache, self.table, self.lens)
        o = qa.qmm_affine(a.view(len(h), HEADS * D), *self.o, G, 4)
        y, h2 = qa.rmsnorm(o, self.norms[1], EPS, resid=h)
        logits = qa.qmm_affine(y, *self.router, G, 4)
        return slots, pos, seq, x, qkv, q, a, o, y, h2, logits, qa.qmoe_affine(y, logits, self.experts, TOP_K, resid=h2)


def _product(x, w, act):
    return host_f64(x) @ od.values(_bits(w[0]), _bits(w[1]), _bits(w[2]), act, G, 4).T


def _check(layer, h, got):
    act = layer.act
    slots, pos, seq, x, qkv, q, a, o, y, h2, logits, out = got
    assert oracle.affine_tolerance_report(host_f64(qkv).reshape(len(h), -1), _product(x, layer.qkv, act))["ok"]
    freq = layer.rot.inv_freq.cpu().numpy()
    rows = _bits(qkv)
    for name, part, at in (("q", rows[:, :HEADS], None), ("k", rows[:, HEADS:HEADS + KVH], layer.cache.k),
                           ("v", rows[:, HEADS + KVH:], layer.cache.v)):
        if name != "v":
            value, slack = od.rotary(part, pos.cpu().numpy(), freq, act, False)
            low, high = od._store(value - slack, act), od._store(value + slack, act)
        if name == "q":
            assert ((_bits(q) == low) | (_bits(q) == high)).all()
            continue
        want = od.quantize_rows(part if name == "v" else low, act, G, 4)
        pg, off = (slots // PAGE).cpu().numpy(), (slots % PAGE).cpu().numpy()
        sure = np.ones(len(h), bool) if name == "v" else (low == high).reshape(len(h), -1).all(1)
        assert sure.mean() > 0.5
        for t, ref in zip(at, want):
            assert (_bits(t)[pg, :, off][sure] == ref[sure]).all(), name
    ref, bound = od.paged_attention(_bits(q), tuple(map(_bits, layer.cache.k)), tuple(map(_bits, layer.cache.v)), act, G, 4,
                                    layer.table.cpu().numpy(), layer.lens.cpu().numpy(), D**-0.5)
    half = 2.0**-8 if act == "bf16" else 2.0**-11
    assert (np.abs(host_f64(a) - ref) <= bound * 1.001 + half * np.abs(ref) + 2.0**-25).all()
    assert oracle.affine_tolerance_report(host_f64(o), _product(a.view(len(h), -1), layer.o, act))["ok"]
    assert oracle.affine_tolerance_report(host_f64(logits), _product(y, layer.router, act))["ok"]
    e = layer.experts
    ref, size, _ = od.moe(_bits(y), host_f64(logits), tuple(map(_bits, e.gate_up)), tuple(map(_bits, e.down)), act, G, 4, TOP_K,
                          True, 1.0, _bits(h2))
    tol = 6 * (2 * np.sqrt(G) + np.sqrt(WIDTH / G)) * 2.0**-24 * size * 1.001 + half * np.abs(ref) + 2.0**-25
    assert (np.abs(host_f64(out) - ref) <= tol).all()


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("batch", [1, 3, 9])
def test_prompts_then_steps(act, batch):
    dev = require_gpu()
    layer = Layer(act, batch * PER + 2, batch, dev)
    g = torch.Generator(device=dev).manual_seed(3)
    prompts = torch.tensor([(7 * i + 14) % 40 for i in range(batch)], dtype=torch.int32, device=dev)
    rows = int(prompts.sum()) + 3
    h = torch.randn((rows, WIDTH), generator=g, device=dev).to(layer.dt)
    layer.tokens(h, prompts, rows)
    one = torch.ones(batch, dtype=torch.int32, device=dev)
    for i in range(4):
        h = torch.randn((batch, WIDTH), generator=g, device=dev).to(layer.dt)
        got = layer.step(h, one)
        torch.cuda.synchronize()
        assert layer.lens.tolist() == (prompts + i + 1).tolist() and int(layer.pool.state[1]) == 0
        assert got[1].tolist() == (prompts + i).tolist() and got[2].tolist() == list(range(batch))
        _check(layer, h, got)


def test_captured_step_replays_with_sequences_that_end():
    dev = require_gpu()
    batch = 5
    one, two = (Layer("f16", batch * PER, batch, dev) for _ in range(2))
    g = torch.Generator(device=dev).manual_seed(4)
    new, keep = torch.ones(batch, dtype=torch.int32, device=dev), torch.zeros(batch, dtype=torch.int32, device=dev)
    h = torch.randn((batch, WIDTH), generator=g, device=dev).half()

    def body(layer):
        layer.lens = qa.kv_pages_trim(layer.pool, layer.table, layer.lens, keep, lens_out=layer.lens)
        return layer.step(h, new)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        body(one)
        body(two)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = body(one)
        for i in range(30):
            h.copy_(torch.randn((batch, WIDTH), generator=g, device=dev))
            keep.fill_(PER * PAGE)
            if i % 7 == 3:
                keep[i % batch] = 0  # a request ends, another takes its place
            graph.replay()
            torch.cuda.synchronize()
            eager = body(two)
            torch.cuda.synchronize()
            for n, (a, b) in enumerate(zip(outs, eager)):
                assert torch.equal(a, b), (i, n)
            for name in ("lens", "table"):
                assert torch.equal(getattr(one, name), getattr(two, name)), (i, name)
            assert torch.equal(one.pool.state, two.pool.state) and torch.equal(one.pool.free_pages, two.pool.free_pages)
    for a, b in zip(one.cache.k + one.cache.v, two.cache.k + two.cache.v):
        assert torch.equal(a, b)
