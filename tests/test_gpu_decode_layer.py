"""The operators of a decoder layer's attention block in a row, as a decode
step runs them: norm into int8 codes, the q/k/v product, the cache write, the
attention over the cache, the output product, the next norm with the residual.
Each stage is checked against fp64 on the inputs that it was given (the
outputs of the stage before it), with that stage's own tolerance."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle
import oracle.decoder as od
from gpu_util import host_f64, require_gpu

pytestmark = pytest.mark.gpu

WIDTH, HEADS, KVH, D, G, PAGE, EPS = 512, 8, 2, 64, 64, 16, 1e-5


def _bits(t):
    t = t.cpu().contiguous()
    return t.numpy().view(np.uint32) if t.dtype == torch.int32 else t.view(torch.int16).numpy().view(np.uint16)


class Layer:
    def __init__(self, bits, pages, dev):
        g = torch.Generator(device=dev).manual_seed(5)

        def weight(n, k):
            return qa.w4a8_quantize_weights(0.05 * torch.randn((n, k), generator=g, device=dev))
        self.qkv, self.o = weight((HEADS + 2 * KVH) * D, WIDTH), weight(WIDTH, HEADS * D)
        self.norms = [1 + 0.1 * torch.randn(WIDTH, generator=g, device=dev) for _ in range(2)]
        self.cache = qa.AffineKVCache.empty(pages, PAGE, KVH, D, G, bits, torch.float16, dev)

    def qkv_rows(self, h):
        """(codes, scales, q/k/v rows [M, HEADS + 2 KVH, D])"""
        x_q, s_x, _ = qa.rmsnorm_w4a8(h, self.norms[0], EPS)
        y, _ = qa.qgemm_w4a8_codes(x_q, s_x, *self.qkv)
        return x_q, s_x, y.view(-1, HEADS + 2 * KVH, D)

    def step(self, h, slots, table, lens):
        x_q, s_x, qkv = self.qkv_rows(h)
        q, k, v = qkv.split((HEADS, KVH, KVH), 1)
        qa.kv_cache_append_affine(self.cache, k, v, slots)
        a = qa.paged_attention_affine(q, self.cache, table, lens)
        o = qa.qgemm_w4a8(a.view(-1, HEADS * D), *self.o)[0]
        y_q, s_y, h2 = qa.rmsnorm_w4a8(o, self.norms[1], EPS, resid=h)
        return x_q, s_x, qkv, a, o, y_q, s_y, h2


def _check_step(layer, h, slots, table, lens, got, bits):
    x_q, s_x, qkv, a, o, y_q, s_y, h2 = got

    def product(q, s, w):
        acc = oracle.w4a8_acc(q.cpu().numpy(), _bits(w[0]), q.shape[0], w[0].shape[0], q.shape[1])
        return acc * host_f64(s)[:, None] * host_f64(w[1])

    def norm(codes, scales, x, r, w):
        hb, n = od.rmsnorm(_bits(x), None if r is None else _bits(r), w.cpu().numpy(), EPS, "f16", "f32")
        s = np.abs(n).max(1) / 127
        assert (np.abs(host_f64(scales) - s) <= 2.0**-21 * s).all()
        assert (np.abs(codes.cpu().numpy() - n / s[:, None]) <= 0.5 + 127 * 2.0**-21).all()
        return hb

    norm(x_q, s_x, h, None, layer.norms[0])
    assert oracle.affine_tolerance_report(host_f64(qkv).reshape(len(h), -1), product(x_q, s_x, layer.qkv))["ok"]
    q, k, v = qkv.split((HEADS, KVH, KVH), 1)
    pg, off = (slots // PAGE).cpu().numpy(), (slots % PAGE).cpu().numpy()
    for x, arrays in ((k, layer.cache.k), (v, layer.cache.v)):
        for t, ref in zip(arrays, od.quantize_rows(_bits(x), "f16", G, bits)):
            assert (_bits(t)[pg, :, off] == ref).all()
    ref, bound = od.paged_attention(_bits(q), tuple(map(_bits, layer.cache.k)), tuple(map(_bits, layer.cache.v)), "f16", G,
                                    bits, table.cpu().numpy(), lens.cpu().numpy(), D**-0.5)
    assert (np.abs(host_f64(a) - ref) <= bound * 1.001 + 2.0**-11 * np.abs(ref) + 2.0**-25).all()
    assert oracle.affine_tolerance_report(host_f64(o), oracle.w4a8(_bits(a).reshape(len(h), -1), _bits(layer.o[0]),
                                                                   _bits(layer.o[1]), len(h), WIDTH, HEADS * D)[3])["ok"]
    assert (_bits(h2) == norm(y_q, s_y, o, h, layer.norms[1])).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_prompt_then_decode_steps(bits):
    dev = require_gpu()
    lens0, steps = [21, 5, 32], 4
    per = 3
    layer = Layer(bits, 3 * per + 1, dev)
    g = torch.Generator(device=dev).manual_seed(6)
    table = torch.randperm(3 * per + 1, generator=g, device=dev)[:3 * per].to(torch.int32).view(3, per)

    def slot(b, t):
        return table[b, t // PAGE].long() * PAGE + t % PAGE

    # the prompts' keys and values in one ragged batch, padded with two rows that go nowhere
    h = torch.randn((sum(lens0) + 2, WIDTH), generator=g, device=dev).half()
    slots = torch.stack([slot(b, t) for b, n in enumerate(lens0) for t in range(n)] + [torch.tensor(-1, device=dev)] * 2)
    _, _, qkv = layer.qkv_rows(h)
    qa.kv_cache_append_affine(layer.cache, qkv[:, HEADS:HEADS + KVH], qkv[:, HEADS + KVH:], slots)
    for i in range(steps):
        lens = torch.tensor([n + i + 1 for n in lens0], dtype=torch.int32, device=dev)
        at = torch.stack([slot(b, n + i) for b, n in enumerate(lens0)])
        h = torch.randn((3, WIDTH), generator=g, device=dev).half()
        got = layer.step(h, at, table, lens)
        torch.cuda.synchronize()
        _check_step(layer, h, at, table, lens, got, bits)


def test_captured_step_replays():
    # one captured step replayed for successive tokens, its inputs rewritten in place, against the eager step on a second cache
    dev = require_gpu()
    table = torch.tensor([[2, 0, 3], [4, 1, 5]], dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(7)
    one, two = Layer(4, 6, dev), Layer(4, 6, dev)
    h, lens = torch.zeros((2, WIDTH), dtype=torch.float16, device=dev), torch.ones(2, dtype=torch.int32, device=dev)
    slots = torch.full((2,), -1, dtype=torch.int64, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one.step(h, slots, table, lens)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = one.step(h, slots, table, lens)
        for t in range(6):
            n = 14 + t  # crosses into the second page
            h.copy_(torch.randn((2, WIDTH), generator=g, device=dev))
            lens.fill_(n + 1)
            slots.copy_(table[:, n // PAGE].long() * PAGE + n % PAGE)
            graph.replay()
            torch.cuda.synchronize()
            eager = two.step(h, slots, table, lens)
            torch.cuda.synchronize()
            for a, b in zip(outs, eager):
                assert torch.equal(a, b), t
    for a, b in zip(one.cache.k + one.cache.v, two.cache.k + two.cache.v):
        assert torch.equal(a, b)
