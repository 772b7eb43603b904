"""GPU tests of qmoe_affine against the fp64 definition (oracle.decoder.moe).

Tolerance, derived from the kernel's roundings: a rounding of fp32 is u =
2^-24 of what it rounds (2 u where the matrix cores may cut; products of codes, which are
subnormal there, at 2^-14 of a code's step times the largest x, which for the
random signs here adds below 2^-18 of the sizes even with 2 bits).  A group's sums
of G products and the sum over K/G groups are taken as random walks with a
factor 6, 6 (2 sqrt(G) + sqrt(K/G)) u of the sizes of what is added (for the
larger of the two products' K): `size` of the oracle, which carries the first
product's error through silu and the second product.  x is exact, h is held to
2^-22, exp, the division and the weights are off by a few u: all below the
factor's least value, 6 (2 sqrt(32) + 1) = 73.  Then half a step of the output
type.  The tests show that a scale 5% off would fail."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle
import oracle.decoder as od
import synth_inputs as si
from gpu_util import TORCH_DT, dev16, dev32, host_f64, require_gpu

pytestmark = pytest.mark.gpu

U = 2.0**-24
HALF = {"bf16": 2.0**-8, "f16": 2.0**-11}


def _experts(E, K, I, G, bits, act, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    triples = []
    for rows, cols in ((2 * I, K), (K, I)):
        packed = rng.integers(0, 2**32, (E, rows, cols * bits // 32), dtype=np.uint32)
        sigma = np.exp(rng.uniform(-spread, spread, (E, rows, cols // G))) / np.sqrt(cols)
        s = sigma * 5.5 / (2**bits - 1) * np.where(rng.random(sigma.shape) < 0.1, -1, 1)  # scales below zero too
        b = -sigma * rng.uniform(2.5, 3.0, sigma.shape)
        triples.append((packed, si.store(s.astype(np.float32), act), si.store(b.astype(np.float32), act)))
    return triples


def _to_device(triples, act, dev, G, bits):
    return qa.AffineExperts(*[(dev32(w, dev), dev16(s, act, dev), dev16(b, act, dev)) for w, s, b in triples], G, bits)


def _compare(got, ref, size, K, I, G, act):
    factor = 6 * (2 * np.sqrt(G) + np.sqrt(max(K, I) / G)) * U
    err, tol = np.abs(got - ref), factor * size * 1.001 + HALF[act] * np.abs(ref) + 2.0**-25
    # a value past the type's largest by half a step or more rounds to infinity: f16, 65520
    over = {"f16": 65520.0, "bf16": 2.0**128 * (1 - 2.0**-9)}[act]
    beyond = np.abs(ref) - factor * size > over
    assert (got[beyond] == np.copysign(np.inf, ref[beyond])).all()
    err = np.where(np.isinf(got) & (np.abs(ref) + factor * size >= over), 0.0, err)
    assert np.isfinite(got[np.abs(ref) + factor * size < over]).all() and not np.isnan(got).any()
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    print(f"[parity] worst {(err / tol)[worst]:.3f} of the bound at {worst}", flush=True)
    assert (err <= tol).all(), f"{(err > tol).sum()} beyond, worst {(err / tol)[worst]} at {worst}"
    return tol


def _check(M, K, I, E, top_k, G, bits, act, renormalize=True, logit="f32", resid=True, seed=0, scale=1.0, logits=None, x=None,
           tell=0.05):
    dev = require_gpu()
    print(f"[case] moe M={M} K={K} I={I} E={E} top_k={top_k} G={G} bits={bits} {act} renorm={renormalize} {logit}", flush=True)
    rng = np.random.default_rng((seed, M, K, E))
    triples = _experts(E, K, I, G, bits, act, (seed, 1))
    if x is None:
        x = si.store(rng.standard_normal((M, K)).astype(np.float32), act)
    if logits is None:
        logits = (1.5 * rng.standard_normal((M, E))).astype(np.float32)
    zb = logits.astype(np.float32) if logit == "f32" else si.store(logits.astype(np.float32), act)
    z = zb.astype(np.float64) if logit == "f32" else oracle.to_f64(zb, act)
    r = si.store(rng.standard_normal((M, K)).astype(np.float32), act) if resid else None
    experts = _to_device(triples, act, dev, G, bits)
    zd = torch.from_numpy(zb).to(dev) if logit == "f32" else dev16(zb, act, dev)
    y = qa.qmoe_affine(dev16(x, act, dev), zd, experts, top_k, renormalize, scale, resid=None if r is None else dev16(r, act, dev))
    torch.cuda.synchronize()
    ref, size, chosen = od.moe(x, z, *triples, act, G, bits, top_k, renormalize, scale, r)
    got = host_f64(y)
    tol = _compare(got, ref, size, K, I, G, act)
    # what the bound can tell: the experts' part 5% off (`tell`: sizes grow with the columns, sums only with their root, so
    # rows of thousands tell less) is far outside in every row
    base = ref - (0 if r is None else oracle.to_f64(r, act))
    part = np.abs(base).max(1) > 1e-3
    assert ((np.abs(tell * base) > 2 * tol).any(1) | ~part).all()
    return got, chosen


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 3, 7])
def test_widths_groups_types(M, G, bits, act):
    _check(M, 256, 384, 6, 2, G, bits, act, seed=G + bits)
    _check(M, 384, 128, 5, 3, G, bits, act, renormalize=False, logit=act, resid=False, seed=G + bits + 1)


@pytest.mark.parametrize("bits,G,K,I", [(4, 32, 32, 32), (4, 32, 96, 160), (8, 32, 32, 96), (8, 64, 64, 192), (4, 64, 192, 64),
                                        (4, 128, 128, 640), (2, 64, 64, 192), (2, 128, 384, 128), (2, 32, 320, 64),
                                        (4, 64, 2048, 64), (8, 128, 128, 2176), (2, 32, 64, 4160)])
@pytest.mark.parametrize("M", [1, 5, 20])
def test_odd_sizes(M, bits, G, K, I):
    _check(M, K, I, 4, 2, G, bits, "bf16", seed=K + I)


@pytest.mark.parametrize("M,E,top_k", [(1, 1, 1), (1, 8, 8), (1, 300, 4), (2, 64, 6), (4, 4, 1), (9, 2, 2), (16, 3, 1), (17, 2, 1),
                                       (33, 64, 2), (64, 4, 2), (65, 130, 8), (256, 3, 2), (255, 1024, 1), (3, 1024, 20)])
def test_batches_and_routes(M, E, top_k):
    _check(M, 64, 64, E, top_k, 32, 4, "f16", seed=M + E)
    _check(M, 64, 64, E, top_k, 32, 8, "bf16", renormalize=False, logit="bf16", seed=M + E + 1)


# From 1024 tiles on (16 rows of gate and up, 32 of down, of every expert that a batch may reach) a wave takes whole rows,
# with x of 4, 8 or 16 rows at a time by how many tokens an expert has; a tile or two a wave.
@pytest.mark.parametrize("act,bits,G", [("bf16", 4, 64), ("f16", 4, 32), ("f16", 4, 128), ("bf16", 8, 64), ("f16", 8, 32),
                                        ("bf16", 8, 128), ("bf16", 2, 64), ("f16", 2, 32), ("f16", 2, 128)])
@pytest.mark.parametrize("M,top_k", [(2, 64), (7, 8), (24, 8), (60, 8)])
def test_many_experts(M, top_k, act, bits, G):
    _check(M, 512, 256, 64, top_k, G, bits, act, seed=G + bits)


@pytest.mark.parametrize("M", [9, 33, 65])
@pytest.mark.parametrize("bits,G,K,I", [(4, 32, 544, 288), (8, 32, 544, 288), (2, 64, 576, 320), (4, 128, 640, 384), (4, 64, 64, 1024),
                                        (8, 64, 1088, 320)])
def test_many_experts_odd_sizes(M, bits, G, K, I):
    _check(M, K, I, 72, 6, G, bits, "bf16", renormalize=False, logit="bf16", seed=K + I)


def test_many_experts_crowded():
    # one expert takes every token, several passes over its rows, and many take none
    rng = np.random.default_rng(13)
    for M in (16, 50):
        z = rng.standard_normal((M, 64)).astype(np.float32)
        z[:, 9] = 8
        z[:, 20:40] = -np.inf
        _check(M, 512, 256, 64, 4, 64, 4, "f16", logits=z)


# Rows of x longer than LDS holds of 16: part by part, a tile a wave.
@pytest.mark.parametrize("bits,G,K,I,E", [(4, 64, 2176, 512, 32), (4, 32, 2080, 512, 32), (8, 64, 2624, 512, 32), (2, 128, 2304, 512, 32),
                                          (4, 128, 1024, 2432, 32), (8, 32, 1024, 2144, 32), (8, 128, 1024, 5248, 32)])
def test_long_rows_of_many_tokens(bits, G, K, I, E):
    _check(33, K, I, E, 4, G, bits, "bf16" if bits == 4 else "f16", seed=K, tell=0.2)


def test_every_token_to_one_expert():
    rng = np.random.default_rng(8)
    z = rng.standard_normal((40, 6)).astype(np.float32)
    z[:, 4] = 9
    _check(40, 128, 128, 6, 1, 64, 4, "bf16", logits=z)
    _check(40, 128, 128, 6, 2, 64, 4, "f16", logits=z)


@pytest.mark.parametrize("M", [1, 2, 12])
def test_ties_go_to_the_lowest_index(M):
    rng = np.random.default_rng(9)
    z = rng.integers(0, 2, (M, 16)).astype(np.float32)  # many equal logits
    z[0] = 1
    for renormalize in (True, False):
        _, chosen = _check(M, 64, 96, 16, 5, 32, 4, "f16", renormalize, logits=z)
        assert chosen[0] == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("M", [1, 3, 9])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masked_logits(M, renormalize):
    # minus infinity is never chosen: fewer choices than top_k, or none, which leaves the residual
    rng = np.random.default_rng(10)
    z = rng.standard_normal((M, 8)).astype(np.float32)
    z[:, 2:] = -np.inf
    z[M - 1] = -np.inf
    got, chosen = _check(M, 64, 64, 8, 4, 32, 4, "bf16", renormalize, logits=z, seed=3)
    assert chosen[M - 1] == [] and all(len(c) == 2 for c in chosen[:-1])
    dev = require_gpu()
    experts = _to_device(_experts(8, 64, 64, 32, 4, "bf16", 1), "bf16", dev, 32, 4)
    x = torch.randn((M, 64), device=dev).bfloat16()
    zd = torch.full((M, 8), float("-inf"), device=dev)
    assert (qa.qmoe_affine(x, zd, experts, 4, renormalize) == 0).all()
    assert torch.equal(qa.qmoe_affine(x, zd, experts, 4, renormalize, resid=x), x)
    # the type's lowest value is a number like any other
    zd[:] = torch.finfo(torch.float32).min
    y = qa.qmoe_affine(x, zd, experts, 4, renormalize)
    assert torch.isfinite(y).all() and (y != 0).any()


@pytest.mark.parametrize("E,K,I", [(6, 128, 64), (64, 512, 256)])
def test_nan_and_infinities_stay_in_their_rows(E, K, I):
    dev = require_gpu()
    experts = _to_device(_experts(E, K, I, 32, 4, "f16", 2), "f16", dev, 32, 4)
    x, z = torch.randn((9, K), device=dev).half(), torch.randn((9, E), device=dev)
    good = qa.qmoe_affine(x, z, experts, 2)
    bad_x, bad_z = x.clone(), z.clone()
    bad_x[2, 5], bad_x[4, 7] = float("nan"), float("inf")
    bad_z[6, 1] = float("nan")
    y = qa.qmoe_affine(bad_x, bad_z, experts, 2)
    keep = [0, 1, 3, 5, 7, 8]
    assert torch.equal(y[keep], good[keep])
    assert torch.isnan(y[6]).all() and not torch.isfinite(y[[2, 4]]).any()


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_one_token_of_any_size(act):
    # one token's two kernels, their several quads of columns a wave, and the sizes at which a batch's take over
    for K, I, E, top_k in ((2048, 512, 8, 2), (64, 6144, 4, 1), (64, 6144, 8, 4), (4096, 64, 6, 6), (2080, 2080, 3, 2), (96, 96, 256, 64)):
        _check(1, K, I, E, top_k, 32, 4, act, seed=K + I, renormalize=E != 6)


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_rows_of_any_size(act):
    # one wide entry among small ones, tiny and large rows, zeros
    rng = np.random.default_rng(11)
    v = rng.standard_normal((8, 256))
    v[0, 3] = 3000
    v[1] *= 1e-3 if act == "f16" else 1e-6
    v[2] *= 200 if act == "f16" else 1e4
    v[3] = 0
    v[4] *= np.exp(rng.uniform(-9, 2, 256))
    _check(8, 256, 128, 3, 2, 64, 4, act, x=si.store(v.astype(np.float32), act), resid=False, seed=5)


def test_weights_that_are_not_finite_stay_in_their_column():
    # a scale next to a row's end is not read for the row before it
    dev = require_gpu()
    triples = _experts(2, 96, 96, 32, 4, "bf16", 3)
    clean = _to_device(triples, "bf16", dev, 32, 4)
    x, z = torch.randn((2, 96), device=dev).bfloat16(), torch.zeros((2, 2), device=dev)
    good = qa.qmoe_affine(x, z, clean, 2)
    triples[1][1][1, 17, 0] = 0x7FC0
    y = qa.qmoe_affine(x, z, _to_device(triples, "bf16", dev, 32, 4), 2)
    bad = torch.zeros(96, dtype=torch.bool)
    bad[17] = True
    assert torch.isnan(y[:, bad]).all() and torch.equal(y[:, ~bad], good[:, ~bad])


def test_in_place_and_repeated():
    dev = require_gpu()
    experts = _to_device(_experts(9, 256, 96, 32, 4, "bf16", 4), "bf16", dev, 32, 4)
    for M in (1, 2, 30):
        x, z, r = torch.randn((M, 256), device=dev).bfloat16(), torch.randn((M, 9), device=dev), torch.randn((M, 256), device=dev).bfloat16()
        first = qa.qmoe_affine(x, z, experts, 3, resid=r)
        for _ in range(3):
            assert torch.equal(qa.qmoe_affine(x, z, experts, 3, resid=r), first)
        out = r.clone()
        assert qa.qmoe_affine(x, z, experts, 3, resid=out, out=out) is out and torch.equal(out, first)


def test_batch_rows_do_not_depend_on_each_other():
    # a row of a batch against the same row alone: other launches, the same sums to within the bound of both
    dev = require_gpu()
    triples = _experts(5, 256, 256, 64, 4, "f16", 6)
    experts = _to_device(triples, "f16", dev, 64, 4)
    x, z = torch.randn((50, 256), device=dev).half(), torch.randn((50, 5), device=dev)
    y = qa.qmoe_affine(x, z, experts, 2)
    one = torch.cat([qa.qmoe_affine(x[i:i + 1].contiguous(), z[i:i + 1].contiguous(), experts, 2) for i in range(50)])
    ref, size, _ = od.moe(x.cpu().view(torch.int16).numpy().view(np.uint16), z.cpu().double().numpy(), *triples, "f16", 64, 4, 2, True)
    for got in (y, one):
        _compare(host_f64(got), ref, size, 256, 256, 64, "f16")


def test_empty_batch():
    dev = require_gpu()
    experts = _to_device(_experts(2, 64, 64, 32, 4, "f16", 4), "f16", dev, 32, 4)
    assert qa.qmoe_affine(torch.zeros((0, 64), device=dev).half(), torch.zeros((0, 2), device=dev), experts, 1).shape == (0, 64)


def test_captured_call_follows_its_replays():
    # the routes of the replay, not of the capture; eager work on other shapes in between
    dev = require_gpu()
    for M, E, K, I in ((1, 16, 256, 128), (6, 16, 256, 128), (20, 64, 512, 256)):
        experts = _to_device(_experts(E, K, I, 64, 4, "bf16", 7), "bf16", dev, 64, 4)
        x, z = torch.randn((M, K), device=dev).bfloat16(), torch.randn((M, E), device=dev)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            qa.qmoe_affine(x, z, experts, 4, resid=x)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                y = qa.qmoe_affine(x, z, experts, 4, resid=x)
        for i in range(6):
            x.normal_()
            z.normal_()
            if i == 3:
                z[0] = float("-inf")
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            want = qa.qmoe_affine(x, z, experts, 4, resid=x)
            torch.cuda.synchronize()
            assert torch.equal(y, want), (M, i)


def test_two_streams():
    dev = require_gpu()
    experts = _to_device(_experts(16, 256, 128, 64, 4, "bf16", 7), "bf16", dev, 64, 4)
    xs, zs = torch.randn((2, 8, 20, 256), device=dev).bfloat16(), torch.randn((2, 8, 20, 16), device=dev)
    want = [[qa.qmoe_affine(xs[s, i], zs[s, i], experts, 4) for i in range(8)] for s in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for i in range(8):
        for s, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[s].append(qa.qmoe_affine(xs[s, i], zs[s, i], experts, 4))
    torch.cuda.synchronize()
    for a, b in zip(want[0] + want[1], got[0] + got[1]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("M,E", [(1, 8), (8, 64), (40, 64), (256, 8)])
def test_inner_precision(M, E, bits):
    """h and its sums beyond the output's 11 bits: Down copies h (code and scale 1), a second call with the first one's
    output as the negative residual returns what the first rounding left, so h is seen to 2^-22.

    Bound on the rms: a product of a code is cut at 2^-14 of the code's step s times the largest x, K independent cuts,
    twice that; two fp32 roundings a group of sums that walk to sqrt(sum (w x)^2), 3 times that; h, silu and the
    remainder's rounding at 2^-20 together.  (Sums of x left 2^-15 off would be twice the bound of 8 bits.)"""
    dev = require_gpu()
    K, G = 1024, 64
    print(f"[case] moe precision M={M} E={E} bits={bits}", flush=True)
    rng = np.random.default_rng((M, E, bits))
    per = 32 // bits

    def pack(c):
        return (c.reshape(*c.shape[:-1], -1, per).astype(np.uint64) << (np.arange(per, dtype=np.uint64) * np.uint64(bits))).sum(-1).astype(np.uint32)

    I = 256
    q = rng.integers(0, 2**bits, (E, 2 * I, K))
    s = (rng.uniform(0.5, 1.0, (E, 2 * I, K // G)) * 0.15 / 2**bits).astype(np.float16)
    b = (-s.astype(np.float64) * (2**bits - 1) / 2).astype(np.float16)
    d = np.zeros((E, K, I), np.int64)
    n = np.arange(K)
    d[:, n, n % I] = 1
    triples = [(pack(q), s.view(np.uint16), b.view(np.uint16)),
               (pack(d), np.ones((E, K, I // G), np.float16).view(np.uint16), np.zeros((E, K, I // G), np.uint16))]
    ex = _to_device(triples, "f16", dev, G, bits)
    x = rng.standard_normal((M, K)).astype(np.float16)
    z = rng.standard_normal((M, E)).astype(np.float32)
    xd, zd = torch.from_numpy(x).to(dev), torch.from_numpy(z).to(dev)
    y0 = qa.qmoe_affine(xd, zd, ex, 1)
    y1 = qa.qmoe_affine(xd, zd, ex, 1, resid=-y0)
    got = host_f64(y0) + host_f64(y1)
    x64 = x.astype(np.float64)
    ref, var, size = np.empty((M, K)), [], []
    for m, e in enumerate(z.argmax(1)):
        step, off = s[e].astype(np.float64).repeat(G, -1), b[e].astype(np.float64).repeat(G, -1)
        a = (q[e] * step + off) @ x64[m]
        g, u = a[:I], a[I:]
        silu = g / (1 + np.exp(-g))
        ref[m] = (silu * u)[n % I]
        walk = np.sqrt(((q[e] * step) ** 2) @ x64[m] ** 2).max() + np.sqrt((off**2) @ x64[m] ** 2).max()
        delta = 2 * np.sqrt(K) * 2.0**-14 * step.max() * np.abs(x64[m]).max() + 3 * np.sqrt(2 * K / G) * U * walk
        var.append(delta**2 * ((1.1 * u) ** 2 + silu**2).mean())
    rms = np.sqrt(((got - ref) ** 2).mean())
    tol = np.sqrt(np.mean(var)) + 2.0**-20 * np.sqrt((ref**2).mean())
    print(f"[parity] rms {rms:.3g} of {np.sqrt((ref**2).mean()):.3g}, bound {tol:.3g}", flush=True)
    assert rms <= tol
