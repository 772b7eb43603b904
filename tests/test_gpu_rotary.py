"""GPU tests of rotary_frequencies, rotary and kv_cache_append_rotary_affine.

rotary computes in fp64 and rounds once, so an output is the rounding of a
value within the oracle's fp64 slack of the definition, which is one number but
next to a rounding border.  The
fused append is held to the two calls that it stands for, bit for bit."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle
import oracle.decoder as od
import synth_inputs as si
from gpu_util import TORCH_DT, dev16, require_gpu

pytestmark = pytest.mark.gpu


def _host(t):
    t = t.cpu().contiguous()
    return t.numpy().view(np.uint32) if t.dtype == torch.int32 else t.view(torch.int16).numpy().view(np.uint16)


def _values(shape, act, seed):
    rng = np.random.default_rng(seed)
    return si.store((rng.standard_normal(shape) * np.exp(rng.uniform(-3, 3, shape))).astype(np.float32), act)


def _same(got, ref, slack, act):
    # rounding is monotonic: the roundings of the values within the slack are those from the lower end's to the upper end's
    # (one number, but next to a border, and more than two where a value near zero is a small difference of large products)
    low, high = (oracle.to_f64(od._store(v, act), act) for v in (ref - slack, ref + slack))
    g = oracle.to_f64(_host(got), act)
    bad = ~((low <= g) & (g <= high))
    assert not bad.any(), f"{bad.sum()} of {bad.size} differ, first at {np.argwhere(bad)[0]}"


def _check(T, H, HK, D, R, interleaved, act, far=5000, seed=0, magnitude=1.0, layout="dense", in_place=False):
    dev = require_gpu()
    print(f"[case] rotary T={T} H={H}/{HK} D={D} R={R} interleaved={interleaved} {act} {layout} in_place={in_place}", flush=True)
    rng = np.random.default_rng((seed, T, D))
    pos = rng.integers(0, far, T).astype(np.int32)
    if T > 2:
        pos[:3] = (0, far - 1, -17)
    freq = od.rotary_frequencies(R, 10000.0)
    q, k = _values((T, H, D), act, (seed, 1)), _values((T, HK, D), act, (seed, 2))
    qd, kd = dev16(q, act, dev), dev16(k, act, dev)
    buf = None
    if layout == "slices":  # of one buffer, as a fused q/k/v product leaves them
        buf = torch.full((T, H + 2 * HK, D + 8), 9.0, dtype=TORCH_DT[act], device=dev)
        buf[:, :H, :D], buf[:, H:H + HK, 8:] = qd, kd
        qd, kd = buf[:, :H, :D], buf[:, H:H + HK, 8:]
    elif layout == "odd":  # rows at addresses of two bytes
        buf = torch.full((T, H + HK, D + 3), 9.0, dtype=TORCH_DT[act], device=dev)
        buf[:, :H, 1:D + 1], buf[:, H:, 3:] = qd, kd
        qd, kd = buf[:, :H, 1:D + 1], buf[:, H:, 3:]
    elif layout == "heads first":
        qd, kd = qd.transpose(0, 1).contiguous().transpose(0, 1), kd.transpose(0, 1).contiguous().transpose(0, 1)
    before = None if buf is None else buf.clone()
    rot = qa.Rotary(torch.from_numpy(freq).to(dev), interleaved, magnitude)
    out = qa.rotary(qd, kd, torch.from_numpy(pos).to(dev), rot, *((qd, kd) if in_place else ()))
    torch.cuda.synchronize()
    for got, x in zip(out, (q, k)):
        _same(got, *od.rotary(x, pos, freq, act, interleaved, magnitude), act)
        if R < D:
            assert np.array_equal(_host(got)[..., R:], x[..., R:])
    if before is not None:  # what lies beside the rows, and without in_place the rows themselves
        if in_place:
            qd.copy_(before[:, :H, qd.storage_offset() % buf.shape[2]:][..., :D])
            off = 8 if layout == "slices" else 3
            kd.copy_(before[:, H:H + HK, off:off + D])
        assert torch.equal(buf.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (128, 128), (128, 64), (96, 96), (96, 48), (256, 256), (256, 32), (80, 80), (40, 8),
                                 (72, 24), (30, 30), (7, 4), (2, 2), (64, 62), (1024, 1024)])
def test_head_sizes(D, R, interleaved, act):
    _check(5, 6, 2, D, R, interleaved, act, seed=D + R)


@pytest.mark.parametrize("T", [1, 2, 3, 63, 257, 1023, 2048, 5003])
@pytest.mark.parametrize("H,HK,D,R", [(32, 8, 64, 64), (5, 1, 128, 64), (3, 0, 64, 32), (0, 3, 96, 96)])
def test_lengths(T, H, HK, D, R):
    _check(T, H, HK, D, R, T % 2 == 0, "bf16" if T % 3 else "f16", seed=T)


@pytest.mark.parametrize("layout", ["dense", "slices", "odd", "heads first"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,R,interleaved", [(96, 96, False), (128, 64, False), (128, 64, True), (64, 64, True), (30, 20, False)])
def test_layouts(layout, in_place, D, R, interleaved):
    if layout == "slices" and D % 8:
        D, R = D + 2, R
    _check(300, 4, 2, D, R, interleaved, "bf16", layout=layout, in_place=in_place, seed=1)
    _check(1, 4, 2, D, R, interleaved, "f16", layout=layout, in_place=in_place, seed=2)


@pytest.mark.parametrize("far", [1 << 20, 2**31 - 1])
def test_far_positions(far):
    _check(700, 2, 1, 128, 128, False, "bf16", far=far)
    _check(700, 2, 1, 128, 128, True, "f16", far=far, magnitude=1.2079)


def test_many_heads_of_one_token():
    _check(1, 4096, 1, 128, 128, False, "bf16")
    _check(2, 300, 4096, 64, 32, True, "f16")


def test_empty():
    dev = require_gpu()
    rot = qa.Rotary.make(64, device=dev)
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device=dev)
    a, b = qa.rotary(q, q, torch.zeros(0, dtype=torch.int32, device=dev), rot)
    assert a.shape == b.shape == (0, 4, 64)


def test_values_that_are_not_finite_stay_in_their_pair():
    dev = require_gpu()
    for interleaved in (False, True):
        for act in ("bf16", "f16"):
            q = torch.ones((2, 2, 64), dtype=TORCH_DT[act], device=dev)
            q[0, 0, 3], q[0, 1, 5], q[1, 0, 60] = float("nan"), float("inf"), float("-inf")
            o, _ = qa.rotary(q, q[:, :0], torch.tensor([1, 2], dtype=torch.int32, device=dev), qa.Rotary.make(64, device=dev,
                                                                                                       interleaved=interleaved))
            bad = (~torch.isfinite(o)).nonzero().tolist()
            pair = (lambda j: j ^ 1) if interleaved else (lambda j: (j + 32) % 64)
            want = sorted([t, h, c] for t, h, j in ((0, 0, 3), (0, 1, 5), (1, 0, 60)) for c in (j, pair(j)))
            assert bad == want
            assert torch.isnan(o[0, 0, 3])


@pytest.mark.parametrize("scaling,kw", [(None, {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                        ("bands", dict(factor=8.0, original_len=8192.0)),
                                        ("bands", dict(factor=32.0, original_len=4096.0, low=1.0, high=32.0)),
                                        ("bands", dict(factor=0.5, original_len=100.0, low=0.0, high=0.25))])
@pytest.mark.parametrize("R,base", [(4, 10000.0), (64, 500000.0), (128, 10000.0), (1024, 3.0)])
def test_frequencies(scaling, kw, R, base):
    dev = require_gpu()
    got = qa.Rotary.make(R, base, scaling=scaling, device=dev, **kw).inv_freq.cpu().numpy()
    ref = od.rotary_frequencies(R, base, scaling, **kw)
    # powers of a few steps of fp64 each, an exponent's rounding times the logarithm of the base (at most 18), and the
    # slope of the bands (turns of at most original_len f over high - low, times their distance from plain)
    assert (np.abs(got - ref) <= 2.0**-46 * ref).all()


def _caches(pages, size, HK, D, G, bits, act, dev):
    made = []
    for _ in range(2):
        c = qa.AffineKVCache.empty(pages, size, HK, D, G, bits, TORCH_DT[act], dev)
        for t in c.k + c.v:
            t.view(torch.uint8).fill_(0xA5)
        made.append(c)
    return made


def _check_append(T, H, HK, D, R, G, bits, size, act, interleaved, seed=0, sliced=False, in_place=False):
    dev = require_gpu()
    print(f"[case] append T={T} H={H}/{HK} D={D} R={R} G={G} bits={bits} page={size} {act} {interleaved}", flush=True)
    rng = np.random.default_rng((seed, 5))
    pages = -(-T // size) + 2
    one, two = _caches(pages, size, HK, D, G, bits, act, dev)
    slots = rng.permutation(pages * size)[:T].astype(np.int64)
    slots[rng.random(T) < 0.2] = -1
    if T > 3:
        slots[1], slots[2] = pages * size, 2**40  # outside
    slots = torch.from_numpy(slots).to(dev)
    pos = torch.from_numpy(rng.integers(0, 1 << 20, T).astype(np.int32)).to(dev)
    qkv = dev16(_values((T, H + 2 * HK, D), act, (seed, 6)), act, dev)
    if T > 4 and act == "bf16":
        qkv[4, H, 0], qkv[4, H + HK, 1] = float("nan"), float("inf")
    q, k, v = qkv.split((H, HK, HK), 1)
    if not sliced:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    rot = qa.Rotary.make(R, interleaved=interleaved, scaling="bands", factor=8.0, original_len=8192.0, device=dev)
    want, kt = qa.rotary(q, k, pos, rot)
    qa.kv_cache_append_affine(one, kt, v, slots)
    got = qa.kv_cache_append_rotary_affine(two, q, k, v, pos, slots, rot, q_out=q if in_place else None)
    torch.cuda.synchronize()
    assert torch.equal(got.contiguous().view(torch.int16), want.view(torch.int16))
    for a, b in zip(one.k + one.v, two.k + two.v):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("D,G,R", [(32, 32, 32), (64, 32, 64), (64, 64, 32), (96, 32, 96), (96, 32, 48), (128, 64, 128),
                                   (128, 128, 64), (160, 32, 160), (192, 64, 96), (256, 128, 256)])
def test_append_rows(D, G, R, act, bits):
    _check_append(37, 6, 3, D, R, G, bits, 16, act, False, seed=D + bits)
    _check_append(37, 5, 1, D, R, G, bits, 48, act, True, seed=D + bits, sliced=True)


@pytest.mark.parametrize("T,H,HK", [(1, 32, 8), (1, 0, 3), (2, 1, 1), (16, 40, 8), (600, 3, 5), (2049, 32, 8)])
def test_append_batches(T, H, HK):
    _check_append(T, H, HK, 128, 128, 64, 4, 16, "bf16", False, seed=T)
    _check_append(T, H, HK, 96, 32, 32, 8, 64, "f16", True, seed=T, sliced=True, in_place=True)


def test_captured_on_a_fresh_stream():
    dev = require_gpu()
    rot = qa.Rotary.make(128, device=dev)
    one, two = _caches(4, 16, 2, 128, 64, 4, "f16", dev)
    q, kv = torch.randn((3, 8, 128), device=dev).half(), torch.randn((2, 3, 2, 128), device=dev).half()
    pos, slots = torch.zeros(3, dtype=torch.int32, device=dev), torch.full((3,), -1, dtype=torch.int64, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = qa.kv_cache_append_rotary_affine(one, q, *kv, pos, slots, rot)
        for i in range(5):
            pos.copy_(torch.tensor([i, 100 * i, 7], device=dev))
            slots.copy_(torch.tensor([i, 20 + i, -1 if i % 2 else 40], device=dev))
            q.normal_()
            kv.normal_()
            graph.replay()
            torch.cuda.synchronize()
            want = qa.kv_cache_append_rotary_affine(two, q, *kv, pos, slots, rot)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            for a, b in zip(one.k + one.v, two.k + two.v):
                assert torch.equal(a, b)
