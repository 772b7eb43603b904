"""GPU tests of kv_cache_append_affine (bit for bit the rows that the oracle's
quantize_pack_affine gives) and kv_cache_read_affine (code * scale + bias
rounded to fp32, then to the type: exact)."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle.decoder as od
import synth_inputs as si
from gpu_util import TORCH_DT, dev16, require_gpu

pytestmark = pytest.mark.gpu


def _host(t):
    t = t.cpu()
    return t.numpy().view(np.uint32) if t.dtype == torch.int32 else t.view(torch.int16).numpy().view(np.uint16)


def _rows(T, H, D, act, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, D)) * np.exp(rng.uniform(-3, 3, (T, H, 1)))
    x[0, 0] = x[0, 0, 0]  # a row of one value: scale 0
    return si.store(x.astype(np.float32), act)


def _fill(cache, byte):
    for t in cache.k + cache.v:
        t.view(torch.uint8).fill_(byte)


def _check(T, H, D, G, bits, size, pages, act, seed, slots=None, strided=False):
    dev = require_gpu()
    print(f"[case] kv T={T} H={H} D={D} G={G} bits={bits} page={size} {act}", flush=True)
    rng = np.random.default_rng((seed, 1))
    if slots is None:
        slots = rng.permutation(pages * size)[:T]
    slots = np.asarray(slots, np.int64)
    k, v = _rows(T, H, D, act, (seed, 2)), _rows(T, H, D, act, (seed, 3))
    cache = qa.AffineKVCache.empty(pages, size, H, D, G, bits, TORCH_DT[act], dev)
    _fill(cache, 0xA5)
    before = [_host(t).copy() for t in cache.k + cache.v]
    kd, vd = dev16(k, act, dev), dev16(v, act, dev)
    if strided:  # slices of one buffer, as a fused q/k/v product leaves them
        qkv = torch.full((T, 3 * H, D + 8), 9.0, dtype=TORCH_DT[act], device=dev)
        qkv[:, H:2 * H, :D], qkv[:, 2 * H:, 8:] = kd, vd
        kd, vd = qkv[:, H:2 * H, :D], qkv[:, 2 * H:, 8:]
    sd = torch.from_numpy(slots).to(dev)
    qa.kv_cache_append_affine(cache, kd, vd, sd)
    ko, vo = qa.kv_cache_read_affine(cache, sd)
    torch.cuda.synchronize()
    ok = (slots >= 0) & (slots < pages * size)
    pg, off = slots[ok] // size, slots[ok] % size
    for x, arrays, old, got in ((k, cache.k, before[:3], ko), (v, cache.v, before[3:], vo)):
        want = od.quantize_rows(x[ok], act, G, bits)
        for part, (t, w) in enumerate(zip(arrays, want)):
            expect = old[part].copy()
            expect[pg, :, off] = w
            assert (_host(t) == expect).all(), f"array {part}"  # the named rows, and every other as it was
        ref = np.zeros((T, H, D), np.uint16)
        ref[ok] = si.store(od.values(*want, act, G, bits).astype(np.float32), act)
        assert (_host(got) == ref).all(), "read"


@pytest.mark.parametrize("D,G", [(32, 32), (64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 64),
                                 (224, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_layouts_and_types(D, G, bits, act):
    _check(21, 3, D, G, bits, 16, 3, act, (70, D, G, bits))


@pytest.mark.parametrize("T,H,size,pages", [(1, 1, 16, 1), (1, 8, 16, 4), (2, 5, 48, 2), (100, 7, 64, 5), (1000, 2, 80, 13),
                                            (4096, 8, 128, 33)])
def test_sizes(T, H, size, pages):
    _check(T, H, 128, 64, 4, size, pages, "bf16", (71, T))


@pytest.mark.parametrize("bits", [4, 8])
def test_strided_inputs(bits):
    _check(33, 2, 64, 64, bits, 16, 4, "f16", (72, bits), strided=True)


def test_slots_outside_are_skipped_and_read_as_zeros():
    # padding, past the end, the far ends of int64 and what 32 bits would fold back into range
    slots = [-1, 5, 2 * 16, (1 << 32) + 3, -(1 << 63), (1 << 63) - 1, 31, -(1 << 32) + 1, 0]
    _check(9, 2, 64, 32, 4, 16, 2, "bf16", (73,), slots=slots)


def test_broadcast_rows():
    # one head's rows for every head (a head stride of 0)
    dev = require_gpu()
    x = _rows(4, 1, 64, "bf16", (74,))
    one = dev16(x, "bf16", dev)
    cache = qa.AffineKVCache.empty(1, 16, 3, 64, 64, 8, torch.bfloat16, dev)
    sd = torch.arange(4, device=dev)
    qa.kv_cache_append_affine(cache, one.expand(4, 3, 64), one.expand(4, 3, 64), sd)
    k, v = qa.kv_cache_read_affine(cache, sd)
    w = od.quantize_rows(x, "bf16", 64, 8)
    ref = si.store(od.values(*w, "bf16", 64, 8).astype(np.float32), "bf16")
    for t in (k, v):
        assert (_host(t) == np.broadcast_to(ref, (4, 3, 64))).all()


def test_infinite_and_subnormal_values():
    dev = require_gpu()
    x = np.zeros((4, 1, 32), np.float32)
    x[0, 0, 3] = np.inf
    x[1, 0] = np.linspace(-65504, 65504, 32)
    x[2, 0] = np.arange(32) * 2.0**-24
    xb = si.f16_bits(x)
    cache = qa.AffineKVCache.empty(1, 16, 1, 32, 32, 4, torch.float16, dev)
    sd = torch.arange(4, device=dev)
    xd = dev16(xb, "f16", dev)
    qa.kv_cache_append_affine(cache, xd, xd, sd)
    torch.cuda.synchronize()
    w = od.quantize_rows(xb, "f16", 32, 4)
    for t, ref in zip(cache.k, w):
        assert (_host(t)[0, 0, 1:4] == ref[1:4, 0]).all()
    assert np.isinf(cache.k[1][0, 0, 0, 0].item())


def test_cache_past_4_gib():
    # the last page's rows lie beyond 32-bit byte offsets
    dev = require_gpu()
    pages, size, H, D = 70000, 64, 8, 128
    k = (torch.empty((pages, H, size, D), dtype=torch.int8, device=dev).view(torch.int32),
         torch.zeros((pages, H, size, 2), dtype=torch.float16, device=dev),
         torch.zeros((pages, H, size, 2), dtype=torch.float16, device=dev))
    assert k[0].numel() * 4 > 1 << 32
    cache = qa.AffineKVCache(k, k, 64, 8)
    x = _rows(3, H, D, "f16", (75,))
    slots = torch.tensor([pages * size - 1, (pages - 1) * size, 0], device=dev)
    xd = dev16(x, "f16", dev)
    qa.kv_cache_append_affine(cache, xd, xd, slots)
    ko, vo = qa.kv_cache_read_affine(cache, slots)
    w = od.quantize_rows(x, "f16", 64, 8)
    ref = si.store(od.values(*w, "f16", 64, 8).astype(np.float32), "f16")
    assert (_host(ko) == ref).all() and (_host(vo) == ref).all()
    assert (_host(k[0][-1, :, -1]) == w[0][0]).all()


def test_reads_repeat_a_slot_and_take_given_outputs():
    dev = require_gpu()
    cache = qa.AffineKVCache.empty(2, 16, 2, 64, 64, 4, torch.bfloat16, dev)
    x = dev16(_rows(2, 2, 64, "bf16", (76,)), "bf16", dev)
    qa.kv_cache_append_affine(cache, x, x, torch.tensor([3, 17], device=dev))
    outs = tuple(torch.empty((5, 2, 64), dtype=torch.bfloat16, device=dev) for _ in range(2))
    k, v = qa.kv_cache_read_affine(cache, torch.tensor([3, 3, 17, 3, 17], device=dev), out=outs)
    assert k is outs[0] and v is outs[1]
    assert torch.equal(k[0], k[1]) and torch.equal(k[0], k[3]) and torch.equal(k[2], k[4]) and not torch.equal(k[0], k[2])


def test_empty_calls():
    dev = require_gpu()
    cache = qa.AffineKVCache.empty(1, 16, 2, 64, 64, 4, torch.bfloat16, dev)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=dev)
    slots = torch.empty(0, dtype=torch.int64, device=dev)
    qa.kv_cache_append_affine(cache, none, none, slots)
    assert qa.kv_cache_read_affine(cache, slots)[0].shape == (0, 2, 64)


def test_python_refusals():
    dev = require_gpu()
    cache = qa.AffineKVCache.empty(1, 16, 2, 64, 64, 4, torch.bfloat16, dev)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device=dev)
    s = torch.zeros(3, dtype=torch.int64, device=dev)
    for bad in ((x[:2], x, s), (x, x.half(), s), (x, x, s.int()), (x, x[..., :32], s), (x.cpu(), x, s),
                (x.transpose(1, 2).contiguous().transpose(1, 2), x, s)):
        with pytest.raises(ValueError):
            qa.kv_cache_append_affine(cache, *bad)
    with pytest.raises(qa.QaffError):  # rows off the 16-byte grid
        qa.kv_cache_append_affine(cache, torch.zeros((3, 2, 72), dtype=torch.bfloat16, device=dev)[..., 4:68], x, s)
    with pytest.raises(ValueError):
        qa.kv_cache_read_affine(cache, s, out=(x.half(), x))


@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_codes_are_the_ieee_quotients(bits, act):
    # two million values a case in groups of every magnitude (the reciprocal's ends included), short significands that
    # give exact ties, and groups of one value apart from the rest
    dev = require_gpu()
    rng = np.random.default_rng((77, bits))
    T, H, D, G = 4096, 4, 128, 32
    x = rng.standard_normal((T, H, D // G, G))
    x[: T // 4] = np.round(x[: T // 4] * 4) / 4
    x[T // 4: T // 2] *= rng.integers(1, 64, (T // 4, H, D // G, 1))
    x[T // 2: T // 2 + 256, :, :, 0] *= 1000
    lim = 30 if act == "bf16" else 4
    scale = np.exp2(rng.uniform(-lim, lim, (T, H, D // G, 1)))
    if act == "bf16":
        scale[-512:] = np.exp2(rng.uniform(-130, 124, (512, H, D // G, 1)))
    x = si.store((x * scale).reshape(T, H, D).astype(np.float32), act)
    cache = qa.AffineKVCache.empty(T // 16, 16, H, D, G, bits, TORCH_DT[act], dev)
    xd = dev16(x, act, dev)
    qa.kv_cache_append_affine(cache, xd, xd, torch.arange(T, device=dev))
    for t, ref in zip(cache.k, od.quantize_rows(x, act, G, bits)):
        got = _host(t).transpose(0, 2, 1, 3).reshape(T, H, -1)
        assert (got == ref).all()
