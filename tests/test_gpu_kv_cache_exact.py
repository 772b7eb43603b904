"""The cache's rows where bits are easily lost: values read back from scales
and biases of any size against the definition (code * scale + bias rounded to
fp32, then to the type), and rows that hold NaN, infinities and zeros of both
signs against quantize_pack_affine of the same rows."""
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


@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_values_of_scales_and_biases_of_any_size(bits, act):
    # a million values: sums that fp32 rounds, some of them to the middle between two values of the type
    dev = require_gpu()
    rng = np.random.default_rng((78, bits))
    pages, H, size, D, G = 64, 4, 32, 128, 32
    rows = (pages, H, size)
    trip = []
    for _ in range(2):
        s = np.exp2(rng.uniform(-9, 3, (*rows, D // G)))
        b = rng.standard_normal((*rows, D // G)) * s * np.exp2(rng.uniform(-4, 10, (*rows, D // G)))
        trip.append((rng.integers(0, 1 << 32, (*rows, D * bits // 32), dtype=np.uint32),
                     *(si.store(x.astype(np.float32), act) for x in (s, b))))
    dt = TORCH_DT[act]
    cache = qa.AffineKVCache(*[(torch.from_numpy(t[0].view(np.int32)).to(dev), dev16(t[1], act, dev), dev16(t[2], act, dev))
                               for t in trip], G, bits)
    assert cache.dtype == dt
    slots = torch.arange(pages * size, device=dev)
    for got, t in zip(qa.kv_cache_read_affine(cache, slots), trip):
        ref = si.store(od.values(*t, act, G, bits).astype(np.float32), act)
        got = _host(got).reshape(pages, size, H, D).transpose(0, 2, 1, 3)
        assert (got == ref).all(), int((got != ref).sum())


@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_rows_that_are_not_finite_or_zero(bits, G, act):
    dev = require_gpu()
    D, T = 128, 256
    rng = np.random.default_rng((79, G, bits))
    x = si.store(rng.standard_normal((T, 1, D)).astype(np.float32), act)
    inf, quiet, signal = (0x7F80, 0x7FC0, 0x7F81) if act == "bf16" else (0x7C00, 0x7E00, 0x7C01)
    pick = lambda vals, shape: rng.choice(np.array(vals, np.uint16), shape)
    x[0:32, 0, ::7] = pick([quiet, quiet | 0x8000, signal, signal | 0x8000], x[0:32, 0, ::7].shape)
    x[32:64, 0, 5::40] = pick([inf, inf | 0x8000], x[32:64, 0, 5::40].shape)
    x[64:80, 0, ::9] = pick([inf, inf | 0x8000, quiet, signal | 0x8000], x[64:80, 0, ::9].shape)
    x[80], x[81], x[82], x[83] = quiet, signal, inf, inf | 0x8000
    x[84:116] = pick([0, 0x8000], x[84:116].shape)                 # zeros of both signs
    x[116:160] &= 0x7FFF                                            # a minimum that is a zero of either sign
    x[116:160, 0, ::5] = pick([0, 0x8000], x[116:160, 0, ::5].shape)
    x[160:200] |= 0x8000                                            # and a maximum
    x[160:200, 0, ::5] = pick([0, 0x8000], x[160:200, 0, ::5].shape)
    x[200:232] = pick([1, 0x8001, 0, 0x8000, 3], x[200:232].shape)  # subnormals
    xd = dev16(x, act, dev)
    cache = qa.AffineKVCache.empty(T // 16, 16, 1, D, G, bits, TORCH_DT[act], dev)
    qa.kv_cache_append_affine(cache, xd, xd, torch.arange(T, device=dev))
    # a signaling NaN counts as a quiet one
    calm = np.where((x & 0x7FFF) == signal, x ^ signal ^ quiet, x)
    want = qa.quantize_pack_affine(dev16(calm, act, dev)[:, 0], G, bits, TORCH_DT[act])
    for arrays in (cache.k, cache.v):
        for got, ref in zip(arrays, want):
            same = (_host(got).reshape(T, -1) == _host(ref)).all(axis=1)
            assert same.all(), np.nonzero(~same)[0]
