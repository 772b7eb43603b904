"""Values read back from the cache where bits are easily lost: scales and
biases of any size, against the definition (code * scale + bias rounded to
fp32, then to the type)."""
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
