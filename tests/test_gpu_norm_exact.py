"""rmsnorm and rmsnorm_w4a8 bit for bit against their definition: rstd from
fp64 rounded once, every other step one IEEE fp32 operation (numpy's).  The
order of the kernel's fp64 sum is its own, so rows whose rstd lies within
2^-10 of a step from a rounding boundary are left out; K squares sum to
within K 2^-53 of their size whatever the order, 2^-15 of a step at K = 16384."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle
import oracle.decoder as od
import synth_inputs as si
from gpu_util import dev16, require_gpu

pytestmark = pytest.mark.gpu
F = np.float32


def _definition(h, w, eps):
    """(rows whose rstd is certain, n f32, s_x f32, x_q) from h and w as fp64 values of their types."""
    exact = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    rstd = exact.astype(F)
    step = np.spacing(rstd).astype(np.float64)
    sure = np.abs(np.abs(exact - rstd.astype(np.float64)) / step - 0.5) > 2.0**-10
    n = (h.astype(F) * rstd[:, None]) * w.astype(F)
    s = np.abs(n).max(axis=1) / F(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s[:, None] > 0, np.rint(n / s[:, None]), F(0))
    return sure, n, s, np.clip(q, -127, 127).astype(np.int8)


def _bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def _check(x, r, w, act, w_dtype, eps):
    dev = require_gpu()
    h_ref, _ = od.rmsnorm(x, r, w, eps, act, w_dtype)
    sure, n, s, q = _definition(oracle.to_f64(h_ref, act), oracle.to_f64(w, w_dtype), eps)
    assert sure.mean() > 0.9
    xd, wd, rd = dev16(x, act, dev), dev16(w, w_dtype, dev), None if r is None else dev16(r, act, dev)
    y, h = qa.rmsnorm(xd, wd, eps, resid=rd)
    x_q, s_x, h2 = qa.rmsnorm_w4a8(xd, wd, eps, resid=rd)
    torch.cuda.synchronize()
    assert (_bits(h) == h_ref).all() and (_bits(h2) == h_ref).all()
    assert (_bits(y) == si.store(n, act))[sure].all()
    assert (s_x.cpu().numpy() == s)[sure].all()
    assert (x_q.cpu().numpy() == q)[sure].all()


@pytest.mark.parametrize("K", [64, 500, 512, 1024, 2048, 4096, 8192, 14336, 16384, 16392, 7, 1001])
@pytest.mark.parametrize("act,w_dtype", [("bf16", "bf16"), ("f16", "f32"), ("f16", "bf16")])
def test_every_output(K, act, w_dtype):
    print(f"[case] rmsnorm exact K={K} {act} {w_dtype}", flush=True)
    rng = np.random.default_rng((65, K))
    x = rng.standard_normal((40, K)).astype(F) * np.exp(rng.uniform(-3, 3, (40, 1))).astype(F)
    x[:, :: max(1, K // 8)] *= 20
    w = si.store((1 + 0.1 * rng.standard_normal(K)).astype(F), w_dtype)
    r = si.store(rng.standard_normal((40, K)).astype(F), act) if K % 3 else None
    _check(si.store(x, act), r, w, act, w_dtype, 1e-5)


@pytest.mark.parametrize("K", [1784, 1785, 2048, 8192])
def test_codes_next_to_a_half(K):
    # rows of +-1, whose rstd is 1: n is +-weight.  The weights are (k + 1/2) s for every k, and up to three steps of fp32
    # on either side, so that the fp32 quotient decides the code; scales of many magnitudes
    rng = np.random.default_rng((66, K))
    x = si.f16_bits(rng.choice([-1.0, 1.0], (2, K)).astype(F))
    for e in (-100, -91, -89, -20, -1, 0, 1, 3, 30, 80, 89, 92, 110):
        top = F(127) * F(rng.uniform(1, 2) * 2.0**e)
        w = [((np.arange(-127, 127) + 0.5) * np.float64(top / F(127))).astype(F)]
        for side in (np.inf, -np.inf):
            v = w[0]
            for _ in range(3):
                v = np.nextafter(v, F(side))
                w.append(v)
        w = np.concatenate(w)
        w = np.concatenate([[top], w, top * rng.uniform(-1, 1, K).astype(F)])[:K].astype(F)
        assert len(w) == K and np.abs(w).max() == top
        print(f"[case] codes K={K} scale 2^{e}", flush=True)
        _check(x, None, rng.permutation(w).astype(F), "f16", "f32", 0.0)
