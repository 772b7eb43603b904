"""Pins of the fp64 definitions in oracle/decoder.py, by closed forms."""
import numpy as np
import pytest
import torch

import oracle
import oracle.decoder as od
import synth_inputs as si


def test_rmsnorm_of_a_constant_row_is_its_sign_times_the_weight():
    x = si.bf16_bits(np.array([[2.0] * 8, [-4.0] * 8]))
    w = np.arange(1, 9, dtype=np.float32)
    h, n = od.rmsnorm(x, None, w, 0.0, "bf16", "f32")
    assert (h == x).all()
    np.testing.assert_allclose(n, [w, -w], rtol=1e-15)


def test_rmsnorm_adds_the_residual_and_rounds_the_sum_once():
    x, r = si.bf16_bits(np.array([[256.0, 1.0]])), si.bf16_bits(np.array([[1.0, 1.0]]))
    h, n = od.rmsnorm(x, r, np.ones(2, np.float32), 0.0, "bf16", "f32")
    hv = oracle.to_f64(h, "bf16")
    assert hv.tolist() == [[256.0, 2.0]]  # 257 is a tie of bf16, to even
    np.testing.assert_allclose((n * n).mean(), 1.0, rtol=1e-15)


@pytest.mark.parametrize("bits", [2, 4, 8])
def test_cache_rows_round_trip_values_on_the_grid(bits):
    # values scale * code + bias with both ends present and exact scale and bias come back exactly
    rng = np.random.default_rng(7)
    c = rng.integers(0, 2**bits, (3, 2, 64))
    c[..., ::32], c[..., 1::32] = 0, 2**bits - 1
    x = si.f16_bits(0.25 * c - 2.0)
    w, s, b = od.quantize_rows(x, "f16", 32, bits)
    assert (od.codes(w, bits) == c).all()
    assert (od.values(w, s, b, "f16", 32, bits) == 0.25 * c - 2.0).all()


def _cache(rng, pages, kvh, size, D, G, bits, dt):
    return tuple(od.quantize_rows(si.store(rng.standard_normal((pages, kvh, size, D)).astype(np.float32), dt), dt, G, bits)
                 for _ in range(2))


def test_attention_equals_torch_softmax_attention_in_float64():
    rng = np.random.default_rng(8)
    k, v = _cache(rng, 6, 2, 16, 64, 32, 4, "bf16")
    q = si.bf16_bits(rng.standard_normal((1, 4, 64)))
    table = np.array([[4, 0, 5]], np.int32)
    out, bound = od.paged_attention(q, k, v, "bf16", 32, 4, table, [41], 0.125)
    kd, vd = (torch.from_numpy(od.values(*t, "bf16", 32, 4)[table[0]].transpose(1, 0, 2, 3).reshape(2, 48, 64)[:, :41].copy())
              for t in (k, v))
    qd = torch.from_numpy(oracle.to_f64(q, "bf16")).view(2, 2, 64)
    ref = torch.softmax(0.125 * qd @ kd.transpose(1, 2), -1) @ vd
    np.testing.assert_allclose(out[0], ref.view(4, 64).numpy(), rtol=1e-12, atol=1e-13)
    assert (bound > 0).all() and (bound < 0.05).all()


def test_attention_masks():
    rng = np.random.default_rng(9)
    k, v = _cache(rng, 4, 1, 16, 64, 64, 8, "f16")
    q = si.f16_bits(rng.standard_normal((4, 1, 64)))
    table = np.array([[1, 2], [1, 2], [-1, 4], [3, 9]], np.int32)
    out, _ = od.paged_attention(q, k, v, "f16", 64, 8, table, [0, 20, 32, 40], 0.125, window=1)
    vv = od.values(*v, "f16", 64, 8)
    assert (out[0] == 0).all()                       # no token
    np.testing.assert_allclose(out[1, 0], vv[2, 0, 3], rtol=1e-14)   # the newest token alone
    assert (out[2] == 0).all() and (out[3] == 0).all()  # pages outside the cache
