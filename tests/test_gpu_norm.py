"""GPU parity of rmsnorm, rmsnorm_w4a8 and qgemm_w4a8_codes against the fp64 oracle.

Tolerances: n = (h * rstd) * w has three roundings to fp32 (rstd and two
products), each half a step, 2^-24 relative, so |n - n64| <= 2^-22 |n64|; a
dense output adds half a step of its type (2^-8 bf16, 2^-11 f16; at the
bottom of f16 half its smallest step, 2^-25).  A scale adds the rounding of
its division: 2^-22 again covers four.  A code is the nearest whole number of
n / s_x, off in the quotient by at most 127 * 2^-21."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle
import oracle.decoder as od
import synth_inputs as si
from gpu_util import TORCH_DT, dev16, host_f64, require_gpu

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": 2.0**-8, "f16": 2.0**-11}


def _inputs(M, K, act, w_dtype, seed, resid=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, :: max(1, K // 8)] *= 20.0
    r = si.store(rng.standard_normal((M, K)).astype(np.float32), act) if resid else None
    return si.store(x, act), r, si.store((1 + 0.1 * rng.standard_normal(K)).astype(np.float32), w_dtype)


def _bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def _check_dense(y, ref, act, what):
    err = np.abs(host_f64(y) - ref)
    tol = (HALF_STEP[act] + 2.0**-22) * np.abs(ref) + (2.0**-25 if act == "f16" else 0.0)
    assert (err <= tol).all(), f"{what}: {np.max(err - tol)}"


def _check_codes(x_q, s_x, ref, what):
    s_ref = np.abs(ref).max(axis=1) / 127.0
    s = host_f64(s_x)
    assert (np.abs(s - s_ref) <= 2.0**-21 * s_ref).all(), what
    q = x_q.cpu().numpy().astype(np.float64)
    exact = ref / np.where(s_ref > 0, s_ref, 1.0)[:, None]
    assert (np.abs(q - exact) <= 0.5 + 127 * 2.0**-21).all(), what
    assert (np.abs(q).max(axis=1) == np.where(s_ref > 0, 127, 0)).all(), what


def _run(M, K, act, w_dtype="f32", resid=True, eps=1e-5, seed=0):
    dev = require_gpu()
    print(f"[case] rmsnorm M={M} K={K} {act} w={w_dtype} resid={resid}", flush=True)
    x, r, w = _inputs(M, K, act, w_dtype, (60, M, K, seed), resid)
    h_ref, n_ref = od.rmsnorm(x, r, w, eps, act, w_dtype)
    xd, wd, rd = dev16(x, act, dev), dev16(w, w_dtype, dev), None if r is None else dev16(r, act, dev)
    y, h = qa.rmsnorm(xd, wd, eps, resid=rd)
    x_q, s_x, h2 = qa.rmsnorm_w4a8(xd, wd, eps, resid=rd)
    torch.cuda.synchronize()
    assert (_bits(h) == h_ref).all() and (_bits(h2) == h_ref).all()
    _check_dense(y, n_ref, act, "dense")
    _check_codes(x_q, s_x, n_ref, "codes")


@pytest.mark.parametrize("K", [1, 2, 7, 8, 31, 64, 100, 504, 512, 520, 1000, 1024, 2048, 2056, 4096, 4104, 8192, 8200, 14336,
                               16384, 16392, 16401, 40000])
def test_row_lengths(K):
    _run(3, K, "bf16", seed=1)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 17, 130])
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("resid", [False, True])
def test_rows_and_types(M, act, resid):
    _run(M, 520, act, w_dtype=act, resid=resid, seed=2)


@pytest.mark.parametrize("act,w_dtype", [("bf16", "f16"), ("f16", "bf16"), ("f16", "f32")])
def test_weight_types(act, w_dtype):
    _run(5, 2048, act, w_dtype=w_dtype, seed=3)


def test_many_rows():
    _run(2048, 1024, "f16", seed=4)


@pytest.mark.parametrize("off", [0, 1, 8])
@pytest.mark.parametrize("K", [1024, 1000, 33])
def test_row_strides_and_starts(off, K):
    # rows inside a wider buffer, at aligned and at odd starts; the buffer around them stays as it is
    dev = require_gpu()
    x, r, w = _inputs(6, K, "f16", "f16", (61, off, K))
    h_ref, n_ref = od.rmsnorm(x, r, w, 1e-5, "f16", "f16")
    wide = [torch.full((6, K + 48), 7.0, dtype=torch.float16, device=dev) for _ in range(3)]
    xs, rs, hs = (t[:, off:off + K] for t in wide)
    xs.copy_(dev16(x, "f16", dev))
    rs.copy_(dev16(r, "f16", dev))
    wd = dev16(w, "f16", dev)
    x_q, s_x, h = qa.rmsnorm_w4a8(xs, wd, resid=rs, resid_out=hs)
    y, _ = qa.rmsnorm(xs, wd, resid=rs, resid_out=hs)
    assert h is hs
    assert (_bits(hs.contiguous()) == h_ref).all()
    _check_codes(x_q, s_x, n_ref, "codes")
    _check_dense(y, n_ref, "f16", "dense")
    for t in wide:
        assert (t[:, :off] == 7).all() and (t[:, off + K:] == 7).all()


@pytest.mark.parametrize("K", [1024, 1001, 20000])
@pytest.mark.parametrize("into", ["resid", "x"])
def test_residual_updated_in_place(K, into):
    dev = require_gpu()
    x, r, w = _inputs(4, K, "bf16", "bf16", (62, K))
    h_ref, n_ref = od.rmsnorm(x, r, w, 1e-5, "bf16", "bf16")
    xd, rd = dev16(x, "bf16", dev), dev16(r, "bf16", dev)
    y, h = qa.rmsnorm(xd, dev16(w, "bf16", dev), resid=rd, resid_out=rd if into == "resid" else xd)
    assert (_bits(h) == h_ref).all()
    _check_dense(y, n_ref, "bf16", "dense")


def test_rows_of_zeros_and_of_extremes():
    dev = require_gpu()
    K = 256
    x = np.zeros((4, K), np.float32)
    x[1, 5] = 3e38          # its square passes fp32
    x[2] = 1e-38            # the squares vanish in fp32
    x[3, 0] = 1.0
    w = np.ones(K, np.float32)
    xb = si.bf16_bits(x)
    for eps in (0.0, 1e-6):
        rows = slice(1, 4) if eps == 0.0 else slice(0, 4)  # 0 / 0 in a row of zeros without eps
        _, n_ref = od.rmsnorm(xb[rows], None, w, eps, "bf16", "f32")
        y, _ = qa.rmsnorm(dev16(xb[rows], "bf16", dev), dev16(w, "f32", dev), eps)
        x_q, s_x, _ = qa.rmsnorm_w4a8(dev16(xb[rows], "bf16", dev), dev16(w, "f32", dev), eps)
        _check_dense(y, n_ref, "bf16", f"eps {eps}")
        _check_codes(x_q, s_x, n_ref, f"eps {eps}")


@pytest.mark.parametrize("K", [256, 257])
def test_nan_and_infinity_reach_their_own_row_only(K):
    dev = require_gpu()
    x, _, w = _inputs(4, K, "f16", "f16", (63, K), False)
    xd, wd = dev16(x, "f16", dev), dev16(w, "f16", dev)
    clean, _ = qa.rmsnorm(xd, wd)
    xd[1, 7] = float("nan")
    xd[3, 9] = float("inf")
    y, _ = qa.rmsnorm(xd, wd)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[2], clean[2])
    assert torch.isnan(y[1]).all()
    assert torch.isnan(y[3, 9])


def test_empty_batch():
    dev = require_gpu()
    w = torch.ones(64, dtype=torch.bfloat16, device=dev)
    y, h = qa.rmsnorm(torch.empty((0, 64), dtype=torch.bfloat16, device=dev), w)
    assert y.shape == (0, 64) and h.shape == (0, 64)


@pytest.mark.parametrize("M,N,K", [(1, 96, 64), (3, 100, 4096), (16, 260, 4128), (17, 130, 512), (130, 1024, 1024),
                                   (64, 300, 8192)])
def test_product_from_codes_equals_the_product_from_activations(M, N, K):
    # the same codes and scales give the same accumulators and outputs
    dev = require_gpu()
    c = si.w4a8_case(M, N, K, seed=(64, M, N, K))
    x = dev16(c.x, "f16", dev)
    w = torch.from_numpy(np.ascontiguousarray(c.w_q4).view(np.int32)).to(dev)
    sw = dev16(c.s_w, "f16", dev)
    y, x_q, s_x, acc = qa.qgemm_w4a8(x, w, sw, want_acc=True)
    y2, acc2 = qa.qgemm_w4a8_codes(x_q, s_x, w, sw, want_acc=True)
    y3, none = qa.qgemm_w4a8_codes(x_q, s_x, w, sw)
    torch.cuda.synchronize()
    q, s, acc_ref, y_ref = oracle.w4a8(c.x, c.w_q4, c.s_w, M, N, K)
    assert (acc2.cpu().numpy() == acc_ref).all() and torch.equal(acc, acc2)
    assert torch.equal(y2, y3) and none is None
    rep = oracle.affine_tolerance_report(host_f64(y2), y_ref)
    assert rep["ok"], rep


@pytest.mark.parametrize("K", [8, 6])
def test_more_rows_than_one_launch_takes(K):
    # 2^21 rows a launch: the rows around the cut as a call of their own has them
    dev = require_gpu()
    M, n = (1 << 21) + 5, 1 << 21
    x = torch.randn((M, K), device=dev).bfloat16()
    w = torch.randn(K, device=dev)
    y, h = qa.rmsnorm(x, w, resid=x)
    x_q, s_x, h2 = qa.rmsnorm_w4a8(x, w, resid=x)
    part = slice(n - 3, M)
    xp = x[part].contiguous()
    yp, hp = qa.rmsnorm(xp, w, resid=xp)
    qp, sp, _ = qa.rmsnorm_w4a8(xp, w, resid=xp)
    assert torch.equal(y[part], yp) and torch.equal(h[part], hp) and torch.equal(h, h2)
    assert torch.equal(x_q[part], qp) and torch.equal(s_x[part], sp)


def test_norm_refusals():
    dev = require_gpu()
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        qa.rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        qa.rmsnorm(x, w, resid=x.half())
    with pytest.raises(ValueError):
        qa.rmsnorm(x, w, resid_out=x)
    with pytest.raises(ValueError):
        qa.rmsnorm(x.t(), w[:2])
    with pytest.raises(qa.QaffError):
        qa.rmsnorm(x, w, eps=-1.0)
    with pytest.raises(qa.QaffError):  # overlapping output rows
        qa.rmsnorm(x, w, resid=x, resid_out=torch.zeros(64, dtype=torch.bfloat16, device=dev).expand(2, 64))
    with pytest.raises(ValueError):
        qa.qgemm_w4a8_codes(torch.zeros((2, 64), dtype=torch.int8, device=dev), torch.zeros(3, device=dev),
                            torch.zeros((8, 8), dtype=torch.int32, device=dev),
                            torch.zeros(8, dtype=torch.float16, device=dev))
