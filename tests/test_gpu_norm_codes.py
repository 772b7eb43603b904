"""rmsnorm_w4a8 on values that are not finite: the row's scale is not finite
either, its codes keep to [-127, 127], and the product that takes them is not
finite in that row and untouched in the others."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def _inputs(M, K, seed):
    dev = require_gpu()
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((M, K), generator=g, device=dev)
    return x, 1 + 0.1 * torch.randn(K, generator=g, device=dev), g


# K: rows in registers of one wave to sixteen, and the kernel for any K
KS = [64, 512, 1024, 2048, 4096, 8192, 16384, 100, 513, 16392]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("act", [torch.float16, torch.bfloat16])
def test_a_row_that_is_not_finite(act, K, bad):
    x, w, _ = _inputs(5, K, 1)
    x = x.to(act)
    clean = qa.rmsnorm_w4a8(x, w)
    for at in (0, K // 2, K - 1):
        y = x.clone()
        y[3, at] = bad
        x_q, s_x, h = qa.rmsnorm_w4a8(y, w)
        torch.cuda.synchronize()
        assert torch.isnan(s_x[3])
        assert x_q[3].to(torch.int32).abs().max() <= 127
        for r in (0, 1, 2, 4):
            assert torch.equal(x_q[r], clean[0][r]) and s_x[r] == clean[1][r]
        # by way of the residual
        z = torch.zeros_like(x)
        z[3, at] = bad
        x_q2, s_x2, _ = qa.rmsnorm_w4a8(x, w, resid=z)
        assert torch.isnan(s_x2[3]) and torch.equal(s_x2[:3], s_x[:3]) and torch.equal(x_q2[:3], x_q[:3])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("K", KS)
def test_a_weight_that_is_not_finite(K, bad):
    x, w, _ = _inputs(3, K, 2)
    w[K // 3] = bad
    x_q, s_x, _ = qa.rmsnorm_w4a8(x.half(), w)
    torch.cuda.synchronize()
    assert (torch.isnan(s_x) if bad != bad else torch.isinf(s_x)).all()
    assert x_q.to(torch.int32).abs().max() <= 127


@pytest.mark.parametrize("M,N,K", [(1, 96, 512), (3, 100, 4096), (16, 260, 4128), (17, 130, 512), (130, 1024, 1024),
                                   (64, 300, 8192)])
def test_the_product_of_such_a_row_is_not_finite(M, N, K):
    x, w, g = _inputs(M, K, 3)
    w_q4, s_w = qa.w4a8_quantize_weights(torch.randn((N, K), generator=g, device=x.device))
    x = x.half()
    clean, _ = qa.qgemm_w4a8_codes(*qa.rmsnorm_w4a8(x, w)[:2], w_q4, s_w)
    x[M // 2, K // 5] = float("nan")
    y, _ = qa.qgemm_w4a8_codes(*qa.rmsnorm_w4a8(x, w)[:2], w_q4, s_w)
    torch.cuda.synchronize()
    others = torch.arange(M, device=x.device) != M // 2
    assert torch.isnan(y[M // 2]).all() and torch.equal(y[others], clean[others])


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("K", KS)
def test_a_row_of_zeros(K, eps):
    x, w, _ = _inputs(3, K, 4)
    x[1] = 0
    x[1, ::2] = -0.0
    x_q, s_x, _ = qa.rmsnorm_w4a8(x.half(), w, eps)
    torch.cuda.synchronize()
    assert s_x[1] == 0 and (x_q[1] == 0).all() and (s_x[[0, 2]] > 0).all()
