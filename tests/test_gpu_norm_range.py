"""Norms of rows at the ends of FP32's range, as include/fp8q.h states them, beside ordinary rows."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

pytestmark = pytest.mark.gpu


def rows(H):
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn((6, H), device="cuda", generator=g)
    return x, 1.0 + 0.1 * torch.randn(H, device="cuda", generator=g), torch.randn(H, device="cuda", generator=g)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("H", [64, 1000, 8200])
def test_squares_that_fp32_does_not_hold(H, center):
    x, w, b = rows(H)
    want, _, _ = fq.fp8q_layer_norm(x, w, b, center=center)
    x[2] *= 1e20
    x[4, 3] = 2e19  # one value is enough
    for bias in (b, None):
        y, mean, rstd = fq.fp8q_layer_norm(x, w, bias, center=center)
        for row in (2, 4):
            assert rstd[row] == 0 and torch.equal(y[row], torch.zeros_like(b) if bias is None else b)
        if bias is not None:
            assert torch.equal(y[[0, 1, 3, 5]], want[[0, 1, 3, 5]])
    dx, dw, db = fq.fp8q_layer_norm_backward(torch.ones_like(x), x, w, mean, rstd, want_bias=True)
    assert not dx[[2, 4]].any() and torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("H", [64, 1000, 8200])
def test_sums_that_fp32_does_not_hold(H):
    x, w, b = rows(H)
    want, _, _ = fq.fp8q_layer_norm(x, w, b)
    x[2] = 3e38
    y, mean, rstd = fq.fp8q_layer_norm(x, w, b)
    assert torch.isinf(mean[2]) and torch.isnan(y[2]).all() and torch.equal(y[[0, 1, 3, 4, 5]], want[[0, 1, 3, 4, 5]])


def test_squares_that_vanish():
    x, w, b = rows(64)
    x[1], x[3] = 0.0, x[3] * 1e-25
    y, _, rstd = fq.fp8q_layer_norm(x, w, b, center=False)
    # eps alone: 1 / sqrt(1e-5), and values of 1e-22 vanish beside the bias
    assert rstd[1] == rstd[3] and torch.equal(y[1], b) and torch.equal(y[3], b)
    y, _, rstd = fq.fp8q_layer_norm(x, w, b, center=False, eps=0.0)
    assert torch.isinf(rstd[[1, 3]]).all() and not torch.isfinite(y[[1, 3]]).any() and torch.isfinite(y[[0, 2, 4, 5]]).all()
