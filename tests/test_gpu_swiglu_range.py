"""The SwiGLU gradient over BF16's whole range: every product of a gate, a value and a gradient from
0 to the largest finite ones.  A factor that is nearly zero and two large ones give what their
product is, not inf * 0, and nothing overflows that is finite.  The forward quantizer's h likewise."""
import itertools

import numpy as np
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

pytestmark = pytest.mark.gpu

TOP = 3.3895313892515355e38   # the largest finite BF16
GATES = [0.0, 1e-38, 1e-3, 1.0, 2.4, 20.0, 60.0, 86.0, 95.0, 150.0, 1e20, 1e30, TOP]
VALUES = [0.0, 1e-38, 1e-30, 1e-10, 1.0, 1e10, 1e20, 1e30, TOP]


def inputs(dtype):
    g, u, d = np.array(list(itertools.product([s * x for x in GATES for s in (1, -1)], [s * x for x in VALUES for s in (1, -1)],
                                              VALUES)), np.float64).T
    n = -(-g.size // 64) * 64
    g, u, d = (torch.from_numpy(np.pad(x, (0, n - x.size))).reshape(-1, 64) for x in (g, u, d))
    return torch.cat([g, u], 1).to(torch.bfloat16).cuda(), d.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extremes(dtype):
    gu, dh = inputs(dtype)
    dgu, h = fq.fp8q_swiglu_backward(gu, dh, want_h=True)
    torch.cuda.synchronize()
    g, u = gu.double().cpu().numpy()[:, :64], gu.double().cpu().numpy()[:, 64:]
    d = dh.double().cpu().numpy()
    t = np.exp(-np.abs(g))
    s, c = np.where(g >= 0, 1.0, t) / (1 + t), np.where(g >= 0, t, 1.0) / (1 + t)
    f = s * (1 + g * c)
    got = dgu.double().cpu().numpy()
    # At most 16 half-steps of FP32 and BF16's half step; s and what it is multiplied with
    # first lose up to 2^-149 below FP32's normal range, which the other factors then scale; and half
    # a step of BF16's subnormals.
    low = 4 * 2.0 ** -149
    for what, x, ref, big, lost in (
            ("h", h.double().cpu().numpy(), g * s * u, np.abs(g * s * u), np.abs(u) * (1 + np.abs(g))),
            ("du", got[:, 64:], d * g * s, np.abs(d * g * s), np.abs(d) * (1 + np.abs(g))),
            ("dg", got[:, :64], d * u * f, np.abs(d * u) * s * (1 + np.abs(g) * c), np.abs(d * u) * (1 + np.abs(g)))):
        assert not np.isnan(x).any(), f"{what}: {int(np.isnan(x).sum())} of {x.size} are NaN"
        tol = 16 * 2.0 ** -24 * big * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + low * lost + 2.0 ** -133
        # beyond the largest BF16 and half a step: inf, or the largest within the error
        over = np.abs(ref) - tol > TOP
        assert np.all(np.isinf(x[over]) & (np.sign(x[over]) == np.sign(ref[over]))), f"{what}: finite where it is past BF16"
        inside = np.abs(ref) + tol < TOP
        err = np.abs(x[inside] - ref[inside])
        worst = np.argmax(err - tol[inside])
        assert np.all(err <= tol[inside]), f"{what}: {x[inside][worst]} for {ref[inside][worst]}"


def test_forward_of_a_closed_gate():
    """Tiles in which the product of gate and value passes FP32 where h does not: h of 0 beside ordinary
    ones, and h of a half-closed gate, whose codes are those of h."""
    g = torch.full((4, 128), 1.5)
    u = torch.linspace(-2, 2, 128).repeat(4, 1)
    g[0, 3], u[0, 3] = -1e20, 1e20                       # h = 0
    g[1, :], u[1, :] = -3e38, torch.linspace(1e38, 3e38, 128)
    g[2, 7], u[2, 7] = -50.0, 3e37                       # h = -2.9e17 where g u is past FP32
    gu = torch.cat([g, u], 1).to(torch.bfloat16).cuda()
    xq, sa = fq.fp8q_swiglu_quantize_act_1x128(gu)
    torch.cuda.synchronize()
    x = gu.double().cpu().numpy()
    with np.errstate(over="ignore"):
        h = x[:, :128] * x[:, 128:] / (1 + np.exp(-x[:, :128]))
    scale = sa[0].double().cpu().numpy()
    # a few ulps of the largest h over 448
    assert np.all(np.abs(scale * 448 - np.abs(h).max(1)) <= 2.0 ** -20 * np.abs(h).max(1)), scale
    got = xq.view(torch.float8_e4m3fn).double().cpu().numpy() * scale[:, None]
    # half a step of E4M3, normal or subnormal, beside h's own ulps
    tol = (2.0 ** -4 + 2.0 ** -20) * np.abs(h) + 2.0 ** -10 * scale[:, None]
    assert np.all(np.abs(got - h) <= tol)
