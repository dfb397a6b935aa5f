"""The range of Newton-Schulz coefficients that include/fp8q.h states, without a GPU: by the model of the kernels' roundings,
and by the refusal of an a that FP16 does not hold."""
import ctypes
import os
import re

import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
from test_gpu_muon import by_products

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = {k: int(v) for k, v in re.findall(r"\b(FP8Q_[A-Z0-9_]+)\s*=\s*(-?\d+)", open(os.path.join(ROOT, "include", "fp8q.h")).read())}
A = 1 << 20  # a fake, 16-byte aligned device address (never dereferenced)

# (coefficients, steps) that lead two equal rows, whose A_01 is s^2 / 2, to the edges: s = 5.64 before the last step; C = 15.98 on
# its diagonal, with either sign; C_01 = 15.9 / 2; s = 1 kept by a large a (one step: at s = 1 another one multiplies an error by
# |a + 3 b| = 28.8, so that 2^-12 of C_01 = 7.45 grows to 5 % after two and to 150 % after three)
INSIDE = [((5.64, 0.0, 0.0), 2), ((15.98, 0.0, 0.0), 1), ((-15.98, 0.0, 0.0), 1), ((0.0, 15.9, 0.0), 1), ((15.9, -14.9, 0.0), 1)]
OUTSIDE = [((5.67, 0.0, 0.0), 2), ((8.0, -0.1, 0.0), 2), ((3.0, 0.0, 0.0), 3)]


def equal_rows(device="cpu"):
    x = torch.randn((1, 64), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    return torch.cat([x, x]).to(device)


@pytest.mark.parametrize("abc,steps", INSIDE)
def test_model_inside(abc, steps):
    """Off by three halves of FP16's step, 2^-12, of what C_01 brings, a step: its rounding, the row's factor d / dh, which it is
    multiplied by too, and the rest lo, which it is not multiplied with; C_01 is 7.45 beside a result of 1 in the last case and
    no larger than the result in the others."""
    e, m = (by_products(equal_rows(), steps, abc, rounded=r) for r in (False, True))
    c01 = abs(abc[1] / 2 / sum(abc)) if steps == 1 else 1.0
    assert (m - e).norm() <= steps * 3 * 2.0 ** -12 * max(1.0, c01) * e.norm()


@pytest.mark.parametrize("abc,steps", OUTSIDE)
def test_model_outside(abc, steps):
    assert not torch.isfinite(by_products(equal_rows(), steps, abc, rounded=True)).all()


@pytest.mark.parametrize("a,status", [(15.99, "FP8Q_ERR_NULL"), (-15.99, "FP8Q_ERR_NULL"), (16.0, "FP8Q_ERR_VALUE"),
                                      (-16.0, "FP8Q_ERR_VALUE"), (1e30, "FP8Q_ERR_VALUE")])
def test_a_that_fp16_does_not_hold(a, status):
    """Before any HIP call; a valid a gets as far as the missing workspace."""
    lib, ns = fq.load_library(), fq._NewtonSchulz(a, -4.7, 2.0, 5)
    assert lib.fp8q_orthogonalize(A, 0, 1, 8, 16, ctypes.byref(ns), A, 0, None) == E[status]
    h = fq._MuonHyper(1e-3, 0.95, 0.1, 1.0, 1.0, ns, 1, None)
    assert lib.fp8q_muon(A, A, 1, A, 1, 8, 16, ctypes.byref(h), 0, 0, None) == E[status]
