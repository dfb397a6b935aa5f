"""Newton-Schulz coefficients at the edges of the range that include/fp8q.h states, and elements of X above one."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
from test_gpu_muon import allowed
from test_muon_range import INSIDE, equal_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("abc,steps", INSIDE)
@pytest.mark.parametrize("tall", [False, True])
def test_inside(abc, steps, tall):
    x = equal_rows("cuda").float()
    x = x.t().contiguous() if tall else x
    e, norm, inside = allowed(x, steps, abc)
    p, m = torch.zeros_like(x), torch.zeros_like(x)
    fq.fp8q_muon(p, x, m, lr=1.0, scale=1.0, nesterov=False, steps=steps, coefficients=abc)
    assert torch.isfinite(p).all() and (-p.double() - e).norm() <= inside


@pytest.mark.parametrize("shape", [(1, 1), (1, 3), (4, 1)])
def test_elements_above_one(shape):
    """A single large element: X_ij up to 5.6, where hi has 11 bits and lo saturates, so X is off by 2^-12 a step at the most."""
    x = torch.full(shape, 1e-3, device="cuda")
    x[0, 0] = 2.0
    abc, steps = (1.77, 0.0, 0.0), 4  # 1.77, 3.13, 5.55, 9.8: what enters a step stays below 5.65
    p, m = torch.zeros_like(x), torch.zeros_like(x)
    fq.fp8q_muon(p, x, m, lr=1.0, scale=1.0, nesterov=False, steps=steps, coefficients=abc)
    want = x.double() / x.double().norm() * 1.77 ** steps
    assert ((-p.double() - want).norm() <= steps * 2.0 ** -12 * want.norm())
