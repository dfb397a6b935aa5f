"""Newton-Schulz products on the GPU within the accuracy that include/fp8q.h states: absolute bounds, taken from the
model of their roundings, with parameters in FP32 so that no rounding to BF16 covers an error."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
from test_gpu_muon import by_products
from test_muon_accuracy import FAR, NEAR, SHAPES, made, off, stated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", NEAR + FAR)
@pytest.mark.parametrize("shape", SHAPES + [(2, 1000, 300), (1, 512, 2048), (1, 4100, 70)])
def test_distance_from_the_exact_result(shape, kind):
    """One step of Muon from zero parameters and momentum with lr = scale = 1: the parameters are minus the update, which
    FP32 rounds by 2^-24 of a value (the matrix itself as well, before: it is what the exact result is of)."""
    u = made(shape, kind, sum(shape) + 1, "cuda").float()
    p, m = torch.zeros_like(u), torch.zeros_like(u)
    fq.fp8q_muon(p, u, m, lr=1.0, scale=1.0, nesterov=False)
    assert torch.equal(m, u)
    assert off(-p.double(), by_products(u)) <= stated(shape, kind)
