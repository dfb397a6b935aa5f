"""The accuracy that include/fp8q.h states for Newton-Schulz products, by the model of the kernels' roundings in 64 bits
(`by_products` of test_gpu_muon.py), without a GPU.  The bounds are absolute: parts of the result's norm."""
import math

import pytest
import torch

from test_gpu_muon import by_products

NEAR = ["normal", "strong", "few", "alike", "one 0.05", "one 0.005", "one 0.002"]  # singular values within a factor of 500
FAR = ["one 0.001", "one 0.0001"]


def made(shape, kind, seed, device="cpu"):
    """float64 [G, P, Q]: noise; 16 directions of falling strength or 5 over noise; rows alike but for noise; one direction over
    noise whose largest singular value is a given part of it."""
    G, P, Q = shape
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x = n(G, P, Q)
    if kind == "strong":
        r = min(16, P, Q)
        x = torch.matmul(n(G, P, r) * 0.7 ** torch.arange(r), n(G, r, Q)) + 0.5 * x
    elif kind == "few":
        r = min(5, P, Q)
        x = 0.02 * x + torch.matmul(n(G, P, r), n(G, r, Q)) / math.sqrt(r)
    elif kind == "alike":
        x = 1.0 + 0.05 * x
    elif kind != "normal":
        one = torch.matmul(n(G, P, 1), n(G, 1, Q))
        x = one / one.flatten(1).norm(dim=1)[:, None, None] + float(kind[4:]) * x / (math.sqrt(P) + math.sqrt(Q))
    return x.to(device)


def stated(shape, kind):
    """include/fp8q.h: the largest distance from the exact result, over its norm."""
    m = min(shape[1:])
    if kind in NEAR:
        return 1e-3 if m >= 128 else max(1e-3, 0.3 / m)
    return 7e-3 if m >= 128 else max(7e-3, min(0.1, 1.0 / m))


def off(got, want):
    return ((got - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).max().item()


# batches of the small ones: their errors differ from matrix to matrix, as few roundings average out
SHAPES = [(200, 2, 2), (200, 3, 40), (200, 8, 8), (100, 8, 64), (100, 64, 8), (60, 16, 16), (30, 16, 256), (30, 33, 32), (10, 64, 64),
          (4, 100, 300), (4, 128, 128), (2, 129, 500), (2, 256, 256)]


@pytest.mark.parametrize("kind", NEAR + FAR)
@pytest.mark.parametrize("shape", SHAPES)
def test_model_stays_within_what_is_stated(shape, kind):
    x = made(shape, kind, sum(shape))
    assert off(by_products(x, rounded=True), by_products(x)) <= stated(shape, kind)
