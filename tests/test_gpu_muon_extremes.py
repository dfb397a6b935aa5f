"""Muon at the largest sizes: sides of 2^20 and of one, batches past 2^31 elements.

Tolerances are those of test_gpu_muon.py, and for sums of K products as long as these what FP32 may lose of A: at most K / 512
additions follow each other in a lane (32 products in one, 16 parts of a sum), each off by 2^-24 of a sum that is no
larger than one; a step multiplies an error of A by at most |b| + 2 |c| = 9 and X by 2 at the most, five steps by 9 * (2^5 - 1)."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
from test_gpu_muon import allowed, matrices

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("shape", [(1, 1 << 20), (1 << 20, 1), (2, (1 << 20) - 3), ((1 << 20) - 1, 3), (70, 1 << 18), (1 << 18, 130)])
def test_long_sides(shape):
    u = matrices(shape, "strong", F32, 7)
    e, norm, inside = allowed(u)
    p, m = torch.zeros_like(u), torch.zeros_like(u)
    c = torch.full(shape, 7.0, device="cuda", dtype=BF16)
    fq.fp8q_muon(p, u, m, lr=1.0, scale=1.0, nesterov=False, copy=c)
    assert torch.equal(m, u) and torch.equal(c, p.bfloat16())
    assert (-p.double() - e).norm() <= inside + max(shape) / 512 * 2.0 ** -24 * 9 * 31 * norm
    out = fq.fp8q_orthogonalize(u)
    assert torch.equal(out, (-p).bfloat16())  # the same products, rounded once


def test_more_than_32_bits_of_parameters():
    """The last matrix of 132 takes the step that it takes alone; the others' gradients are zeros."""
    G, P, Q = 132, 4096, 4096
    g = torch.zeros((G, P, Q), device="cuda", dtype=BF16)
    g[-1] = matrices((P, Q), "normal", BF16, 1)
    p, m = torch.ones((G, P, Q), device="cuda"), torch.zeros((G, P, Q), device="cuda")
    c = torch.zeros((G, P, Q), device="cuda", dtype=BF16)
    fq.fp8q_muon(p, g, m, lr=0.5, scale=1.0, weight_decay=0.5, steps=1, copy=c)
    q, n = torch.ones((P, Q), device="cuda"), torch.zeros((P, Q), device="cuda")
    fq.fp8q_muon(q, g[-1].contiguous(), n, lr=0.5, scale=1.0, weight_decay=0.5, steps=1)
    assert (p[:-1] == 0.75).all() and not m[:-1].any() and (c[:-1] == 0.75).all()
    assert torch.equal(m[-1], n) and torch.equal(c[-1], p[-1].bfloat16())
    # other tiles, the same sums: FP16 roundings in between may differ, by 1e-3 of the update's norm
    assert (p[-1] - q).double().norm() <= 1e-3 * (q - 0.75).double().norm() + 2.0 ** -23 * P
